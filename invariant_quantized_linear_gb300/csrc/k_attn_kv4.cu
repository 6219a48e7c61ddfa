// Attention of new tokens over the 4-bit paged cache.
//
// One warp per (token, q head) walks the positions that the token sees, in
// order, with the running maximum and sum of the softmax (fp32).
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

namespace bi {

namespace {

template <int D>
__global__ void __launch_bounds__(128) attn_kv4_kernel(AttnKv4Args a)
{
    constexpr int E = D / 32, G = D / kKv4Group;
    const Kv4View &c = a.c;
    const int lane = threadIdx.x & 31, d = lane * E;
    const int64_t id = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5;
    const int t = static_cast<int>(id / a.Hq), h = static_cast<int>(id - static_cast<int64_t>(t) * a.Hq);
    if (t >= c.T) return;
    const Kv4Token tok = kv4_token(c, t);
    if (tok.b < 0) return;
    const int hk = h / (a.Hq / c.Hkv), P = 1 << c.page_shift;
    float q[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __uint_as_float(static_cast<uint32_t>(a.q[t * a.ldq + h * D + d + e]) << 16) * a.scale;
        acc[e] = 0.0f;
    }
    float mx = -INFINITY, sum = 0.0f;
    const int n = min(tok.pos + 1, c.max_kv);
    for (int p = 0; p < n; ++p) {
        const int page = kv4_page(c, tok.b, p);
        if (page < 0) continue;
        const unsigned char *block = kv4_block<D>(c, page, hk);
        const int slot = p & (P - 1);
        const uint32_t kw = *reinterpret_cast<const uint32_t *>(
            block + slot * Kv4Layout::k_row(D) + ((d % 64) / 16 * G + d / 64) * 8 + (d % 16) / 8 * 4);
        const uint32_t vw = *reinterpret_cast<const uint16_t *>(
            block + Kv4Layout::v_off(P, D) + slot / 2 * Kv4Layout::v_pair(D) + ((d % 64) / 8 * G + d / 64) * 8 +
            (d % 8) / 4 * 4 + slot % 2 * 2);
        const uint32_t *par =
            reinterpret_cast<const uint32_t *>(block + Kv4Layout::p_off(P, D) + slot * Kv4Layout::p_row(D));
        const uint32_t kp = par[d / 64], vp = par[G + d / 64];
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = (d + e) % 8;
            const float k = fmaf(bf16_lo(kp), static_cast<float>((kw >> (4 * (i / 2 + 4 * (i % 2)))) & 15u), bf16_hi(kp));
            s = fmaf(q[e], k, s);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float m2 = fmaxf(mx, s), f = expf(mx - m2), w = expf(s - m2);
        mx = m2;
        sum = sum * f + w;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float v = fmaf(bf16_lo(vp), static_cast<float>((vw >> (4 * ((d + e) % 4))) & 15u), bf16_hi(vp));
            acc[e] = acc[e] * f + w * v;
        }
    }
    uint16_t *o = a.o + (static_cast<int64_t>(t) * a.Hq + h) * D + d;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = static_cast<uint16_t>(bf16_rne_bits(sum > 0.0f ? acc[e] / sum : 0.0f));
}

}  // namespace

size_t attention_kv4_workspace(int Hq, int Hkv, int D, int B, int T, int max_q, int max_kv)
{
    (void)Hq, (void)Hkv, (void)D, (void)B, (void)T, (void)max_q, (void)max_kv;
    return 16;
}

cudaError_t launch_attention_kv4(const AttnKv4Args &a, int D, bool pdl, cudaStream_t stream)
{
    (void)pdl;
    const int64_t warps = static_cast<int64_t>(a.c.T) * a.Hq;
    const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
    if (D == 64)
        attn_kv4_kernel<64><<<grid, 128, 0, stream>>>(a);
    else
        attn_kv4_kernel<128><<<grid, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace bi
