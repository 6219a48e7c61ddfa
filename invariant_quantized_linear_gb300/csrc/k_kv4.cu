// The 4-bit paged cache's writers and reader: rotation table, rotation with
// the append, gather.
//
// Bound: HBM for many tokens (2 bytes read and 0.5625 written per k and v
// element, 2 + 2 per q element), latency for few.  One warp per token and head:
// the head's reductions (norm, block minima and maxima) stay inside the warp.
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

namespace bi {

namespace {

constexpr int kAppendWarps = 8;

__global__ void __launch_bounds__(256) rope_table_kernel(const double *inv_freq, int n_freq, float amp, int n_pos,
                                                         float2 *rope)
{
    const int64_t n = static_cast<int64_t>(n_pos) * n_freq;
    for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
        const int p = static_cast<int>(i / n_freq), f = static_cast<int>(i - static_cast<int64_t>(p) * n_freq);
        double s, c;
        sincos(p * inv_freq[f], &s, &c);
        rope[i] = make_float2(static_cast<float>(c * amp), static_cast<float>(s * amp));
    }
}

template <int OFF, int STOP>
__device__ __forceinline__ float warp_fold(float v)
{
#pragma unroll
    for (int o = OFF; o >= STOP; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Codes of a head's x[E] per lane (E = D / 32 consecutive elements, bf16 values):
// the group's parameters are reduced over the 16 (D = 128) or 32 (D = 64) lanes
// that hold it.  Returns the codes, E nibbles in element order.
template <int D>
__device__ __forceinline__ void quantise_lane(const float (&x)[D / 32], uint32_t (&code)[D / 32], uint32_t &param)
{
    constexpr int E = D / 32, LANES = kKv4Group / E;
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e) {
        lo = fminf(lo, x[e]);
        hi = fmaxf(hi, x[e]);
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const uint32_t sb = bf16_rne_bits(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float s = __uint_as_float(sb << 16);
    param = sb | (__float_as_uint(lo) & 0xFFFF0000u);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float c = s > 0.0f ? __fdiv_rn(__fsub_rn(x[e], lo), s) : 0.0f;
        code[e] = static_cast<uint32_t>(max(0, min(15, __float2int_rn(c))));
    }
}

template <int D>
__device__ __forceinline__ void store_key(unsigned char *block, int slot, const uint32_t (&code)[D / 32], uint32_t param,
                                          int P)
{
    constexpr int E = D / 32, G = D / kKv4Group;
    const int lane = threadIdx.x & 31, d = lane * E;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int i = (d + e) % 8;
        w |= code[e] << (4 * (i / 2 + 4 * (i % 2)));
    }
#pragma unroll
    for (int o = 1; o < 8 / E; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
    if (d % 8 == 0)
        *reinterpret_cast<uint32_t *>(block + slot * Kv4Layout::k_row(D) + ((d % 64) / 16 * G + d / 64) * 8 +
                                      (d % 16) / 8 * 4) = w;
    if (d % 64 == 0)
        *reinterpret_cast<uint32_t *>(block + Kv4Layout::p_off(P, D) + slot * Kv4Layout::p_row(D) + d / 64 * 4) = param;
}

template <int D>
__device__ __forceinline__ void store_value(unsigned char *block, int slot, const uint32_t (&code)[D / 32],
                                            uint32_t param, int P)
{
    constexpr int E = D / 32, G = D / kKv4Group;
    const int lane = threadIdx.x & 31, d = lane * E;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) w |= code[e] << (4 * ((d + e) % 4));
#pragma unroll
    for (int o = 1; o < 4 / E; o <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, o);
    if (d % 4 == 0)
        *reinterpret_cast<uint16_t *>(block + Kv4Layout::v_off(P, D) + slot / 2 * Kv4Layout::v_pair(D) +
                                      ((d % 64) / 8 * G + d / 64) * 8 + (d % 8) / 4 * 4 + slot % 2 * 2) =
            static_cast<uint16_t>(w);
    if (d % 64 == 0)
        *reinterpret_cast<uint32_t *>(block + Kv4Layout::p_off(P, D) + slot * Kv4Layout::p_row(D) + (G + d / 64) * 4) =
            param;
}

// One warp per (token, head): heads 0 .. Hq - 1 are q, then Hkv of k, then Hkv of v.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kAppendWarps) rope_append_kernel(RopeAppendArgs a, int pdl)
{
    constexpr int E = D / 32;
    __shared__ float sx[kAppendWarps][D];
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, heads = a.Hq + 2 * a.c.Hkv;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kAppendWarps + warp;
    const int t = static_cast<int>(id / heads), h = static_cast<int>(id - static_cast<int64_t>(t) * heads);
    if (t >= a.c.T) return;
    const Kv4Token tok = kv4_token(a.c, t);
    if (tok.b < 0) return;
    const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.c.Hkv;
    const int hk = is_k ? h - a.Hq : h - a.Hq - a.c.Hkv;
    const bool known = tok.pos >= 0 && tok.pos < a.n_pos;
    uint16_t *qo = a.q_out + (static_cast<int64_t>(t) * a.Hq + h) * D + lane * E;
    if (!known || (!is_q && tok.page < 0)) {
        if (is_q) {
#pragma unroll
            for (int e = 0; e < E; ++e) qo[e] = 0;
        }
        return;
    }
    const uint16_t *src = (is_q ? a.q + t * a.ldq + h * D : is_k ? a.k + t * a.ldk + hk * D : a.v + t * a.ldv + hk * D);
    float x[E];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(src + lane * E + 2 * e);
        x[2 * e] = bf16_lo(w);
        x[2 * e + 1] = bf16_hi(w);
    }
    if (is_q || is_k) {
        float *s = sx[warp];
        const uint16_t *w = is_q ? a.q_norm : a.k_norm;
#pragma unroll
        for (int e = 0; e < E; ++e) s[lane * E + e] = x[e];
        __syncwarp();
        if (w) {
            // squares: halves, neighbours, halves again
            float p = 0.0f;
            if (lane < D / 4) {
                const float u0 = s[2 * lane], u1 = s[2 * lane + D / 2], v0 = s[2 * lane + 1], v1 = s[2 * lane + 1 + D / 2];
                p = __fadd_rn(__fadd_rn(__fmul_rn(u0, u0), __fmul_rn(u1, u1)),
                              __fadd_rn(__fmul_rn(v0, v0), __fmul_rn(v1, v1)));
            }
            p = warp_fold<D / 8, 1>(p);
            const float sum = __shfl_sync(0xffffffffu, p, 0);
            const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(sum / D, a.eps)));
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[e] = __fmul_rn(__fmul_rn(x[e], r), __uint_as_float(static_cast<uint32_t>(w[lane * E + e]) << 16));
            __syncwarp();
#pragma unroll
            for (int e = 0; e < E; ++e) s[lane * E + e] = x[e];
            __syncwarp();
        }
        const float2 *cs = a.rope + static_cast<int64_t>(tok.pos) * (a.rot / 2);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = lane * E + e;
            if (d < a.rot) {
                const int half = a.rot / 2;
                const bool second = INTERLEAVED ? (d & 1) : d >= half;
                const int i = INTERLEAVED ? d / 2 : (second ? d - half : d);
                const float o = s[INTERLEAVED ? (d ^ 1) : (second ? d - half : d + half)];
                const float2 f = cs[i];
                x[e] = second ? __fadd_rn(__fmul_rn(x[e], f.x), __fmul_rn(o, f.y))
                              : __fsub_rn(__fmul_rn(x[e], f.x), __fmul_rn(o, f.y));
            }
        }
    }
    if (is_q) {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) *reinterpret_cast<uint32_t *>(qo + 2 * e) = pack_bf16x2(x[2 * e], x[2 * e + 1]);
        return;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = __uint_as_float(bf16_rne_bits(x[e]) << 16);
    uint32_t code[E], param;
    quantise_lane<D>(x, code, param);
    unsigned char *block = kv4_block<D>(a.c, tok.page, hk);
    const int P = 1 << a.c.page_shift, slot = tok.pos & (P - 1);
    if (is_k)
        store_key<D>(block, slot, code, param, P);
    else
        store_value<D>(block, slot, code, param, P);
}

// One warp per (token, kv head), first the key, then the value.
template <int D>
__global__ void __launch_bounds__(256) kv4_gather_kernel(Kv4View c, uint16_t *k_out, uint16_t *v_out)
{
    constexpr int E = D / 32, G = D / kKv4Group;
    const int lane = threadIdx.x & 31;
    const int64_t id = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
    const int t = static_cast<int>(id / c.Hkv), h = static_cast<int>(id - static_cast<int64_t>(t) * c.Hkv);
    if (t >= c.T) return;
    const Kv4Token tok = kv4_token(c, t);
    if (tok.b < 0) return;
    const int d = lane * E;
    uint32_t kw = 0, vw = 0, kp = 0, vp = 0;
    if (tok.page >= 0) {
        const unsigned char *block = kv4_block<D>(c, tok.page, h);
        const int P = 1 << c.page_shift, slot = tok.pos & (P - 1);
        kw = *reinterpret_cast<const uint32_t *>(block + slot * Kv4Layout::k_row(D) + ((d % 64) / 16 * G + d / 64) * 8 +
                                                 (d % 16) / 8 * 4);
        vw = *reinterpret_cast<const uint16_t *>(block + Kv4Layout::v_off(P, D) + slot / 2 * Kv4Layout::v_pair(D) +
                                                 ((d % 64) / 8 * G + d / 64) * 8 + (d % 8) / 4 * 4 + slot % 2 * 2);
        const uint32_t *par =
            reinterpret_cast<const uint32_t *>(block + Kv4Layout::p_off(P, D) + slot * Kv4Layout::p_row(D));
        kp = par[d / 64];
        vp = par[G + d / 64];
    }
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int i = (d + e) % 8;
        k[e] = __fmaf_rn(bf16_lo(kp), static_cast<float>((kw >> (4 * (i / 2 + 4 * (i % 2)))) & 15u), bf16_hi(kp));
        v[e] = __fmaf_rn(bf16_lo(vp), static_cast<float>((vw >> (4 * ((d + e) % 4))) & 15u), bf16_hi(vp));
    }
    const int64_t at = (static_cast<int64_t>(t) * c.Hkv + h) * D + d;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
        *reinterpret_cast<uint32_t *>(k_out + at + 2 * e) = pack_bf16x2(k[2 * e], k[2 * e + 1]);
        *reinterpret_cast<uint32_t *>(v_out + at + 2 * e) = pack_bf16x2(v[2 * e], v[2 * e + 1]);
    }
}

}  // namespace

cudaError_t launch_rope_table(const double *inv_freq, int n_freq, float amp, int n_pos, float2 *rope,
                              cudaStream_t stream)
{
    const int64_t n = static_cast<int64_t>(n_pos) * n_freq;
    const int64_t grid = (n + 255) / 256;
    rope_table_kernel<<<static_cast<unsigned>(grid < 4096 ? grid : 4096), 256, 0, stream>>>(inv_freq, n_freq, amp, n_pos,
                                                                                         rope);
    return cudaGetLastError();
}

cudaError_t launch_rope_append_kv4(const RopeAppendArgs &a, int D, bool interleaved, bool pdl, cudaStream_t stream)
{
    const int64_t warps = static_cast<int64_t>(a.c.T) * (a.Hq + 2 * a.c.Hkv);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((warps + kAppendWarps - 1) / kAppendWarps));
    cfg.blockDim = dim3(32 * kAppendWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    const int p = pdl ? 1 : 0;
    if (D == 64)
        return interleaved ? cudaLaunchKernelEx(&cfg, rope_append_kernel<64, true>, a, p)
                           : cudaLaunchKernelEx(&cfg, rope_append_kernel<64, false>, a, p);
    return interleaved ? cudaLaunchKernelEx(&cfg, rope_append_kernel<128, true>, a, p)
                       : cudaLaunchKernelEx(&cfg, rope_append_kernel<128, false>, a, p);
}

cudaError_t launch_kv4_gather(const Kv4View &c, int D, uint16_t *k_out, uint16_t *v_out, cudaStream_t stream)
{
    const int64_t warps = static_cast<int64_t>(c.T) * c.Hkv;
    const unsigned grid = static_cast<unsigned>((warps + 7) / 8);
    if (D == 64)
        kv4_gather_kernel<64><<<grid, 256, 0, stream>>>(c, k_out, v_out);
    else
        kv4_gather_kernel<128><<<grid, 256, 0, stream>>>(c, k_out, v_out);
    return cudaGetLastError();
}

}  // namespace bi
