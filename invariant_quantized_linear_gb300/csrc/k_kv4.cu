// The 4-bit paged cache's writers and reader: rotation table, rotation with
// the append, gather.
//
// Bound: HBM for many tokens (2 bytes read and 0.5625 written per k and v
// element, 2 + 2 per q element), latency for few.  A lane holds 8 consecutive
// elements of a head (one 16-byte load, one word of key codes), so 16 lanes
// hold a head of 128 and a warp works on two heads at a time (four of 64); its
// rotations and norm weights are the same for every head of the token and stay
// in registers.  A token's heads are shared by as many warps as it takes to
// fill the GPU: one warp a token for long prompts, one warp for every two heads
// of a single token.
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

namespace bi {

namespace {

constexpr int kAppendWarps = 4;                      // warps of a CTA
constexpr int kBatch = 4;                            // heads (of a lane) in flight
constexpr int kTargetWarps = 16;                     // warps a SM that a call is cut into, if it has the heads

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

__device__ __forceinline__ float elem(const uint32_t (&w)[4], int e)
{
    return e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
}

// The sum of a head's squares in the order of the definition: halves (d and
// d + D / 2), neighbours, then halves again.  w: the lane's 8 elements, pn: those
// D / 2 further (or back).  Squares of bf16 values are exact, so the first step
// is one fused multiply-add.  Each later step halves the values a lane holds as
// long as it holds several: lanes that would add the same pairs share them.
template <int D>
__device__ __forceinline__ float square_sum(const uint32_t (&w)[4], const uint32_t (&pn)[4])
{
    constexpr int L = D / 8;
    const int lane = threadIdx.x & 31;
    float p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float x = elem(w, 2 * j + i), y = elem(pn, 2 * j + i);
            s[i] = __fmaf_rn(y, y, __fmul_rn(x, x));
        }
        p[j] = __fadd_rn(s[0], s[1]);
    }
    // a lane (of the first L / 2; the others hold the same) has neighbours' sums 4 l .. 4 l + 3
    const bool up = lane & (L / 4), one = lane & (L / 8);
    float a = up ? p[2] : p[0], b = up ? p[3] : p[1];
    a = __fadd_rn(a, __shfl_xor_sync(0xffffffffu, up ? p[0] : p[2], L / 4));
    b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, up ? p[1] : p[3], L / 4));
    float v = __fadd_rn(one ? b : a, __shfl_xor_sync(0xffffffffu, one ? a : b, L / 8));
    if constexpr (D == 128) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 1));
    v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, L / 4));
    return __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, L / 8));
}

// Codes of the lane's 8 elements x (bf16 values), one nibble each in element
// order, and the parameters of their group of 64 (8 lanes).  (x - z) / s by
// quotient_rn: r = RN(1 / s), and s has 8 bits, so that no quotient lies close
// enough to the middle of two fp32 numbers to be rounded another way.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], uint32_t &param)
{
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        lo = fminf(lo, x[e]);
        hi = fmaxf(hi, x[e]);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const uint32_t sb = bf16_rne_bits(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float s = __uint_as_float(sb << 16);
    param = sb | (__float_as_uint(lo) & 0xFFFF0000u);
    uint32_t codes = 0;
    if (s >= kQuotientMinScale && s <= 0x1p64f) {
        const float r = __fdiv_rn(1.0f, s);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = __fadd_rn(quotient_rn(__fsub_rn(x[e], lo), s, r), 12582912.0f);   // rne, as in code_byte
            codes |= static_cast<uint32_t>(min(15, __float_as_int(u) - 0x4B400000)) << (4 * e);
        }
    } else if (s > 0.0f) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            codes |= static_cast<uint32_t>(max(0, min(15, __float2int_rn(__fdiv_rn(__fsub_rn(x[e], lo), s))))) << (4 * e);
    }
    return codes;
}

// Nibbles in element order to the order of a key word: element i at 4 (i / 2 + 4 (i % 2)).
__device__ __forceinline__ uint32_t key_word(uint32_t c)
{
    const uint32_t even = c & 0x0F0F0F0Fu, odd = (c >> 4) & 0x0F0F0F0Fu;       // a nibble in each byte
    const uint32_t e = (even | (even >> 4)) & 0x00FF00FFu, o = (odd | (odd >> 4)) & 0x00FF00FFu;
    return __byte_perm(e, o, 0x6420);
}

__device__ __forceinline__ uint32_t key_word_inverse(uint32_t k)
{
    const uint32_t e = __byte_perm(k, 0u, 0x4140), o = __byte_perm(k, 0u, 0x4342);
    const uint32_t even = (e | (e << 4)) & 0x0F0F0F0Fu, odd = (o | (o << 4)) & 0x0F0F0F0Fu;
    return even | (odd << 4);
}

// Where the lane's 8 elements (from d on) stand in a block: a key word, and two half words of a position pair's values.
template <int D>
struct Places {
    int key, value, par;
    __device__ __forceinline__ Places(int d, int slot, int P)
    {
        constexpr int G = D / kKv4Group;
        key = slot * Kv4Layout::k_row(D) + ((d % 64) / 16 * G + d / 64) * 8 + (d % 16) / 8 * 4;
        value = Kv4Layout::v_off(P, D) + slot / 2 * Kv4Layout::v_pair(D) + ((d % 64) / 8 * G + d / 64) * 8 + slot % 2 * 2;
        par = Kv4Layout::p_off(P, D) + slot * Kv4Layout::p_row(D) + d / 64 * 4;
    }
};

// Warps parts t .. of token t, a run of heads each: q heads 0 .. Hq - 1, then the kv heads' k, then their v.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kAppendWarps) rope_append_kernel(RopeAppendArgs a, int parts, int pdl)
{
    constexpr int L = D / 8, HEADS = 32 / L, G = D / kKv4Group;
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const int lane = threadIdx.x & 31, l = lane % L, d = 8 * l;
    const int64_t id = (static_cast<int64_t>(blockIdx.x) * (32 * kAppendWarps) + threadIdx.x) >> 5;
    const int t = static_cast<int>(id / parts), part = static_cast<int>(id - static_cast<int64_t>(t) * parts);
    if (t >= a.c.T) return;
    const int heads = a.Hq + 2 * a.c.Hkv, steps = (heads + HEADS - 1) / HEADS;
    const int per = (steps + parts - 1) / parts, first = part * per, last = min(steps, first + per);

    // head h of the token: what it is and where it stands
    auto source = [&](int h) {
        return h < a.Hq ? a.q + t * a.ldq + h * D
                        : h < a.Hq + a.c.Hkv ? a.k + t * a.ldk + (h - a.Hq) * D
                                             : a.v + t * a.ldv + (h - a.Hq - a.c.Hkv) * D;
    };
    uint4 raw[kBatch];
    auto load = [&](int step) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = (step + i) * HEADS + lane / L;
            raw[i] = step + i < last && h < heads ? *reinterpret_cast<const uint4 *>(source(h) + d) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load(first);
    const Kv4Token tok = kv4_token(a.c, t);
    if (tok.b < 0) return;
    if (tok.pos < 0 || tok.pos >= a.n_pos) {
        for (int step = first; step < last; ++step) {
            const int h = step * HEADS + lane / L;
            if (h < a.Hq)
                *reinterpret_cast<uint4 *>(a.q_out + (static_cast<int64_t>(t) * a.Hq + h) * D + d) = make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    const int P = 1 << a.c.page_shift;
    const Places<D> at(d, tok.pos & (P - 1), P);

    // the lane's rotations: out = x co + partner si, si with its sign
    const int half = a.rot / 2;
    float co[8], si[8];
    const float2 *cs = a.rope + static_cast<int64_t>(tok.pos) * half;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        co[e] = 1.0f;
        si[e] = 0.0f;
        if (d + e < a.rot) {
            const bool second = INTERLEAVED ? e % 2 : d + e >= half;
            const float2 f = __ldg(cs + (INTERLEAVED ? (d + e) / 2 : second ? d + e - half : d + e));
            co[e] = f.x;
            si[e] = second ? f.y : -f.y;
        }
    }
    // the partner words of the half layout: word j's comes from word j ^ swap of lane from[j]
    const int swap = half / 2 % 4;                    // 0 or 2: half is a multiple of 4
    int from[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int w = 4 * l + j + (d + 2 * j >= half ? -half / 2 : half / 2);
        from[j] = (lane - l) + min(max(w, 0) / 4, L - 1);
    }
    uint32_t wq[4] = {}, wk[4] = {}, wqp[4], wkp[4];
    if (a.q_norm) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(a.q_norm + d));
        wq[0] = v.x, wq[1] = v.y, wq[2] = v.z, wq[3] = v.w;
    }
    if (a.k_norm) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(a.k_norm + d));
        wk[0] = v.x, wk[1] = v.y, wk[2] = v.z, wk[3] = v.w;
    }
    auto partner = [&](const uint32_t (&w)[4], uint32_t (&p)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = __shfl_sync(0xffffffffu, swap ? w[j ^ 2] : w[j], from[j]);
    };
    if constexpr (!INTERLEAVED) {
        partner(wq, wqp);
        partner(wk, wkp);
    }

    for (int step0 = first; step0 < last; step0 += kBatch) {
        uint4 now[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) now[i] = raw[i];
        if (step0 + kBatch < last) load(step0 + kBatch);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (step0 + i >= last) break;
            const int h = (step0 + i) * HEADS + lane / L;
            const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.c.Hkv, is_v = !is_q && !is_k;
            const uint32_t w[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = elem(w, e);
            if ((step0 + i) * HEADS < a.Hq + a.c.Hkv) {   // some q or k in the warp
                uint32_t p[4];
                if constexpr (!INTERLEAVED) partner(w, p);
                const bool norm = is_q ? a.q_norm != nullptr : is_k && a.k_norm != nullptr;
                float y[8];                                // partners
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = INTERLEAVED ? elem(w, e ^ 1) : elem(p, e);
                if (a.q_norm || a.k_norm) {
                    uint32_t pn[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) pn[j] = __shfl_xor_sync(0xffffffffu, w[j], L / 2);
                    const float sum = square_sum<D>(w, pn);
                    const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(sum / D, a.eps)));
                    if (norm) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float u = is_q ? elem(wq, e) : elem(wk, e);
                            const float v = INTERLEAVED ? (is_q ? elem(wq, e ^ 1) : elem(wk, e ^ 1))
                                                        : (is_q ? elem(wqp, e) : elem(wkp, e));
                            x[e] = __fmul_rn(__fmul_rn(x[e], r), u);
                            y[e] = __fmul_rn(__fmul_rn(y[e], r), v);
                        }
                    }
                }
                if (!is_v) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (d + e < a.rot) x[e] = __fadd_rn(__fmul_rn(x[e], co[e]), __fmul_rn(y[e], si[e]));
                }
            }
            const uint32_t o[4] = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                   pack_bf16x2(x[6], x[7])};
            if (is_q)
                *reinterpret_cast<uint4 *>(a.q_out + (static_cast<int64_t>(t) * a.Hq + h) * D + d) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            if ((step0 + i + 1) * HEADS <= a.Hq) continue;     // q heads only
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = elem(o, e);
            uint32_t param;
            const uint32_t codes = quantise8(x, param);
            if (is_q || h >= heads || tok.page < 0) continue;
            unsigned char *block = kv4_block<D>(a.c, tok.page, is_k ? h - a.Hq : h - a.Hq - a.c.Hkv);
            if (is_k) {
                *reinterpret_cast<uint32_t *>(block + at.key) = key_word(codes);
            } else {
                *reinterpret_cast<uint16_t *>(block + at.value) = static_cast<uint16_t>(codes);
                *reinterpret_cast<uint16_t *>(block + at.value + 4) = static_cast<uint16_t>(codes >> 16);
            }
            if (d % kKv4Group == 0) *reinterpret_cast<uint32_t *>(block + at.par + (is_k ? 0 : 4 * G)) = param;
        }
    }
}

// A lane holds 8 elements of a (token, kv head), the key's and the value's.
template <int D>
__global__ void __launch_bounds__(128) kv4_gather_kernel(Kv4View c, uint16_t *k_out, uint16_t *v_out, int parts)
{
    constexpr int L = D / 8, HEADS = 32 / L, G = D / kKv4Group;
    const int lane = threadIdx.x & 31, d = lane % L * 8;
    const int64_t id = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5;
    const int t = static_cast<int>(id / parts), part = static_cast<int>(id - static_cast<int64_t>(t) * parts);
    if (t >= c.T) return;
    const Kv4Token tok = kv4_token(c, t);
    if (tok.b < 0) return;
    const int P = 1 << c.page_shift;
    const Places<D> at(d, tok.pos & (P - 1), P);
    const int steps = (c.Hkv + HEADS - 1) / HEADS, per = (steps + parts - 1) / parts;
    for (int step = part * per; step < min(steps, (part + 1) * per); ++step) {
        const int h = step * HEADS + lane / L;
        if (h >= c.Hkv) break;
        uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
        if (tok.page >= 0) {
            const unsigned char *block = kv4_block<D>(c, tok.page, h);
            const uint32_t kc = key_word_inverse(*reinterpret_cast<const uint32_t *>(block + at.key));
            const uint32_t vc = *reinterpret_cast<const uint16_t *>(block + at.value) |
                                static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(block + at.value + 4)) << 16;
            const uint32_t kp = *reinterpret_cast<const uint32_t *>(block + at.par),
                           vp = *reinterpret_cast<const uint32_t *>(block + at.par + 4 * G);
            uint32_t ko[4], vo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int sh = 4 * (2 * e + i);
                    y[i] = __fmaf_rn(bf16_lo(kp), static_cast<float>((kc >> sh) & 15u), bf16_hi(kp));
                    y[2 + i] = __fmaf_rn(bf16_lo(vp), static_cast<float>((vc >> sh) & 15u), bf16_hi(vp));
                }
                ko[e] = pack_bf16x2(y[0], y[1]);
                vo[e] = pack_bf16x2(y[2], y[3]);
            }
            k = make_uint4(ko[0], ko[1], ko[2], ko[3]);
            v = make_uint4(vo[0], vo[1], vo[2], vo[3]);
        }
        const int64_t to = (static_cast<int64_t>(t) * c.Hkv + h) * D + d;
        *reinterpret_cast<uint4 *>(k_out + to) = k;
        *reinterpret_cast<uint4 *>(v_out + to) = v;
    }
}

// Warps that share a token's `steps` heads so that T tokens fill `sms` SMs.
int parts_of(int T, int steps, int sms)
{
    const int want = (kTargetWarps * sms + T - 1) / T;
    const int parts = want < steps ? want : steps;
    const int per = (steps + parts - 1) / parts;
    return (steps + per - 1) / per;
}

template <int D, bool INTERLEAVED>
cudaError_t launch_append(const RopeAppendArgs &a, int sms, bool pdl, cudaStream_t stream)
{
    constexpr int HEADS = 32 / (D / 8);
    const int parts = parts_of(a.c.T, (a.Hq + 2 * a.c.Hkv + HEADS - 1) / HEADS, sms);
    const int64_t warps = static_cast<int64_t>(a.c.T) * parts;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((warps + kAppendWarps - 1) / kAppendWarps));
    cfg.blockDim = dim3(32 * kAppendWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, rope_append_kernel<D, INTERLEAVED>, a, parts, pdl ? 1 : 0);
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

cudaError_t launch_rope_append_kv4(const RopeAppendArgs &a, int D, bool interleaved, int sms, bool pdl,
                                   cudaStream_t stream)
{
    if (D == 64)
        return interleaved ? launch_append<64, true>(a, sms, pdl, stream) : launch_append<64, false>(a, sms, pdl, stream);
    return interleaved ? launch_append<128, true>(a, sms, pdl, stream) : launch_append<128, false>(a, sms, pdl, stream);
}

cudaError_t launch_kv4_gather(const Kv4View &c, int D, uint16_t *k_out, uint16_t *v_out, int sms, cudaStream_t stream)
{
    const int per_warp = 32 / (D / 8), parts = parts_of(c.T, (c.Hkv + per_warp - 1) / per_warp, sms);
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(c.T) * parts + 3) / 4);
    if (D == 64)
        kv4_gather_kernel<64><<<grid, 128, 0, stream>>>(c, k_out, v_out, parts);
    else
        kv4_gather_kernel<128><<<grid, 128, 0, stream>>>(c, k_out, v_out, parts);
    return cudaGetLastError();
}

}  // namespace bi
