// The 4-bit paged cache's writers and reader: rotation table, rotation with
// the append, gather.
//
// Bound: HBM for many tokens (2 bytes read and 0.5625 written per k and v
// element, 2 + 2 per q element), latency for few.  A lane holds 8 elements of a
// head, so 16 lanes hold a head of 128 and a warp works on two heads at a time
// (four of 64); its rotations and norm weights are the same for every head of the
// token and stay in registers.  The 8 are consecutive (one 16-byte load, one word
// of key codes), or, where all of a head is rotated in the half layout, 4 of each
// half, so that an element's partner is in the same lane: no exchange, no element
// normed twice (8178 tokens: 62 us without that form, 44 with it).  A token's
// heads are shared by as many warps as it takes to fill the GPU: one warp a token
// for long prompts, one warp for every two heads of a single token.
// Measured (32 q and 8 kv heads of 128, norms): 8178 tokens 44.5 us, 4.0 TB/s; what
// is left is instructions (issue slots 66 % busy; every lane of a group computes the
// group's two IEEE divisions) and latency at 17.6 warps a SM.  All six forms spill at
// 96 registers (12 to 28 bytes stored a thread).  Heads rotated in part or in pairs
// take 60.5 to 64.5 us: an element's partner is in another lane or is normed twice.
// One token 3.1 us.  Gather of 8178 tokens 9.3 us (output in L2), of one 2.6 us.
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

namespace bi {

namespace {

constexpr int kAppendWarps = 4;                      // warps of a CTA
constexpr int kAppendCtas = 5;                       // CTAs a SM that the registers are to allow (4 and 6: 48 us for 44)
constexpr int kBatch = 3;                            // heads (of a lane) in flight
constexpr int kWholeBatch = 4;                       // the same for heads that are rotated whole; a power of two (2: 48 us)

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

// The parameter word of a group with elements lo .. hi.
__device__ __forceinline__ uint32_t group_param(float lo, float hi)
{
    return bf16_rne_bits(__fdiv_rn(__fsub_rn(hi, lo), 15.0f)) | (__float_as_uint(lo) & 0xFFFF0000u);
}

__device__ __forceinline__ bool quick_scale(float s) { return s >= kQuotientMinScale && s <= 0x1p64f; }

// What codes_of needs to divide by a group's scale.
__device__ __forceinline__ float group_inverse(uint32_t param)
{
    const float s = bf16_lo(param);
    return quick_scale(s) ? __fdiv_rn(1.0f, s) : 0.0f;
}

// Codes of N elements x (bf16 values) of a group, r its group_inverse.  (x - z) / s by quotient_rn: r = RN(1 / s), and s has
// 8 bits, so that no quotient lies close enough to the middle of two fp32 numbers to be rounded another way.
template <int N>
__device__ __forceinline__ void codes_of(const float (&x)[N], uint32_t param, float r, uint32_t (&c)[N])
{
    const float s = bf16_lo(param), z = bf16_hi(param);
    if (quick_scale(s)) {
#pragma unroll
        for (int e = 0; e < N; ++e)                        // rne, as in code_byte; below 15.5: s is off by 2^-9 at most
            c[e] = __float_as_uint(__fadd_rn(quotient_rn(__fsub_rn(x[e], z), s, r), 12582912.0f)) & 15u;
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            c[e] = s > 0.0f ? static_cast<uint32_t>(max(0, min(15, __float2int_rn(__fdiv_rn(__fsub_rn(x[e], z), s))))) : 0u;
    }
}

// Codes of the lane's 8 elements x (bf16 values), one nibble each in element
// order, and the parameters of their group of 64 (8 lanes).
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
    param = group_param(lo, hi);
    uint32_t c[8], codes = 0;
    codes_of(x, param, group_inverse(param), c);
#pragma unroll
    for (int e = 0; e < 8; ++e) codes |= c[e] << (4 * e);
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

// Two fp32 to bf16, rounded to nearest even, in one conversion.
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The lane's 8 elements of a q or k head, normed and rotated, as bf16 pairs.
template <int D, bool INTERLEAVED>
struct Rotation {
    static constexpr int L = D / 8;
    float co[8], si[8];                                    // out = x co + partner si, si with its sign
    int rot, swap, from[4], lane, d;
    bool full;

    __device__ __forceinline__ Rotation(const float2 *cs, int rot_, int lane_) : rot(rot_), lane(lane_)
    {
        const int l = lane % L, half = rot / 2;
        d = 8 * l;
        full = rot == D;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            co[e] = 1.0f;
            si[e] = 0.0f;
            if (d + e < rot) {
                const bool second = INTERLEAVED ? e % 2 : d + e >= half;
                const float2 f = __ldg(cs + (INTERLEAVED ? (d + e) / 2 : second ? d + e - half : d + e));
                co[e] = f.x;
                si[e] = second ? f.y : -f.y;
            }
        }
        // partner words of the half layout: word j's comes from word j ^ swap of lane from[j]
        swap = half / 2 % 4;                               // 0 or 2: half is a multiple of 4
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int w = 4 * l + j + (d + 2 * j >= half ? -half / 2 : half / 2);
            from[j] = (lane - l) + min(max(w, 0) / 4, L - 1);
        }
    }

    __device__ __forceinline__ void partner(const uint32_t (&w)[4], uint32_t (&p)[4]) const
    {
        if constexpr (INTERLEAVED) {
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = (w[j] >> 16) | (w[j] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = __shfl_sync(0xffffffffu, swap ? w[j ^ 2] : w[j], from[j]);
        }
    }

    // wn, wp: the norm's weights and the partners'
    __device__ __forceinline__ void apply(uint32_t (&w)[4], bool norm, const uint32_t (&wn)[4], const uint32_t (&wp)[4],
                                          float eps) const
    {
        uint32_t p[4];
        partner(w, p);
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = elem(w, e);
            y[e] = elem(p, e);
        }
        if (norm) {
            uint32_t pn[4];                                // the words D / 2 further
#pragma unroll
            for (int j = 0; j < 4; ++j) pn[j] = __shfl_xor_sync(0xffffffffu, w[j], L / 2);
            const float sum = square_sum<D>(w, pn);
            const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(sum / D, eps)));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = __fmul_rn(__fmul_rn(x[e], r), elem(wn, e));
                y[e] = __fmul_rn(__fmul_rn(y[e], r), elem(wp, e));
            }
        }
        if (full) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __fadd_rn(__fmul_rn(x[e], co[e]), __fmul_rn(y[e], si[e]));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (d + e < rot) x[e] = __fadd_rn(__fmul_rn(x[e], co[e]), __fmul_rn(y[e], si[e]));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = to_bf16x2(x[2 * j], x[2 * j + 1]);
    }
};

// Heads that are rotated whole in the half layout, normed and rotated: a lane
// has 4 elements of each half, which are one another's partners, and elements go
// two at a time.  out(step, whether the lane has a head, bf16 pairs of both halves).
template <int D, class Out>
__device__ __forceinline__ void turn_whole(const uint16_t *src, const float2 *cs, const uint16_t *norm, float eps, int heads,
                                           int s0, int s1, Out out)
{
    constexpr int L = D / 8, HEADS = 32 / L;
    const int lane = threadIdx.x & 31, l = lane % L, hl = lane / L;
    src += hl * D + 4 * l;
    auto load = [&](int s, uint2 (&w)[2]) {
        w[0] = w[1] = make_uint2(0u, 0u);
        if (s < s1 && s * HEADS + hl < heads) {
            w[0] = __ldcs(reinterpret_cast<const uint2 *>(src + s * (HEADS * D)));
            w[1] = __ldcs(reinterpret_cast<const uint2 *>(src + s * (HEADS * D) + D / 2));
        }
    };
    uint2 ahead[kWholeBatch][2];
#pragma unroll
    for (int i = 0; i < kWholeBatch; ++i) load(s0 + i, ahead[i]);
    f2 co[2], si[2], wn[2][2];                             // pairs of elements; norm weights of both halves
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(cs + 4 * l) + i);
        co[i] = pk(f.x, f.z);
        si[i] = pk(f.y, f.w);
    }
    if (norm) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(norm + 4 * l + h * (D / 2)));
            wn[h][0] = pk(bf16_lo(v.x), bf16_hi(v.x));
            wn[h][1] = pk(bf16_lo(v.y), bf16_hi(v.y));
        }
    }
    const bool up = l & (L / 2);
    auto pairs = [](const uint2 &w, f2 (&x)[2]) {
        x[0] = pk(bf16_lo(w.x), bf16_hi(w.x));
        x[1] = pk(bf16_lo(w.y), bf16_hi(w.y));
    };
#pragma unroll 1
    for (int begin = s0; begin < s1; begin += kWholeBatch) {
        uint2 now[kWholeBatch][2];
#pragma unroll
        for (int i = 0; i < kWholeBatch; ++i) {
            now[i][0] = ahead[i][0];
            now[i][1] = ahead[i][1];
            load(begin + kWholeBatch + i, ahead[i]);
        }
        // 1 / sqrt of the batch's heads: lane i of each four computes the i-th, so that one root and one division serve all
        float r = 0.0f;
        if (norm) {
#pragma unroll
            for (int i = 0; i < kWholeBatch; ++i) {
                // the order of square_sum: halves, neighbours, then halves again; a lane has two neighbours' sums
                f2 x[2][2];
                pairs(now[i][0], x[0]);
                pairs(now[i][1], x[1]);
                const float2 p = upk(fma2(x[1][0], x[1][0], mul2(x[0][0], x[0][0]))),
                             q = upk(fma2(x[1][1], x[1][1], mul2(x[0][1], x[0][1])));
                const float a = __fadd_rn(p.x, p.y), b = __fadd_rn(q.x, q.y);
                float v = __fadd_rn(up ? b : a, __shfl_xor_sync(0xffffffffu, up ? a : b, L / 2));
#pragma unroll
                for (int o = L / 4; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
                v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, L / 2));
                if (lane % kWholeBatch == i) r = v;
            }
            r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(r / D, eps)));
        }
#pragma unroll
        for (int i = 0; i < kWholeBatch; ++i) {
            const int s = begin + i;
            if (s >= s1) break;
            f2 x[2][2];
            pairs(now[i][0], x[0]);
            pairs(now[i][1], x[1]);
            if (norm) {
                const float ri = __shfl_sync(0xffffffffu, r, (lane & ~(kWholeBatch - 1)) + i);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[h][j] = mul2(mul2(x[h][j], pk(ri, ri)), wn[h][j]);
            }
            uint32_t w[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // the sums one at a time: a packed sum of packed products is contracted to one rounding
                const float2 ac = upk(mul2(x[0][j], co[j])), bs = upk(mul2(x[1][j], si[j])),
                             bc = upk(mul2(x[1][j], co[j])), as = upk(mul2(x[0][j], si[j]));
                w[0][j] = to_bf16x2(__fsub_rn(ac.x, bs.x), __fsub_rn(ac.y, bs.y));
                w[1][j] = to_bf16x2(__fadd_rn(bc.x, as.x), __fadd_rn(bc.y, as.y));
            }
            out(s, s * HEADS + hl < heads, w);
        }
    }
}

// Codes and parameters of a key whose halves a lane holds 4 elements of, w as turn_whole gives them: the word of the
// first half for the lane and its odd neighbour (of the second half, if the lane is the odd one), and the parameters of
// the lane's group (of the group of the half that the lane's own half of the lanes stands for, if there are two).
template <int D>
__device__ __forceinline__ uint32_t quantise_whole(const uint32_t (&w)[2][2], uint32_t &param)
{
    constexpr int L = D / 8;
    const int l = threadIdx.x % L;
    float x[2][4], lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[h][2 * j] = bf16_lo(w[h][j]);
            x[h][2 * j + 1] = bf16_hi(w[h][j]);
        }
        lo[h] = fminf(fminf(x[h][0], x[h][1]), fminf(x[h][2], x[h][3]));
        hi[h] = fmaxf(fmaxf(x[h][0], x[h][1]), fmaxf(x[h][2], x[h][3]));
    }
    const bool up = l & (L / 2);
    float a, b;                                            // the smallest and the largest of the lane's group
    if (D == 2 * kKv4Group) {
        a = fminf(up ? lo[1] : lo[0], __shfl_xor_sync(0xffffffffu, up ? lo[0] : lo[1], L / 2));
        b = fmaxf(up ? hi[1] : hi[0], __shfl_xor_sync(0xffffffffu, up ? hi[0] : hi[1], L / 2));
    } else {
        a = fminf(lo[0], lo[1]);
        b = fmaxf(hi[0], hi[1]);
    }
#pragma unroll
    for (int o = kKv4Group / 16; o > 0; o >>= 1) {
        a = fminf(a, __shfl_xor_sync(0xffffffffu, a, o));
        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
    param = group_param(a, b);
    const float r = group_inverse(param);
    uint32_t other = param, half[2];
    float r_other = r;
    if (D == 2 * kKv4Group) {
        other = __shfl_xor_sync(0xffffffffu, param, L / 2);
        r_other = __shfl_xor_sync(0xffffffffu, r, L / 2);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bool mine = up == (h == 1);
        uint32_t c[4];
        codes_of(x[h], mine ? param : other, mine ? r : r_other, c);
        half[h] = c[0] | c[2] << 4 | c[1] << 16 | c[3] << 20;   // where elements 0-3 stand in a key word; 4-7 8 bits up
    }
    const uint32_t got = __shfl_xor_sync(0xffffffffu, l & 1 ? half[0] : half[1], 1);
    return l & 1 ? got | half[1] << 8 : half[0] | got << 8;
}

// `parts` warps a token, a run of steps each; a step is HEADS heads of one
// kind: first the steps of the q heads, then of k, then of v.
// LAYOUT: of the rotation's pairs; WHOLE: HALF with all of a head rotated.
enum { WHOLE, HALF, INTERLEAVED };
template <int D, int LAYOUT>
__global__ void __launch_bounds__(32 * kAppendWarps, kAppendCtas) rope_append_kernel(RopeAppendArgs a, int parts, int pdl)
{
    constexpr int L = D / 8, HEADS = 32 / L, G = D / kKv4Group;
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const int lane = threadIdx.x & 31, d = lane % L * 8, hl = lane / L;
    const int64_t id = (static_cast<int64_t>(blockIdx.x) * (32 * kAppendWarps) + threadIdx.x) >> 5;
    const int t = static_cast<int>(id / parts), part = static_cast<int>(id - static_cast<int64_t>(t) * parts);
    if (t >= a.c.T) return;
    const int q_steps = (a.Hq + HEADS - 1) / HEADS, kv_steps = (a.c.Hkv + HEADS - 1) / HEADS;
    const int steps = q_steps + 2 * kv_steps, per = (steps + parts - 1) / parts;
    const int first = part * per, last = min(steps, first + per);
    const Kv4Token tok = kv4_token(a.c, t);
    if (tok.b < 0) return;
    uint16_t *const qo = a.q_out + (static_cast<int64_t>(t) * a.Hq + hl) * D + d;
    if (tok.pos < 0 || tok.pos >= min(a.n_pos, a.c.max_kv)) {
        for (int step = first; step < min(last, q_steps); ++step)
            if (step * HEADS + hl < a.Hq) *reinterpret_cast<uint4 *>(qo + step * (HEADS * D)) = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const float2 *const cs = a.rope + static_cast<int64_t>(tok.pos) * (a.rot / 2);
    // The steps of one kind that are this warp's, kBatch loads ahead: body(step of the kind, whether the lane has a head,
    // the lane's words).
    auto each = [&](const uint16_t *base, int64_t ld, int heads, int begin, int n, auto body) {
        const int s0 = max(first - begin, 0), s1 = min(last - begin, n);
        if (s0 >= s1) return;
        const uint16_t *src = base + t * ld + hl * D + d;
        auto load = [&](int s) {
            return s < s1 && s * HEADS + hl < heads ? __ldcs(reinterpret_cast<const uint4 *>(src + s * (HEADS * D)))
                                                    : make_uint4(0u, 0u, 0u, 0u);
        };
        uint4 ahead[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) ahead[i] = load(s0 + i);
#pragma unroll 1
        for (int s = s0; s < s1; ++s) {
            uint32_t w[4] = {ahead[0].x, ahead[0].y, ahead[0].z, ahead[0].w};
#pragma unroll
            for (int i = 0; i + 1 < kBatch; ++i) ahead[i] = ahead[i + 1];
            ahead[kBatch - 1] = load(s + kBatch);
            body(s, s * HEADS + hl < heads, w);
        }
    };
    const int P = 1 << a.c.page_shift;
    const Places<D> at(d, tok.pos & (P - 1), P);
    unsigned char *const block = kv4_block<D>(a.c, max(tok.page, 0), hl);
    auto quantise = [&](int s, bool there, const uint32_t (&w)[4], bool key) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = elem(w, e);
        uint32_t param;
        const uint32_t codes = quantise8(x, param);
        if (!there || tok.page < 0) return;
        unsigned char *to = block + s * (HEADS * Kv4Layout::block(P, D));
        if (key) {
            *reinterpret_cast<uint32_t *>(to + at.key) = key_word(codes);
        } else {
            *reinterpret_cast<uint16_t *>(to + at.value) = static_cast<uint16_t>(codes);
            *reinterpret_cast<uint16_t *>(to + at.value + 4) = static_cast<uint16_t>(codes >> 16);
        }
        if (d % kKv4Group == 0) *reinterpret_cast<uint32_t *>(to + at.par + (key ? 0 : 4 * G)) = param;
    };
    if constexpr (LAYOUT == WHOLE) {
        const int l = lane % L;
        uint16_t *const qw = a.q_out + (static_cast<int64_t>(t) * a.Hq + hl) * D + 4 * l;
        if (first < q_steps)
            turn_whole<D>(a.q + t * a.ldq, cs, a.q_norm, a.eps, a.Hq, first, min(last, q_steps),
                          [&](int s, bool there, const uint32_t (&w)[2][2]) {
                              if (!there) return;
                              uint16_t *to = qw + s * (HEADS * D);
                              *reinterpret_cast<uint2 *>(to) = make_uint2(w[0][0], w[0][1]);
                              *reinterpret_cast<uint2 *>(to + D / 2) = make_uint2(w[1][0], w[1][1]);
                          });
        const int k0 = max(first - q_steps, 0), k1 = min(last - q_steps, kv_steps);
        if (k0 < k1) {
            const Places<D> word(4 * (l & ~1) + (l & 1) * (D / 2), tok.pos & (P - 1), P);
            turn_whole<D>(a.k + t * a.ldk, cs, a.k_norm, a.eps, a.c.Hkv, k0, k1,
                          [&](int s, bool there, const uint32_t (&w)[2][2]) {
                              uint32_t param;
                              const uint32_t codes = quantise_whole<D>(w, param);
                              if (!there || tok.page < 0) return;
                              unsigned char *to = block + s * (HEADS * Kv4Layout::block(P, D));
                              *reinterpret_cast<uint32_t *>(to + word.key) = codes;
                              if (l % 8 == 0) *reinterpret_cast<uint32_t *>(to + at.par) = param;
                          });
        }
    } else {
        const Rotation<D, LAYOUT == INTERLEAVED> turn(cs, a.rot, lane);
        auto weights = [&](const uint16_t *norm, uint32_t (&wn)[4], uint32_t (&wp)[4]) {
            const uint4 v = norm ? __ldg(reinterpret_cast<const uint4 *>(norm + d)) : make_uint4(0u, 0u, 0u, 0u);
            wn[0] = v.x, wn[1] = v.y, wn[2] = v.z, wn[3] = v.w;
            turn.partner(wn, wp);
        };
        uint32_t wn[4], wp[4];
        if (first < q_steps) {
            weights(a.q_norm, wn, wp);
            each(a.q, a.ldq, a.Hq, 0, q_steps, [&](int s, bool there, uint32_t (&w)[4]) {
                turn.apply(w, a.q_norm != nullptr, wn, wp, a.eps);
                if (there) *reinterpret_cast<uint4 *>(qo + s * (HEADS * D)) = make_uint4(w[0], w[1], w[2], w[3]);
            });
        }
        if (first < q_steps + kv_steps && last > q_steps) {
            weights(a.k_norm, wn, wp);
            each(a.k, a.ldk, a.c.Hkv, q_steps, kv_steps, [&](int s, bool there, uint32_t (&w)[4]) {
                turn.apply(w, a.k_norm != nullptr, wn, wp, a.eps);
                quantise(s, there, w, true);
            });
        }
    }
    each(a.v, a.ldv, a.c.Hkv, q_steps + kv_steps, kv_steps,
         [&](int s, bool there, uint32_t (&w)[4]) { quantise(s, there, w, false); });
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
                ko[e] = to_bf16x2(y[0], y[1]);
                vo[e] = to_bf16x2(y[2], y[3]);
            }
            k = make_uint4(ko[0], ko[1], ko[2], ko[3]);
            v = make_uint4(vo[0], vo[1], vo[2], vo[3]);
        }
        const int64_t to = (static_cast<int64_t>(t) * c.Hkv + h) * D + d;
        *reinterpret_cast<uint4 *>(k_out + to) = k;
        *reinterpret_cast<uint4 *>(v_out + to) = v;
    }
}

// Warps that share a token's `steps` heads: as many as the SMs hold at once.  (1024 tokens of 40 heads: 9.0 us with 2
// warps a token, 11.9 with 3, which are a second wave; 256 tokens 5.2 with 8, 6.1 with 5.)
int parts_of(int T, int steps, int sms)
{
    const int want = kAppendWarps * kAppendCtas * sms / T;
    const int parts = want < 1 ? 1 : want < steps ? want : steps;
    const int per = (steps + parts - 1) / parts;
    return (steps + per - 1) / per;
}

template <int D, int LAYOUT>
cudaError_t launch_append(const RopeAppendArgs &a, int sms, bool pdl, cudaStream_t stream)
{
    constexpr int HEADS = 32 / (D / 8);
    const int parts = parts_of(a.c.T, (a.Hq + HEADS - 1) / HEADS + 2 * ((a.c.Hkv + HEADS - 1) / HEADS), sms);
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
    return cudaLaunchKernelEx(&cfg, rope_append_kernel<D, LAYOUT>, a, parts, pdl ? 1 : 0);
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
    const int layout = interleaved ? INTERLEAVED : a.rot == D ? WHOLE : HALF;
    if (D == 64)
        return layout == WHOLE  ? launch_append<64, WHOLE>(a, sms, pdl, stream)
               : layout == HALF ? launch_append<64, HALF>(a, sms, pdl, stream)
                                : launch_append<64, INTERLEAVED>(a, sms, pdl, stream);
    return layout == WHOLE  ? launch_append<128, WHOLE>(a, sms, pdl, stream)
           : layout == HALF ? launch_append<128, HALF>(a, sms, pdl, stream)
                            : launch_append<128, INTERLEAVED>(a, sms, pdl, stream);
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
