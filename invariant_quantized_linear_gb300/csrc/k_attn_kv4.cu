// Attention of new tokens over the 4-bit paged cache.
//
// A cached element is z + s c with a 4-bit code c and (s, z) shared by 64
// elements of its position, so scores and outputs split into a product with
// the codes, which tensor cores take, and rank-one terms of the minima:
//   q . k   = sum_g s_g (q_g . c_g) + z_g sum(q_g)
//   sum p v = sum (p s_g) (c_g + z_g / s_g)       (g: the element's group)
// The codes need no arithmetic to become operands: a nibble in the low bits of
// an f16 word is the subnormal c 2^-24 and one nibble up c 2^-20, both exact
// and taken by the tensor cores as they are.  One AND makes two operands, one
// shift serves four.  The factors 16 of the odd nibbles are undone in q (keys)
// and in the result (values).
//
// Operands are transposed, S^T = K q^T and O^T = V^T P^T, so that positions
// (16 of an mma.m16n8k16) and head elements fill the rows, and the few query
// rows the columns, 8 at a time: a decode step of a group of 4 heads wastes
// half a tile instead of three quarters.  The cache's layout puts what a lane
// needs of a 16-position tile into 16 bytes of its own, so a warp copies its
// codes to shared memory (cp.async) and reads them back with no exchange.
//
// q is scaled by a power of two a row so that its largest element is just
// below 2^15: in f16 it is exact down to 2^-24 of that.  The weights p s go
// into f16 (11 bits) with the row's largest s 2^15 or just below, so that what
// is lost lies 2^-29 below the largest weight.  Everything else is fp32.  The
// minima are weighted by the rounded p s times z / s, not by p: a weight's
// rounding then moves the whole value z + s c, and not only its s c, which may
// be much larger than the value.  A group without a scale (all its elements
// equal) has codes 0 and takes |z| / 8 in its place.
//
// Work: a CTA takes kSpan positions of one kv head for a block of query rows;
// warp w takes 64 positions in each of kRounds rounds and keeps the running
// maximum and sum; the eight warps are joined in order, and a second launch
// joins the spans in order.  A row's result is made of the same operations
// whatever else is in the call: spans are counted from position 0, and neither
// maxima nor scales look at a position that the row does not see.
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

#include <cuda_fp16.h>

namespace bi {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlock = 64;                          // positions of a warp and round
constexpr int kRounds = 2;
constexpr int kSpan = kBlock * kWarps * kRounds;    // positions of a CTA
constexpr int kMinExp = -100;                       // least exponent that value scales are normalised to
constexpr float kMinScale = 0x1p-110f;              // groups of smaller scale count as zeros

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t smem, const void *gmem)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem), "l"(gmem) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem), "l"(gmem) : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Four operands of a code word: nibble pairs (0, 4), (1, 5), (2, 6), (3, 7), the odd ones 16-fold.
__device__ __forceinline__ void code_operands(uint32_t w, uint32_t (&o)[4])
{
    o[0] = w & 0x000F000Fu;
    o[1] = w & 0x00F000F0u;
    w >>= 8;
    o[2] = w & 0x000F000Fu;
    o[3] = w & 0x00F000F0u;
}

__device__ __forceinline__ float pow2_int(int e) { return __int_as_float((e + 127) << 23); }   // -126 .. 127

// Shared memory of a CTA for head size D and NB blocks of 8 query rows.
template <int D, int NB>
struct Plan {
    static constexpr int G = D / kKv4Group;
    static constexpr int R = 8 * NB;                       // query rows
    static constexpr int kPiece = D / 8;                   // bytes of a lane's share of 8 positions (16 or 8)
    static constexpr int kCodes = 8 * 32 * kPiece;         // 64 positions of keys (or values)
    static constexpr int kPar = kBlock * 8 * G;            // their parameters
    static constexpr int kPrep = kBlock * 8 * G;           // value scales and z / s of the round, fp32
    static constexpr int kWarp = 2 * kCodes + 2 * kPar + kPrep;
    static constexpr int kQRow = 2 * D + 8;                // bytes of a query row in f16; the 8 spread the banks
    static constexpr int kO = R * D * 4;                   // one warp's outputs; they take the place of its codes
    static constexpr int kQ = kWarps * kWarp;
    static constexpr int kT = kQ + R * kQRow;              // sums of q per row and group
    static constexpr int kF = kT + R * G * 4;              // factor per row
    static constexpr int kM = kF + R * 4;                  // maxima [warp][row]
    static constexpr int kL = kM + kWarps * R * 4;         // sums [warp][row]
    static constexpr int kBytes = kL + kWarps * R * 4;
    static_assert(kO <= kWarp, "a warp's outputs fit in the place of its codes");
};

template <int BYTES>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[BYTES / 4])
{
    if constexpr (BYTES == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
    else
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}

// Query rows r0 .. of a kv head to shared memory: f16 elements scaled by a
// power of two, odd element pairs divided by 16; the sums and the factor that
// turn products with codes into scores in units of log2.
template <int D, int NB>
__device__ __forceinline__ void stage_queries(const AttnKv4Args &a, unsigned char *smem, int t0, int hk, int G, int r0,
                                              int rows)
{
    using P = Plan<D, NB>;
    constexpr int E = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int rl = warp; rl < P::R; rl += kWarps) {
        const int r = r0 + rl;
        uint32_t w[E / 2] = {};
        if (r < rows) {
            const uint16_t *src = a.q + (t0 + r / G) * a.ldq + (hk * G + r % G) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) w[e] = *reinterpret_cast<const uint32_t *>(src + 2 * e);
        }
        float x[E], top = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
            top = fmaxf(top, fabsf(x[e]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // up = 2^(14 - floor(log2 top)), kept in fp32's range; zero and subnormal rows take the largest
        const int ex = max(-100, min(127, static_cast<int>(__float_as_uint(top) >> 23) - 127));
        const float up = pow2_int(14 - ex);
        float sum = 0.0f;
        uint32_t h[E / 2];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] *= up;
            sum += x[e];
        }
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            const int pair = (lane * E / 2 + e) % 4;
            const float f = pair % 2 ? 0.0625f : 1.0f;
            h[e] = pack_f16x2(x[2 * e] * f, x[2 * e + 1] * f);
            *reinterpret_cast<uint32_t *>(smem + P::kQ + rl * P::kQRow + (lane * E + 2 * e) * 2) = h[e];
        }
#pragma unroll
        for (int o = 16 / P::G; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane % (32 / P::G) == 0)
            *reinterpret_cast<float *>(smem + P::kT + (rl * P::G + lane / (32 / P::G)) * 4) = sum * 0x1p-24f;
        if (lane == 0)   // scores = factor * (products with 2^-24 c and up q)
            *reinterpret_cast<float *>(smem + P::kF + rl * 4) =
                fmaxf(fminf(a.scale * 1.4426950408889634f * 0x1p10f * pow2_int(ex), 0x1p126f), 0x1p-126f);
    }
}

template <int D, int NB>
__global__ void __launch_bounds__(kThreads, D * NB > 128 ? 1 : 2) attn_kv4_span_kernel(AttnKv4Args a, int row_blocks, int spans, int pdl)
{
    using P = Plan<D, NB>;
    constexpr int G = P::G, W = P::kPiece / 4, TILES = kBlock / 16;
    extern __shared__ __align__(16) unsigned char smem[];
    const Kv4View &c = a.c;
    const int span = blockIdx.x / row_blocks, rb = blockIdx.x - span * row_blocks, hk = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (pdl) pdl_wait();
    pdl_launch_dependents();
    // the sequence: its token rows t0 .. t0 + nq - 1, row r = token r / GH, head r % GH of the kv head
    const int GH = a.Hq / c.Hkv;
    const int t0 = max(0, __ldg(c.cu_q + b)), t1 = min(c.T, __ldg(c.cu_q + b + 1)), len = __ldg(c.kv_len + b);
    const int new_tokens = __ldg(c.cu_q + b + 1) - __ldg(c.cu_q + b);
    const int nq = min(t1 - t0, c.max_q), rows = nq * GH, r0 = rb * P::R;
    if (r0 >= rows) return;
    const int r_last = min(rows, r0 + P::R) - 1;
    const int first = len - new_tokens;                             // position of token t0
    // positions that row r sees: first + r / GH + 1, within 0 .. max_kv
    const int n_most = min(c.max_kv, first + r_last / GH + 1), n_least = min(c.max_kv, first + r0 / GH + 1);
    const int p0 = span * kSpan;
    if (p0 >= n_most && (span > 0 || n_most > 0)) return;

    const uint32_t base = smem_u32(smem), my = base + warp * P::kWarp;
    const int PS = 1 << c.page_shift;
    // copies of a round's keys with parameters, or values; returns nothing for pages that are not there
    auto page_of = [&](int p) {                                     // lane i < 4: page of positions p + 16 i ..
        const int x = p + 16 * (lane & 3);
        return x < n_most ? kv4_page(c, b, x) : -1;
    };
    auto copy_keys = [&](int p, int pages, int par) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int page = __shfl_sync(0xffffffffu, pages, j >> 1);
            if (page >= 0)
                cp_async<P::kPiece>(my + j * 32 * P::kPiece + lane * P::kPiece,
                                    kv4_block<D>(c, page, hk) + ((p + 8 * j + g) & (PS - 1)) * Kv4Layout::k_row(D) +
                                        t * P::kPiece);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int x = 32 * j + lane, page = __shfl_sync(0xffffffffu, pages, x >> 4);
            if (page >= 0)
                cp_async<8 * G>(my + 2 * P::kCodes + par * P::kPar + x * 8 * G,
                                kv4_block<D>(c, page, hk) + Kv4Layout::p_off(PS, D) +
                                    ((p + x) & (PS - 1)) * Kv4Layout::p_row(D));
        }
        cp_commit();
    };
    auto copy_values = [&](int p, int pages) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int page = __shfl_sync(0xffffffffu, pages, j >> 1);
            if (page >= 0)
                cp_async<P::kPiece>(my + P::kCodes + j * 32 * P::kPiece + lane * P::kPiece,
                                    kv4_block<D>(c, page, hk) + Kv4Layout::v_off(PS, D) +
                                        (((p + 8 * j) & (PS - 1)) / 2 + t) * Kv4Layout::v_pair(D) + g * P::kPiece);
        }
        cp_commit();
    };

    int pages = page_of(p0 + warp * kBlock);
    copy_keys(p0 + warp * kBlock, pages, 0);
    copy_values(p0 + warp * kBlock, pages);
    stage_queries<D, NB>(a, smem, t0, hk, GH, r0, rows);
    __syncthreads();

    // this lane's columns: rows 8 nb + 2 t + i of the block
    float f[NB][2], tq[NB][2][G], m[NB][2], l[NB][2], z[NB][2][G];
    int es[NB][2], n_row[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rl = 8 * nb + 2 * t + i, r = r0 + rl;
            f[nb][i] = *reinterpret_cast<const float *>(smem + P::kF + rl * 4);
#pragma unroll
            for (int k = 0; k < G; ++k) {
                tq[nb][i][k] = *reinterpret_cast<const float *>(smem + P::kT + (rl * G + k) * 4);
                z[nb][i][k] = 0.0f;
            }
            m[nb][i] = -INFINITY;
            l[nb][i] = 0.0f;
            es[nb][i] = kMinExp;
            n_row[nb][i] = min(c.max_kv, first + min(r, r_last) / GH + 1);   // idle rows go with the last
        }
    float o[G][4][NB][4];
#pragma unroll
    for (int k = 0; k < G; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[k][e][nb][i] = 0.0f;

#pragma unroll 1
    for (int round = 0; round < kRounds; ++round) {
        const int p = p0 + (round * kWarps + warp) * kBlock;
        if (p >= n_most) break;
        const bool more = round + 1 < kRounds && p + kWarps * kBlock < n_most;
        // every position of the block is there and seen by every row
        const unsigned there = __ballot_sync(0xffffffffu, pages >= 0) & 15u;
        const bool full = there == 15u && p + kBlock <= n_least;
        cp_wait<1>();
        __syncwarp();
        const uint32_t par = my + 2 * P::kCodes + (round & 1) * P::kPar;

        // ---- scores
        float s[TILES][NB][4];
#pragma unroll
        for (int tile = 0; tile < TILES; ++tile) {
            uint32_t k0[W], k1[W], p_lo[2 * G], p_hi[2 * G];
            lds_words<P::kPiece>(my + (2 * tile) * 32 * P::kPiece + lane * P::kPiece, k0);
            lds_words<P::kPiece>(my + (2 * tile + 1) * 32 * P::kPiece + lane * P::kPiece, k1);
            lds_words<8 * G>(par + (16 * tile + g) * 8 * G, p_lo);
            lds_words<8 * G>(par + (16 * tile + 8 + g) * 8 * G, p_hi);
#pragma unroll
            for (int k = 0; k < G; ++k) {
                float acc[NB][4];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[nb][i] = 0.0f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t x0[4], x1[4];
                    code_operands(k0[2 * k + j], x0);
                    code_operands(k1[2 * k + j], x1);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            uint32_t q[2];
                            lds_words<8>(base + P::kQ + (8 * nb + g) * P::kQRow + (64 * k + 16 * t + 8 * j + 4 * h) * 2, q);
                            mma_f16_16816(acc[nb], x0[2 * h], x1[2 * h], x0[2 * h + 1], x1[2 * h + 1], q[0], q[1]);
                        }
                }
                const float s_lo = bf16_lo(p_lo[k]), z_lo = bf16_hi(p_lo[k]), s_hi = bf16_lo(p_hi[k]), z_hi = bf16_hi(p_hi[k]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u = __fmaf_rn(i < 2 ? z_lo : z_hi, tq[nb][i & 1][k], k ? s[tile][nb][i] : 0.0f);
                        s[tile][nb][i] = __fmaf_rn(i < 2 ? s_lo : s_hi, acc[nb][i], u);
                    }
            }
        }
        // positions that a row does not see, or that are on no page
        if (!full) {
#pragma unroll
            for (int tile = 0; tile < TILES; ++tile)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!((there >> tile) & 1u) || p + 16 * tile + 8 * (i >> 1) + g >= n_row[nb][i & 1])
                            s[tile][nb][i] = -INFINITY;
        }
        // keys are read: the next round's may come; params are double-buffered
        __syncwarp();
        int next_pages = -1;
        if (more) {
            next_pages = page_of(p + kWarps * kBlock);
            copy_keys(p + kWarps * kBlock, next_pages, (round + 1) & 1);
        } else {
            cp_commit();
        }

        // ---- the values' scales and z / s, two positions a lane; nothing for positions that no row sees
        const uint32_t prep = my + 2 * P::kCodes + 2 * P::kPar;
        int e_all = kMinExp;
#pragma unroll
        for (int x = lane; x < kBlock; x += 32) {
            uint32_t w[2 * G];
            lds_words<8 * G>(par + x * 8 * G, w);
            const bool seen = ((there >> (x >> 4)) & 1u) && p + x < n_most;
            float out[2 * G];
#pragma unroll
            for (int k = 0; k < G; ++k) {
                const float zv = bf16_hi(w[G + k]);
                float sv = bf16_lo(w[G + k]);
                sv = sv > 0.0f ? sv : 0.125f * fabsf(zv);
                const bool some = seen && sv >= kMinScale;
                out[2 * k] = some ? sv : 0.0f;
                out[2 * k + 1] = some ? __fdividef(zv, sv) : 0.0f;
                e_all = max(e_all, static_cast<int>(__float_as_uint(out[2 * k]) >> 23) - 126);   // out < 2^e
            }
            if constexpr (G == 2)
                asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(prep + x * 16), "f"(out[0]), "f"(out[1]),
                             "f"(out[2]), "f"(out[3])
                             : "memory");
            else
                asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(prep + x * 8), "f"(out[0]), "f"(out[1]) : "memory");
        }
        __syncwarp();

        // ---- running maxima of the scores and of the value scales' exponents
        float c15[NB][2], mm[NB][2];
        {
            int e_row[NB][2];
            if (full) {
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) e_all = max(e_all, __shfl_xor_sync(0xffffffffu, e_all, x));
            } else {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) e_row[nb][0] = e_row[nb][1] = kMinExp;
#pragma unroll
                for (int tile = 0; tile < TILES; ++tile)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t w[2 * G];
                        lds_words<8 * G>(prep + (16 * tile + 8 * half + g) * 8 * G, w);
                        uint32_t top = w[0];
                        if constexpr (G == 2) top = max(top, w[2]);
                        const int e = static_cast<int>(top >> 23) - 126;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (s[tile][nb][2 * half + i] > -INFINITY) e_row[nb][i] = max(e_row[nb][i], e);
                    }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float top = -INFINITY;
#pragma unroll
                    for (int tile = 0; tile < TILES; ++tile) top = fmaxf(top, fmaxf(s[tile][nb][i], s[tile][nb][2 + i]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    int e = e_all;
                    if (!full) {
                        e = e_row[nb][i];
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) e = max(e, __shfl_xor_sync(0xffffffffu, e, x));
                    }
                    const float m_new = fmaxf(m[nb][i], f[nb][i] * top);         // in units of log2
                    const int e_new = max(es[nb][i], e);
                    // a row that has seen nothing keeps its zeros
                    const float fl = m[nb][i] == -INFINITY ? 0.0f : ex2(m[nb][i] - m_new);
                    const float fo = fl * pow2_int(max(-126, es[nb][i] - e_new));
                    l[nb][i] *= fl;
#pragma unroll
                    for (int k = 0; k < G; ++k) {
                        z[nb][i][k] *= fo;
#pragma unroll
                        for (int e4 = 0; e4 < 4; ++e4) {
                            o[k][e4][nb][i] *= fo;
                            o[k][e4][nb][2 + i] *= fo;
                        }
                    }
                    m[nb][i] = m_new;
                    es[nb][i] = e_new;
                    c15[nb][i] = pow2_int(15 - e_new);
                    mm[nb][i] = m_new == -INFINITY ? 0.0f : m_new;
                }
        }

        // ---- weights and values
        cp_wait<1>();
        __syncwarp();
#pragma unroll
        for (int tile = 0; tile < TILES; ++tile) {
            uint32_t v0[W], v1[W], p_lo[2 * G], p_hi[2 * G];         // p: scale and z / s
            lds_words<P::kPiece>(my + P::kCodes + (2 * tile) * 32 * P::kPiece + lane * P::kPiece, v0);
            lds_words<P::kPiece>(my + P::kCodes + (2 * tile + 1) * 32 * P::kPiece + lane * P::kPiece, v1);
            lds_words<8 * G>(prep + (16 * tile + g) * 8 * G, p_lo);
            lds_words<8 * G>(prep + (16 * tile + 8 + g) * 8 * G, p_hi);
            uint32_t pb[G][NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = ex2(__fmaf_rn(s[tile][nb][i], f[nb][i & 1], -mm[nb][i & 1]));
                    l[nb][i & 1] += w[i];
                    w[i] *= c15[nb][i & 1];
                }
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    const float s_lo = __uint_as_float(p_lo[2 * k]), s_hi = __uint_as_float(p_hi[2 * k]);
                    const __half2 h_lo = __floats2half2_rn(w[0] * s_lo, w[1] * s_lo);
                    const __half2 h_hi = __floats2half2_rn(w[2] * s_hi, w[3] * s_hi);
                    const float2 r_lo = __half22float2(h_lo), r_hi = __half22float2(h_hi);
                    const float z_lo = __uint_as_float(p_lo[2 * k + 1]), z_hi = __uint_as_float(p_hi[2 * k + 1]);
                    z[nb][0][k] = __fmaf_rn(r_hi.x, z_hi, __fmaf_rn(r_lo.x, z_lo, z[nb][0][k]));
                    z[nb][1][k] = __fmaf_rn(r_hi.y, z_hi, __fmaf_rn(r_lo.y, z_lo, z[nb][1][k]));
                    pb[k][nb][0] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h_lo));
                    pb[k][nb][1] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h_hi));
                }
            }
#pragma unroll
            for (int k = 0; k < G; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t x0[4], x1[4];
                    code_operands(v0[2 * k + j], x0);
                    code_operands(v1[2 * k + j], x1);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma_f16_16816(o[k][2 * j + h][nb], x0[2 * h], x0[2 * h + 1], x1[2 * h], x1[2 * h + 1],
                                          pb[k][nb][0], pb[k][nb][1]);
                }
        }
        __syncwarp();
        if (more) copy_values(p + kWarps * kBlock, next_pages);
        else cp_commit();
        pages = next_pages;
    }
    cp_wait<0>();

    // ---- join the lanes that share a row, then the warps
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], x);
#pragma unroll
                for (int k = 0; k < G; ++k) z[nb][i][k] += __shfl_xor_sync(0xffffffffu, z[nb][i][k], x);
            }
            const int rl = 8 * nb + 2 * t + i;
            if (g == 0) {
                *reinterpret_cast<float *>(smem + P::kM + (warp * P::R + rl) * 4) = m[nb][i];
                *reinterpret_cast<float *>(smem + P::kL + (warp * P::R + rl) * 4) = l[nb][i];
            }
        }
    __syncwarp();                                                    // the warp's codes are read
    float *ow = reinterpret_cast<float *>(smem + warp * P::kWarp);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // z carries 2^(15 - es), o 2^-24 of that (the odd elements 2^-20): undone in two steps
            const float up = pow2_int(es[nb][i] - 20);
#pragma unroll
            for (int k = 0; k < G; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        v[2 * h] = __fmaf_rn(o[k][2 * j + h][nb][i], 0x1p24f, z[nb][i][k]) * 0x1p5f * up;
                        v[2 * h + 1] = __fmaf_rn(o[k][2 * j + h][nb][2 + i], 0x1p20f, z[nb][i][k]) * 0x1p5f * up;
                    }
                    *reinterpret_cast<float4 *>(ow + (8 * nb + 2 * t + i) * D + 64 * k + 8 * g + 4 * j) =
                        make_float4(v[0], v[1], v[2], v[3]);
                }
        }
    __syncthreads();
    const float *sm = reinterpret_cast<const float *>(smem + P::kM), *sl = reinterpret_cast<const float *>(smem + P::kL);
    for (int i = threadIdx.x; i < P::R * D / 4; i += kThreads) {
        const int rl = i / (D / 4), d = i % (D / 4) * 4, r = r0 + rl;
        if (r >= rows) break;
        const int tok = r / GH, n = min(c.max_kv, first + tok + 1);
        if (p0 >= n && (span > 0 || n > 0)) continue;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w * P::R + rl]);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (top > -INFINITY) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float e = ex2(sm[w * P::R + rl] - top);
                sum = __fmaf_rn(e, sl[w * P::R + rl], sum);
                const float4 x = *reinterpret_cast<const float4 *>(smem + w * P::kWarp + (rl * D + d) * 4);
                v.x = __fmaf_rn(e, x.x, v.x);
                v.y = __fmaf_rn(e, x.y, v.y);
                v.z = __fmaf_rn(e, x.z, v.z);
                v.w = __fmaf_rn(e, x.w, v.w);
            }
        }
        const int64_t at = static_cast<int64_t>(t0 + tok) * a.Hq + hk * GH + r % GH;
        if (n <= kSpan) {
            const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
            *reinterpret_cast<uint2 *>(a.o + at * D + d) =
                make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        } else {
            float *part = static_cast<float *>(a.ws) + (at * spans + span) * (D + 4);
            *reinterpret_cast<float4 *>(part + 4 + d) = v;
            if (d == 0) *reinterpret_cast<float2 *>(part) = make_float2(top, sum);
        }
    }
}

// One warp per (token, q head) whose token sees more than one span: the spans' results in order.
template <int D>
__global__ void __launch_bounds__(128) attn_kv4_join_kernel(AttnKv4Args a, int spans)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t id = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5;
    const int t = static_cast<int>(id / a.Hq), h = static_cast<int>(id - static_cast<int64_t>(t) * a.Hq);
    pdl_wait();
    if (t >= a.c.T) return;
    const int b = kv4_sequence(a.c, t);
    if (b < 0) return;
    const int begin = __ldg(a.c.cu_q + b), end = __ldg(a.c.cu_q + b + 1);
    uint16_t *o = a.o + (static_cast<int64_t>(t) * a.Hq + h) * D + lane * E;
    const int n = min(a.c.max_kv, __ldg(a.c.kv_len + b) - (end - t) + 1);
    if (t - begin >= a.c.max_q) {
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0;
        return;
    }
    if (n <= kSpan) return;
    const int C = (n + kSpan - 1) / kSpan;
    const float *part = static_cast<const float *>(a.ws) + (static_cast<int64_t>(t) * a.Hq + h) * spans * (D + 4);
    float top = -INFINITY;
    for (int c = lane; c < C; c += 32) top = fmaxf(top, part[static_cast<int64_t>(c) * (D + 4)]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    float sum = 0.0f, v[E] = {};
    if (top > -INFINITY) {
#pragma unroll 8
        for (int c = 0; c < C; ++c) {
            const float *pc = part + static_cast<int64_t>(c) * (D + 4);
            const float2 ml = *reinterpret_cast<const float2 *>(pc);
            const float w = ex2(ml.x - top);
            sum = __fmaf_rn(w, ml.y, sum);
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = __fmaf_rn(w, pc[4 + lane * E + e], v[e]);
        }
    }
    const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
#pragma unroll
    for (int e = 0; e < E / 2; ++e)
        *reinterpret_cast<uint32_t *>(o + 2 * e) = pack_bf16x2(v[2 * e] * inv, v[2 * e + 1] * inv);
}

int spans_of(int max_kv) { return (max_kv + kSpan - 1) / kSpan; }

template <int D, int NB>
cudaError_t launch_span(const AttnKv4Args &a, int spans, bool pdl, cudaStream_t stream)
{
    const int row_blocks = (a.c.max_q * (a.Hq / a.c.Hkv) + 8 * NB - 1) / (8 * NB);
    const int64_t x = static_cast<int64_t>(row_blocks) * spans;
    if (x > 0x7FFFFFFF) return cudaErrorInvalidValue;
    constexpr int bytes = Plan<D, NB>::kBytes;
    const cudaError_t e =
        cudaFuncSetAttribute(attn_kv4_span_kernel<D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(x), static_cast<unsigned>(a.c.Hkv), static_cast<unsigned>(a.c.B));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attn_kv4_span_kernel<D, NB>, a, row_blocks, spans, pdl ? 1 : 0);
}

}  // namespace

size_t attention_kv4_workspace(int Hq, int Hkv, int D, int B, int T, int max_q, int max_kv)
{
    (void)Hkv, (void)B, (void)max_q;
    const int spans = spans_of(max_kv);
    return spans == 1 ? 16 : static_cast<size_t>(T) * Hq * spans * (D + 4) * sizeof(float);
}

cudaError_t launch_attention_kv4(const AttnKv4Args &a, int D, bool pdl, cudaStream_t stream)
{
    const int spans = spans_of(a.c.max_kv);
    const bool few = a.c.max_q * (a.Hq / a.c.Hkv) <= 8;
    cudaError_t e = D == 64 ? (few ? launch_span<64, 1>(a, spans, pdl, stream) : launch_span<64, 2>(a, spans, pdl, stream))
                            : (few ? launch_span<128, 1>(a, spans, pdl, stream) : launch_span<128, 2>(a, spans, pdl, stream));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(a.c.T) * a.Hq + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return D == 64 ? cudaLaunchKernelEx(&cfg, attn_kv4_join_kernel<64>, a, spans)
                   : cudaLaunchKernelEx(&cfg, attn_kv4_join_kernel<128>, a, spans);
}

}  // namespace bi
