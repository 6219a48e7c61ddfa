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
// Work: positions are cut into blocks of 64, chunks of 4 blocks and spans of 4
// chunks, counted from position 0.  A block's result (maximum, sum, weighted
// values) comes from one warp; a chunk folds its blocks in order, a span joins
// its chunks' results under their common maximum, and a row joins its spans the
// same way.  A row's result is this tree whatever else is in the call, since
// neither maxima nor scales look at a position that the row does not see; which
// warp computes what may therefore go by the size of the call:
//   4 warps a CTA, a chunk each, the fold in registers: least work a position,
//     four CTAs a SM overlap one another's latencies;
//   16 warps a CTA, a block each, the fold through shared memory: for calls
//     of few CTAs, where a chunk's four blocks one after the other would be
//     most of the time.
// The CTA that finishes a row block's last span joins the spans (a counter in
// the workspace); a second launch does where a row has many spans or the
// counters do not suffice.
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

#include <cuda_fp16.h>

namespace bi {

namespace {

constexpr int kBlock = 64;                          // positions of a block
constexpr int kChunkBlocks = 4;
constexpr int kChunks = 4;                          // chunks of a span
constexpr int kSpan = kBlock * kChunkBlocks * kChunks;
constexpr int kTiles = kBlock / 16;
constexpr int kMinExp = -100;                       // least exponent that value scales are normalised to
constexpr int kMaxExp = 118;                        // largest that is undone again within fp32
constexpr float kMinScale = 0x1p-110f;              // groups of smaller scale count as zeros
constexpr int kCounters = 16384;                    // row blocks whose spans are counted in the workspace
constexpr int kJoinSpans = 64;                      // spans that a CTA joins itself at most
constexpr size_t kCounterBytes = kCounters * sizeof(int);

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
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Two fp32 lanes in one 64-bit register; each lane of an operation is rounded like the scalar one.
typedef unsigned long long f2;

__device__ __forceinline__ f2 pk(float lo, float hi)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float2 upk(f2 x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}

__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
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

// Shared memory of a CTA of WARPS warps for head size D and NB blocks of 8 query rows.
template <int D, int NB, int WARPS>
struct Plan {
    static constexpr int G = D / kKv4Group;
    static constexpr int R = 8 * NB;                       // query rows
    static constexpr int kPiece = D / 8;                   // bytes of a lane's share of 8 positions (16 or 8)
    static constexpr int kCodes = 8 * 32 * kPiece;         // 64 positions of keys (or values)
    static constexpr int kPar = kBlock * 8 * G;            // their parameters
    static constexpr int kPrep = kBlock * 8 * G;           // value scales and z / s of the block, fp32
    static constexpr int kWarp = 2 * kCodes + 2 * kPar + kPrep;   // parameters of two blocks
    static constexpr int kQRow = 2 * D + 8;                // bytes of a query row in f16; the 8 spread the banks
    static constexpr int kO = R * D * 4;                   // a warp's weighted values take the place of its codes
    static constexpr int kLZ = 32 * 2 * NB * (1 + G) * 4;  // and behind them its lanes' sums (16-warp form)
    static constexpr int kQ = WARPS * kWarp;
    static constexpr int kT = kQ + R * kQRow;              // sums of q per row and group
    static constexpr int kF = kT + R * G * 4;              // factor per row
    static constexpr int kN = kF + R * 4;                  // positions that a row sees
    static constexpr int kM = kN + R * 4;                  // maxima [warp][row]
    static constexpr int kL = kM + WARPS * R * 4;          // sums [chunk][row]
    static constexpr int kZ = kL + kChunks * R * 4;        // weighted minima [chunk][row][group] (16-warp form)
    static constexpr int kFlag = kZ + kChunks * R * G * 4;
    static constexpr int kBytes = kFlag + 16;
    static_assert(kO + kLZ <= kWarp, "a warp's results fit in the place of its codes");
};

template <int BYTES>
__device__ __forceinline__ void lds_words(const unsigned char *p, uint32_t (&w)[BYTES / 4])
{
    if constexpr (BYTES == 16) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    }
}

// D = A(16x16) B(16x8) + D in f16 with fp32 sums; not volatile, so that independent chains may interleave.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The rows of a CTA: query rows r0 .. r_last of one kv head, row r = (token r / GH of the sequence, head r % GH).
struct Rows {
    int t0, first, GH, r0, r_last, hk;
    uint64_t magic;                              // 2^32 / GH + 1: r / GH for r * GH < 2^32
    __device__ __forceinline__ int token(int r) const { return static_cast<int>((r * magic) >> 32); }
};

// Positions that row r sees.
__device__ __forceinline__ int row_positions(const AttnKv4Args &a, const Rows &w, int r)
{
    return min(a.c.max_kv, w.first + w.token(r) + 1);
}

// Query rows to shared memory: f16 elements scaled by a power of two, odd
// element pairs divided by 16; the sums and the factor that turn products with
// codes into scores in units of log2.
template <int D, int NB, int WARPS>
__device__ __forceinline__ void stage_queries(const AttnKv4Args &a, unsigned char *smem, const Rows &rows)
{
    using P = Plan<D, NB, WARPS>;
    constexpr int E = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int rl = warp; rl < P::R; rl += WARPS) {
        const int r = rows.r0 + rl, tok = rows.token(min(r, rows.r_last));
        uint32_t w[E / 2] = {};
        if (r <= rows.r_last) {
            const uint16_t *src = a.q + (rows.t0 + tok) * a.ldq + (rows.hk * rows.GH + r - tok * rows.GH) * D + lane * E;
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
        // up = 2^(14 - floor(log2 top)), kept in fp32's range
        const int ex = max(-100, min(127, static_cast<int>(__float_as_uint(top) >> 23) - 127));
        const float up = pow2_int(14 - ex);
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] *= up;
            sum += x[e];
        }
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            const float f = (lane * E / 2 + e) % 2 ? 0.0625f : 1.0f;
            const __half2 h = __floats2half2_rn(x[2 * e] * f, x[2 * e + 1] * f);
            *reinterpret_cast<__half2 *>(smem + P::kQ + rl * P::kQRow + (lane * E + 2 * e) * 2) = h;
        }
#pragma unroll
        for (int o = 16 / P::G; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane % (32 / P::G) == 0)
            *reinterpret_cast<float *>(smem + P::kT + (rl * P::G + lane / (32 / P::G)) * 4) = sum * 0x1p-24f;
        if (lane == 0) {
            // scores = factor * (products with 2^-24 c and up q); idle rows go with the last
            *reinterpret_cast<float *>(smem + P::kF + rl * 4) =
                fmaxf(fminf(a.scale * 1.4426950408889634f * 0x1p10f * pow2_int(ex), 0x1p126f), 0x1p-126f);
            *reinterpret_cast<int *>(smem + P::kN + rl * 4) = min(a.c.max_kv, rows.first + tok + 1);
        }
    }
}

// The fold of a block's result into a chunk's: weights of the two sides.
__device__ __forceinline__ float fold_weights(float m, float mb, float &wa, float &wb)
{
    const float top = fmaxf(m, mb), ref = top == -INFINITY ? 0.0f : top;
    wa = ex2(m - ref);
    wb = ex2(mb - ref);
    return top;
}

// out[row] from the joined value v (4 elements at d) and sum.
template <int D>
__device__ __forceinline__ void write_out(const AttnKv4Args &a, int64_t at, int d, const float4 &v, float sum)
{
    const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    *reinterpret_cast<uint2 *>(a.o + at * D + d) =
        make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
}

// A row's spans joined in order, 4 elements at d; part: the row's span results (D + 4 floats each: maximum, sum, values from 4 on).
template <int D>
__device__ __forceinline__ void join_spans(const float *part, int n, int d, float4 &v, float &sum)
{
    float top = -INFINITY;
#pragma unroll 4
    for (int c = 0; c < n; ++c) top = fmaxf(top, __ldcg(part + static_cast<int64_t>(c) * (D + 4)));
    sum = 0.0f;
    v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (top == -INFINITY) return;
#pragma unroll 4
    for (int c = 0; c < n; ++c) {
        const float *pc = part + static_cast<int64_t>(c) * (D + 4);
        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(pc));
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(pc + 4 + d));
        const float w = ex2(ml.x - top);
        sum = __fmaf_rn(w, ml.y, sum);
        v.x = __fmaf_rn(w, x.x, v.x);
        v.y = __fmaf_rn(w, x.y, v.y);
        v.z = __fmaf_rn(w, x.z, v.z);
        v.w = __fmaf_rn(w, x.w, v.w);
    }
}

struct SpanArgs {
    AttnKv4Args a;
    uint64_t magic;
    int row_blocks, spans;
    int count;                                   // whether the last CTA of a row block joins its spans
    int pdl;
};

template <int D, int NB, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 512 : 128, WIDE ? 1 : (D * NB > 128 ? 3 : 4)) attn_kv4_span_kernel(SpanArgs p)
{
    constexpr int WARPS = WIDE ? kChunks * kChunkBlocks : kChunks;
    constexpr int BLOCKS = WIDE ? 1 : kChunkBlocks;       // a warp's blocks
    using P = Plan<D, NB, WARPS>;
    constexpr int G = P::G, W = P::kPiece / 4;
    extern __shared__ __align__(16) unsigned char smem[];
    const AttnKv4Args &a = p.a;
    const Kv4View &c = a.c;
    const int span = blockIdx.x / p.row_blocks, rb = blockIdx.x - span * p.row_blocks, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (p.pdl) pdl_wait();
    pdl_launch_dependents();

    // pages of the warp's positions, 16 a lane; the lengths are on their way meanwhile
    const int p0 = span * kSpan, pw = p0 + warp * (BLOCKS * kBlock);
    int pages = lane < BLOCKS * 4 ? kv4_page(c, b, pw + 16 * lane) : -1;
    const int cu0 = __ldg(c.cu_q + b), cu1 = __ldg(c.cu_q + b + 1), len = __ldg(c.kv_len + b);
    Rows rows;
    rows.t0 = max(0, cu0);
    rows.GH = a.Hq / c.Hkv;
    rows.hk = blockIdx.y;
    rows.magic = p.magic;
    rows.r0 = rb * P::R;
    rows.first = len - (cu1 - cu0);                       // position of the first new token
    const int tokens = min(c.T, cu1) - rows.t0, n_rows = min(tokens, c.max_q) * rows.GH;
    if (blockIdx.x == 0)                                  // tokens past max_q are left out: zeros
        for (int64_t i = static_cast<int64_t>(c.max_q) * rows.GH * (D / 4) + threadIdx.x;
             i < static_cast<int64_t>(tokens) * rows.GH * (D / 4); i += 32 * WARPS) {
            const int64_t r = i / (D / 4), tok = r / rows.GH;
            write_out<D>(a, (rows.t0 + tok) * a.Hq + rows.hk * rows.GH + r - tok * rows.GH, static_cast<int>(i % (D / 4)) * 4,
                         make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f);
        }
    if (rows.r0 >= n_rows) return;
    rows.r_last = min(n_rows, rows.r0 + P::R) - 1;
    const int n_most = row_positions(a, rows, rows.r_last), n_least = row_positions(a, rows, rows.r0);
    if (p0 >= n_most && (span > 0 || n_most > 0)) return;
    if (pw + 16 * lane >= n_most) pages = -1;

    unsigned char *mine = smem + warp * P::kWarp;
    const uint32_t my = smem_u32(mine);
    const int PS = 1 << c.page_shift;
    const int64_t head = static_cast<int64_t>(rows.hk) * Kv4Layout::block(PS, D);
    // copies of a block's keys and parameters, or of its values; pages that are not there are left out
    auto copy_keys = [&](int blk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int page = __shfl_sync(0xffffffffu, pages, blk * 4 + i), slot = (pw + blk * kBlock + 16 * i) & (PS - 1);
            if (page >= 0) {
                const unsigned char *src = c.pool + page * c.page_stride + head;
                cp_async<P::kPiece>(my + (64 * i + lane) * P::kPiece, src + slot * Kv4Layout::k_row(D) + lane * P::kPiece);
                cp_async<P::kPiece>(my + (64 * i + 32 + lane) * P::kPiece,
                                    src + slot * Kv4Layout::k_row(D) + (32 + lane) * P::kPiece);
                if (lane < 16)
                    cp_async<8 * G>(my + 2 * P::kCodes + (blk & 1) * P::kPar + (16 * i + lane) * 8 * G,
                                    src + Kv4Layout::p_off(PS, D) + (slot + lane) * Kv4Layout::p_row(D));
            }
        }
        cp_commit();
    };
    auto copy_values = [&](int blk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int page = __shfl_sync(0xffffffffu, pages, blk * 4 + i), slot = (pw + blk * kBlock + 16 * i) & (PS - 1);
            if (page >= 0) {
                const unsigned char *src = c.pool + page * c.page_stride + head + Kv4Layout::v_off(PS, D) +
                                           (slot / 2 + t) * Kv4Layout::v_pair(D) + g * P::kPiece;
                cp_async<P::kPiece>(my + P::kCodes + (64 * i + lane) * P::kPiece, src);
                cp_async<P::kPiece>(my + P::kCodes + (64 * i + 32 + lane) * P::kPiece, src + 4 * Kv4Layout::v_pair(D));
            }
        }
        cp_commit();
    };
    copy_keys(0);
    copy_values(0);
    stage_queries<D, NB, WARPS>(a, smem, rows);
    __syncthreads();

    // this lane's columns: rows 8 nb + 2 t + i of the row block
    f2 f[NB], l[NB], z[NB][G], o[G][4][NB][2];
    float m[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        f[nb] = *reinterpret_cast<const f2 *>(smem + P::kF + (8 * nb + 2 * t) * 4);
        m[nb][0] = m[nb][1] = -INFINITY;
        l[nb] = 0;
#pragma unroll
        for (int k = 0; k < G; ++k) {
            z[nb][k] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k][e][nb][0] = o[k][e][nb][1] = 0;
        }
    }

#pragma unroll 1
    for (int blk = 0; blk < BLOCKS; ++blk) {
        const int pb = pw + blk * kBlock;
        if (pb >= n_most) break;
        const bool more = blk + 1 < BLOCKS && pb + kBlock < n_most;
        // bit i: positions 16 i .. of the block are on a page; full: and every row sees the whole block
        const unsigned there = (__ballot_sync(0xffffffffu, pages >= 0) >> (4 * blk)) & 15u;
        const bool full = there == 15u && pb + kBlock <= n_least;
        cp_wait<1>();
        __syncwarp();
        const unsigned char *par = mine + 2 * P::kCodes + (blk & 1) * P::kPar;

        // ---- scores: the tiles' chains of products side by side
        float s[kTiles][NB][4];
        {
            uint32_t kw[2 * kTiles][W];
#pragma unroll
            for (int i = 0; i < 2 * kTiles; ++i) lds_words<P::kPiece>(mine + (i * 32 + lane) * P::kPiece, kw[i]);
#pragma unroll
            for (int k = 0; k < G; ++k) {
                float acc[kTiles][NB][4];
#pragma unroll
                for (int tile = 0; tile < kTiles; ++tile)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[tile][nb][i] = 0.0f;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t q[NB][2];
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            lds_words<8>(smem + P::kQ + (8 * nb + g) * P::kQRow + (64 * k + 16 * t + 8 * j + 4 * h) * 2, q[nb]);
#pragma unroll
                        for (int tile = 0; tile < kTiles; ++tile) {
                            uint32_t x0[4], x1[4];
                            code_operands(kw[2 * tile][2 * k + j], x0);
                            code_operands(kw[2 * tile + 1][2 * k + j], x1);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                mma(acc[tile][nb], x0[2 * h], x1[2 * h], x0[2 * h + 1], x1[2 * h + 1], q[nb][0], q[nb][1]);
                        }
                    }
                f2 tq[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    tq[nb] = pk(*reinterpret_cast<const float *>(smem + P::kT + ((8 * nb + 2 * t) * G + k) * 4),
                                *reinterpret_cast<const float *>(smem + P::kT + ((8 * nb + 2 * t + 1) * G + k) * 4));
#pragma unroll
                for (int tile = 0; tile < kTiles; ++tile)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t w =
                            *reinterpret_cast<const uint32_t *>(par + (16 * tile + 8 * half + g) * 8 * G + 4 * k);
                        const f2 sk = pk(bf16_lo(w), bf16_lo(w)), zk = pk(bf16_hi(w), bf16_hi(w));
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            float *x = &s[tile][nb][2 * half];
                            const f2 u = fma2(zk, tq[nb], k ? pk(x[0], x[1]) : 0ull);
                            const float2 r = upk(fma2(sk, pk(acc[tile][nb][2 * half], acc[tile][nb][2 * half + 1]), u));
                            x[0] = r.x;
                            x[1] = r.y;
                        }
                    }
            }
        }
        // positions that a row does not see, or that are on no page
        if (!full) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int n = *reinterpret_cast<const int *>(smem + P::kN + (8 * nb + 2 * t + i) * 4) - pb - g;
#pragma unroll
                    for (int tile = 0; tile < kTiles; ++tile)
#pragma unroll
                        for (int half = 0; half < 2; ++half)
                            if (!((there >> tile) & 1u) || 16 * tile + 8 * half >= n) s[tile][nb][2 * half + i] = -INFINITY;
                }
        }
        // the keys are read: the next block's may come (parameters are double-buffered)
        __syncwarp();
        if (more) copy_keys(blk + 1);
        else cp_commit();

        // ---- the values' scales and z / s, two positions a lane; nothing for positions that no row sees
        unsigned char *prep = mine + 2 * P::kCodes + 2 * P::kPar;
        int e_all = kMinExp;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int x = lane + 32 * i;
            uint32_t w[2 * G];
            lds_words<8 * G>(par + x * 8 * G, w);
            const bool seen = ((there >> (x >> 4)) & 1u) && pb + x < n_most;
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
                *reinterpret_cast<float4 *>(prep + x * 16) = make_float4(out[0], out[1], out[2], out[3]);
            else
                *reinterpret_cast<float2 *>(prep + x * 8) = make_float2(out[0], out[1]);
        }
        __syncwarp();

        // ---- the block's maxima of scores and of value scales' exponents, per row
        float mb[NB][2];
        int es[NB][2];
        if (full) {
            e_all = __reduce_max_sync(0xffffffffu, e_all);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) es[nb][0] = es[nb][1] = e_all;
        } else {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) es[nb][0] = es[nb][1] = kMinExp;
#pragma unroll
            for (int tile = 0; tile < kTiles; ++tile)
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
                            if (s[tile][nb][2 * half + i] > -INFINITY) es[nb][i] = max(es[nb][i], e);
                }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) es[nb][i] = max(es[nb][i], __shfl_xor_sync(0xffffffffu, es[nb][i], x));
        }
        f2 ref[NB];                                       // weights are 2^(f s - ref) = 2^(15 - es) e^(score - max)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int tile = 0; tile < kTiles; ++tile) top = fmaxf(top, fmaxf(s[tile][nb][i], s[tile][nb][2 + i]));
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float2 ff = upk(f[nb]);
                mb[nb][i] = top * (i ? ff.y : ff.x);       // in units of log2
            }
            const float r0 = mb[nb][0] == -INFINITY ? 0.0f : mb[nb][0], r1 = mb[nb][1] == -INFINITY ? 0.0f : mb[nb][1];
            ref[nb] = pk(static_cast<float>(15 - es[nb][0]) - r0, static_cast<float>(15 - es[nb][1]) - r1);
        }

        // ---- weights, rounded to f16 after the value's scale, as operands
        uint32_t w16[kTiles][G][NB][2];
        f2 lb[NB], zb[NB][G];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            lb[nb] = 0;
#pragma unroll
            for (int k = 0; k < G; ++k) zb[nb][k] = 0;
        }
#pragma unroll
        for (int tile = 0; tile < kTiles; ++tile)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t pr[2 * G];
                lds_words<8 * G>(prep + (16 * tile + 8 * half + g) * 8 * G, pr);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const float2 x = upk(fma2(pk(s[tile][nb][2 * half], s[tile][nb][2 * half + 1]), f[nb], ref[nb]));
                    const f2 w = pk(ex2(x.x), ex2(x.y));
                    lb[nb] = add2(lb[nb], w);
#pragma unroll
                    for (int k = 0; k < G; ++k) {
                        const float sv = __uint_as_float(pr[2 * k]), zr = __uint_as_float(pr[2 * k + 1]);
                        const float2 ws = upk(mul2(w, pk(sv, sv)));
                        const __half2 h = __floats2half2_rn(ws.x, ws.y);
                        const float2 back = __half22float2(h);
                        zb[nb][k] = fma2(pk(back.x, back.y), pk(zr, zr), zb[nb][k]);
                        w16[tile][k][nb][half] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h));
                    }
                }
            }

        // ---- weights of the fold: the chunk's side, and the block's with its power of two undone
        f2 wa[NB], wo[NB], wq[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float x[2], y[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[nb][i] = fold_weights(m[nb][i], mb[nb][i], x[i], y[i]);
                y[i] *= pow2_int(min(es[nb][i], kMaxExp) - 20);   // 2^(es - 15), its 2^5 left out
            }
            wa[nb] = pk(x[0], x[1]);
            const f2 wb = pk(y[0], y[1]);
            l[nb] = fma2(mul2(lb[nb], pk(32.0f, 32.0f)), wb, mul2(l[nb], wa[nb]));
#pragma unroll
            for (int k = 0; k < G; ++k) z[nb][k] = fma2(mul2(zb[nb][k], pk(32.0f, 32.0f)), wb, mul2(z[nb][k], wa[nb]));
            wo[nb] = mul2(wb, pk(0x1p29f, 0x1p29f));        // and products carry 2^-24, odd elements 2^-20
            wq[nb] = mul2(wb, pk(0x1p25f, 0x1p25f));
        }

        // ---- weighted values
        cp_wait<1>();
        {
            uint32_t vw[2 * kTiles][W];
#pragma unroll
            for (int i = 0; i < 2 * kTiles; ++i) lds_words<P::kPiece>(mine + P::kCodes + (i * 32 + lane) * P::kPiece, vw[i]);
#pragma unroll
            for (int k = 0; k < G; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float acc[2][NB][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[h][nb][i] = 0.0f;
#pragma unroll
                    for (int tile = 0; tile < kTiles; ++tile) {
                        uint32_t x0[4], x1[4];
                        code_operands(vw[2 * tile][2 * k + j], x0);
                        code_operands(vw[2 * tile + 1][2 * k + j], x1);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                mma(acc[h][nb], x0[2 * h], x0[2 * h + 1], x1[2 * h], x1[2 * h + 1], w16[tile][k][nb][0],
                                    w16[tile][k][nb][1]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            f2 *x = o[k][2 * j + h][nb];   // elements 2 h and 2 h + 1 of the word, two rows each
                            x[0] = fma2(pk(acc[h][nb][0], acc[h][nb][1]), wo[nb], mul2(x[0], wa[nb]));
                            x[1] = fma2(pk(acc[h][nb][2], acc[h][nb][3]), wq[nb], mul2(x[1], wa[nb]));
                        }
                }
        }
        __syncwarp();
        if (more) copy_values(blk + 1);
        else cp_commit();
    }
    cp_wait<0>();
    __syncwarp();                                          // the warp's codes are read; its results take their place

    float *ow = reinterpret_cast<float *>(mine);
    float *sm = reinterpret_cast<float *>(smem + P::kM), *sl = reinterpret_cast<float *>(smem + P::kL);
    if (g == 0)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            *reinterpret_cast<float2 *>(sm + warp * P::R + 8 * nb + 2 * t) = make_float2(m[nb][0], m[nb][1]);
    // sums over the lanes that share a row (after the fold, lane by lane)
    auto over_lanes = [&](f2 x) {
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) x = add2(x, __shfl_xor_sync(0xffffffffu, x, i));
        return x;
    };
    if constexpr (!WIDE) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const f2 sum = over_lanes(l[nb]);
            if (g == 0) *reinterpret_cast<f2 *>(sl + warp * P::R + 8 * nb + 2 * t) = sum;
#pragma unroll
            for (int k = 0; k < G; ++k) z[nb][k] = over_lanes(z[nb][k]);
        }
    } else {
        f2 *lz = reinterpret_cast<f2 *>(mine + P::kO) + lane * (NB * (1 + G));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            lz[nb * (1 + G)] = l[nb];
#pragma unroll
            for (int k = 0; k < G; ++k) {
                lz[nb * (1 + G) + 1 + k] = z[nb][k];
                z[nb][k] = 0;
            }
        }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < G; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 e0 = upk(o[k][2 * j][nb][0]), e1 = upk(o[k][2 * j][nb][1]), e2 = upk(o[k][2 * j + 1][nb][0]),
                             e3 = upk(o[k][2 * j + 1][nb][1]), zz = upk(z[nb][k]);
                float *dst = ow + (8 * nb + 2 * t) * D + 64 * k + 8 * g + 4 * j;
                if constexpr (WIDE) {
                    *reinterpret_cast<float4 *>(dst) = make_float4(e0.x, e1.x, e2.x, e3.x);
                    *reinterpret_cast<float4 *>(dst + D) = make_float4(e0.y, e1.y, e2.y, e3.y);
                } else {
                    *reinterpret_cast<float4 *>(dst) = make_float4(e0.x + zz.x, e1.x + zz.x, e2.x + zz.x, e3.x + zz.x);
                    *reinterpret_cast<float4 *>(dst + D) = make_float4(e0.y + zz.y, e1.y + zz.y, e2.y + zz.y, e3.y + zz.y);
                }
            }
    __syncthreads();
    if constexpr (WIDE) {
        // chunk `warp`: the lanes' sums folded over its blocks as a single warp would, then over the lanes
        if (warp < kChunks) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                f2 ll = 0, zz[G];
                float mm[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < G; ++k) zz[k] = 0;
#pragma unroll
                for (int j = 0; j < kChunkBlocks; ++j) {
                    const int wj = warp * kChunkBlocks + j;
                    const f2 *lz = reinterpret_cast<const f2 *>(smem + wj * P::kWarp + P::kO) + (lane * NB + nb) * (1 + G);
                    float x[2], y[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        mm[i] = fold_weights(mm[i], sm[wj * P::R + 8 * nb + 2 * t + i], x[i], y[i]);
                    const f2 fa = pk(x[0], x[1]), fb = pk(y[0], y[1]);
                    ll = fma2(lz[0], fb, mul2(ll, fa));
#pragma unroll
                    for (int k = 0; k < G; ++k) zz[k] = fma2(lz[1 + k], fb, mul2(zz[k], fa));
                }
                const f2 sum = over_lanes(ll);
                if (g == 0) *reinterpret_cast<f2 *>(sl + warp * P::R + 8 * nb + 2 * t) = sum;
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    const float2 v = upk(over_lanes(zz[k]));
                    float *dst = reinterpret_cast<float *>(smem + P::kZ) + (warp * P::R + 8 * nb + 2 * t) * G + k;
                    if (g == 0) {
                        dst[0] = v.x;
                        dst[G] = v.y;
                    }
                }
            }
        }
        __syncthreads();
    }

    // ---- the span's chunks joined in order
    for (int i = threadIdx.x; i < P::R * D / 4; i += 32 * WARPS) {
        const int rl = i / (D / 4), d = i % (D / 4) * 4, r = rows.r0 + rl;
        if (r > rows.r_last) break;
        const int tok = rows.token(r), n = min(c.max_kv, rows.first + tok + 1);
        if (p0 >= n && (span > 0 || n > 0)) continue;
        float mc[kChunks], top = -INFINITY, sum = 0.0f;
        float4 vc[kChunks];
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
            if constexpr (WIDE) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float mm = -INFINITY;
#pragma unroll
                for (int j = 0; j < kChunkBlocks; ++j) {
                    const int wj = ch * kChunkBlocks + j;
                    float x, y;
                    mm = fold_weights(mm, sm[wj * P::R + rl], x, y);
                    const float4 u = *reinterpret_cast<const float4 *>(smem + wj * P::kWarp + (rl * D + d) * 4);
                    v.x = __fmaf_rn(u.x, y, v.x * x);
                    v.y = __fmaf_rn(u.y, y, v.y * x);
                    v.z = __fmaf_rn(u.z, y, v.z * x);
                    v.w = __fmaf_rn(u.w, y, v.w * x);
                }
                const float zz = reinterpret_cast<const float *>(smem + P::kZ)[(ch * P::R + rl) * G + d / kKv4Group];
                mc[ch] = mm;
                vc[ch] = make_float4(v.x + zz, v.y + zz, v.z + zz, v.w + zz);
            } else {
                mc[ch] = sm[ch * P::R + rl];
                vc[ch] = *reinterpret_cast<const float4 *>(smem + ch * P::kWarp + (rl * D + d) * 4);
            }
            top = fmaxf(top, mc[ch]);
        }
        const float base = top == -INFINITY ? 0.0f : top;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
            const float e = ex2(mc[ch] - base);
            sum = __fmaf_rn(e, sl[ch * P::R + rl], sum);
            v.x = __fmaf_rn(e, vc[ch].x, v.x);
            v.y = __fmaf_rn(e, vc[ch].y, v.y);
            v.z = __fmaf_rn(e, vc[ch].z, v.z);
            v.w = __fmaf_rn(e, vc[ch].w, v.w);
        }
        const int64_t at = static_cast<int64_t>(rows.t0 + tok) * a.Hq + rows.hk * rows.GH + r - tok * rows.GH;
        if (n <= kSpan) {
            write_out<D>(a, at, d, v, sum);
        } else {
            float *part = reinterpret_cast<float *>(static_cast<char *>(a.ws) + kCounterBytes) + (at * p.spans + span) * (D + 4);
            *reinterpret_cast<float4 *>(part + 4 + d) = v;
            if (d == 0) *reinterpret_cast<float2 *>(part) = make_float2(top, sum);
        }
    }

    // ---- the row block's last CTA joins the spans
    if (!p.count || n_most <= kSpan) return;
    int *flag = reinterpret_cast<int *>(smem + P::kFlag);
    __syncthreads();
    if (threadIdx.x == 0) {
        int *counter = static_cast<int *>(a.ws) + (static_cast<int64_t>(b) * c.Hkv + rows.hk) * p.row_blocks + rb;
        const bool last = atom_add_acq_rel_gpu(counter, 1) == (n_most + kSpan - 1) / kSpan - 1;
        if (last) *counter = 0;
        *flag = last;
    }
    __syncthreads();
    if (!*flag) return;
    for (int i = threadIdx.x; i < P::R * D / 4; i += 32 * WARPS) {
        const int rl = i / (D / 4), d = i % (D / 4) * 4, r = rows.r0 + rl;
        if (r > rows.r_last) break;
        const int tok = rows.token(r), n = min(c.max_kv, rows.first + tok + 1);
        if (n <= kSpan) continue;
        const int64_t at = static_cast<int64_t>(rows.t0 + tok) * a.Hq + rows.hk * rows.GH + r - tok * rows.GH;
        float4 v;
        float sum;
        join_spans<D>(reinterpret_cast<const float *>(static_cast<char *>(a.ws) + kCounterBytes) + at * p.spans * (D + 4),
                      (n + kSpan - 1) / kSpan, d, v, sum);
        write_out<D>(a, at, d, v, sum);
    }
}

// D / 4 threads per (token, q head): the spans' results in order, where the
// span kernel does not join them itself.
template <int D>
__global__ void __launch_bounds__(128) attn_kv4_join_kernel(AttnKv4Args a, int spans)
{
    constexpr int L = D / 4;
    const int64_t id = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) / L;
    const int d = threadIdx.x % L * 4;
    const int t = static_cast<int>(min(id / a.Hq, static_cast<int64_t>(a.c.T - 1)));
    pdl_wait();
    const int b = kv4_sequence(a.c, t);
    if (b < 0 || id >= static_cast<int64_t>(a.c.T) * a.Hq) return;
    const int begin = __ldg(a.c.cu_q + b), end = __ldg(a.c.cu_q + b + 1);
    const int n = min(a.c.max_kv, __ldg(a.c.kv_len + b) - (end - t) + 1);
    if (t - begin >= a.c.max_q || n <= kSpan) return;
    float4 v;
    float sum;
    join_spans<D>(reinterpret_cast<const float *>(static_cast<char *>(a.ws) + kCounterBytes) + id * spans * (D + 4),
                  (n + kSpan - 1) / kSpan, d, v, sum);
    write_out<D>(a, id, d, v, sum);
}

int spans_of(int max_kv) { return (max_kv + kSpan - 1) / kSpan; }

template <int D, int NB, bool WIDE>
cudaError_t launch_span(const SpanArgs &p, cudaStream_t stream)
{
    constexpr int WARPS = WIDE ? kChunks * kChunkBlocks : kChunks, bytes = Plan<D, NB, WARPS>::kBytes;
    const cudaError_t e =
        cudaFuncSetAttribute(attn_kv4_span_kernel<D, NB, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.row_blocks * p.spans), static_cast<unsigned>(p.a.c.Hkv),
                       static_cast<unsigned>(p.a.c.B));
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attn_kv4_span_kernel<D, NB, WIDE>, p);
}

template <int D, int NB>
cudaError_t launch_span(const SpanArgs &p, bool wide, cudaStream_t stream)
{
    return wide ? launch_span<D, NB, true>(p, stream) : launch_span<D, NB, false>(p, stream);
}

}  // namespace

size_t attention_kv4_workspace(int Hq, int D, int T, int max_kv)
{
    const int spans = spans_of(max_kv);
    return kCounterBytes + (spans == 1 ? 0 : static_cast<size_t>(T) * Hq * spans * (D + 4) * sizeof(float));
}

cudaError_t launch_attention_kv4(const AttnKv4Args &a, int D, bool pdl, cudaStream_t stream)
{
    const int GH = a.Hq / a.c.Hkv, rows = a.c.max_q * GH, NB = rows <= 8 ? 1 : 2;
    SpanArgs p;
    p.a = a;
    p.magic = (1ull << 32) / GH + 1;
    p.row_blocks = (rows + 8 * NB - 1) / (8 * NB);
    p.spans = spans_of(a.c.max_kv);
    p.pdl = pdl ? 1 : 0;
    if (static_cast<int64_t>(p.row_blocks) * p.spans > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const int64_t groups = static_cast<int64_t>(a.c.B) * a.c.Hkv * p.row_blocks;
    p.count = groups <= kCounters && p.spans <= kJoinSpans;
    // 16 warps a CTA where every CTA has a SM to itself
    const bool wide = groups * p.spans <= a.sms;
    cudaError_t e = D == 64 ? (NB == 1 ? launch_span<64, 1>(p, wide, stream) : launch_span<64, 2>(p, wide, stream))
                            : (NB == 1 ? launch_span<128, 1>(p, wide, stream) : launch_span<128, 2>(p, wide, stream));
    if (e != cudaSuccess || p.count || p.spans == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(a.c.T) * a.Hq * (D / 4) + 127) / 128));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return D == 64 ? cudaLaunchKernelEx(&cfg, attn_kv4_join_kernel<64>, a, p.spans)
                   : cudaLaunchKernelEx(&cfg, attn_kv4_join_kernel<128>, a, p.spans);
}

}  // namespace bi
