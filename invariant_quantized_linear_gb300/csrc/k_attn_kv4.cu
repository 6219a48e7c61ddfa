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
// and in the result (values).  A value's even nibble stays in its byte, with the
// odd one: their sums' difference, in fp32, is the even nibbles' (an error of 2^-18
// of the group's range, below the weights' 2^-11), and one operation less a word.
//
// Operands are transposed, S^T = K q^T and O^T = V^T P^T, so that positions
// (16 of an mma.m16n8k16) and head elements fill the rows, and the few query
// rows the columns, 8 at a time: a decode step of a group of 4 heads wastes
// half a tile instead of three quarters.  The cache's layout puts what a lane
// needs of a tile's 8 positions into D / 8 bytes of its own.  A warp has its
// blocks copied to shared memory as they lie (bulk copies on two barriers: keys
// with parameters, values; the next block's follow as soon as this one's are
// read) and each lane loads its own words, with no exchange.  Values' words of
// four lanes share banks (head size 128); copies that would spread them, a
// quarter of a block each, cost what they save (126.7 for 127.3 us, b 96, 8191
// positions; head size 64, b 6, 40000: 50.8 for 49.0 us).
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
// Both rank-one terms are products for the tensor cores too, one a tile and
// group: z (bf16 as it stands in the cache) with sum(q) in three bf16 parts,
// and the weights with z / s in two f16 parts, as two more rows of V^T.
//
// Work: positions are cut into blocks of 64 and spans of 32 blocks, counted from
// position 0; every fourth block of a span makes a chunk.  A block's result
// (maximum, sum, weighted values) comes from one warp; a chunk folds its blocks
// in order, a span joins its four chunks' results under their common maximum,
// and a row joins its spans the same way.  A row's result is this tree whatever
// else is in the call, since neither maxima nor scales look at a position that
// the row does not see; which warp computes what may therefore go by the size
// of the call:
//   a span a CTA, a chunk a warp, the fold in registers: least work a position,
//     2 to 5 CTAs a SM overlap one another's latencies;
//   a span a cluster of 8 CTAs, a block a warp, the fold over the cluster's
//     shared memory: for calls that leave SMs idle, where a chunk's eight
//     blocks one after the other would be most of the time.
// Both round in the same order (in a cluster a block's exponent travels with its
// result), and so do 8 and 16 rows a CTA.  A position that a row does not see has
// weight zero and finite operands: value groups that are not finite are set aside
// before the products (set_aside; one reduction a block, 0.5 to 2 % of a call).
// The CTA that finishes a row block's last span joins the spans (a counter in
// the workspace); a second launch does where a row has many spans or the
// counters do not suffice.
//
// Bound: HBM by its bytes (0.5625 B an element) up to 16 query rows a kv head;
// within a span it reads 6.2 TB/s, instructions, shared memory and HBM all near
// their rates; a CTA's start and end (3.1 us) and the last wave are the rest.  With
// more rows instructions: every 16 rows unpack the codes for themselves, so that a
// prompt of 2731 tokens runs at 159 TFLOP/s, a twelfth of the tensor cores' rate.
// Measured (32 q and 8 kv heads of 128; one call repeated in a graph, so that caches
// below 100 MB come from L2; emptying L2 in between adds 1 % at most): b 304, 2048
// positions each 133 us, 5.4 TB/s of codes and parameters; b 96, up to 8191: 127 us,
// 4.5; b 1, 131072: 43.5 us, 3.5; b 64, 8 tokens, 4096: 142 us; b 1, 517: 6.7 us; 28 and
// 4 heads of 64, b 6, 5 tokens, up to 40000: 48.6 us; prompts of 1024 tokens behind 1024
// positions, of 2731, and three of those: 152, 385 and 1373 us.
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

#include <cuda_fp16.h>

namespace bi {

namespace {

constexpr int kBlock = 64;                          // positions of a block
constexpr int kChunkBlocks = 8;
constexpr int kChunks = 4;                          // chunks of a span
constexpr int kSpan = kBlock * kChunkBlocks * kChunks;
constexpr int kTiles = kBlock / 16;
constexpr int kThreads = 32 * kChunks;
constexpr int kCluster = kChunkBlocks;              // CTAs that share a span
constexpr int kMinExp = -100;                       // least exponent that value scales are normalised to
constexpr int kMaxExp = 118;                        // largest that is undone again within fp32
constexpr float kMinScale = 0x1p-110f;              // groups of smaller scale count as zeros
constexpr uint32_t kInfBits = 0x7F800000u;          // scales from here on are infinite or NaN
constexpr float kMaxRatio = 65504.0f;               // largest z / s that f16 holds (of a valid group: 4096)
constexpr int kCounters = 16384;                    // row blocks whose spans are counted in the workspace
constexpr int kJoinSpans = 16;                      // spans that a CTA joins itself at most, and a run of the second launch
constexpr size_t kStatusBytes = 256;                // the status word, then the counters, then the spans' results
constexpr size_t kCounterBytes = kStatusBytes + kCounters * sizeof(int);

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// `bytes` (a multiple of 16) from global to shared memory by the copy engine, counted on `bar`.
__device__ __forceinline__ void bulk_copy(uint32_t smem, unsigned long long gmem, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem),
                 "l"(gmem), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
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

// The same with the even nibbles not taken out of their bytes: c0 + 16 c1, 16 c1 and so on.
__device__ __forceinline__ void byte_operands(uint32_t w, uint32_t (&o)[4])
{
    o[0] = w & 0x00FF00FFu;
    o[1] = w & 0x00F000F0u;
    o[2] = __byte_perm(w, 0u, 0x4341);
    o[3] = o[2] & 0x00F000F0u;
}

__device__ __forceinline__ float pow2_int(int e) { return __int_as_float((e + 127) << 23); }   // -126 .. 127

// Shared memory of a CTA for head size D and NB blocks of 8 query rows.
template <int D, int NB, bool SPLIT>
struct Plan {
    static constexpr int kBlocks = SPLIT ? 1 : kChunkBlocks;   // blocks of a warp
    static constexpr int G = D / kKv4Group;
    static constexpr int R = 8 * NB;                       // query rows
    static constexpr int kPiece = D / 8;                   // bytes of a lane's share of 8 positions (16 or 8)
    static constexpr int kCodes = 8 * 32 * kPiece;         // 64 positions of keys (or values)
    static constexpr int kPar = kBlock * 8 * G;            // their parameters
    static constexpr int kScale = kBlock * 4 * G;          // value scales of the block, fp32 [position][group]
    static constexpr int kRatio = kBlock * 4 * G;          // their z / s, two f16 parts [tile][group][part][16 positions]
    static constexpr int kZero = 16 * 2;                   // zeros for the rows of V^T that are not there
    static constexpr int kWarp = 2 * kCodes + kPar + kScale + kRatio + kZero;
    static constexpr int kQRow = 2 * D + 8;                // bytes of a query row in f16; the 8 spread the banks
    static constexpr int kO = R * D * 4;                   // a result's values; they take the place of the warp's codes
    static constexpr int kLZ = (32 + 8 * G) * NB * 8;      // and, in a cluster, its sums lane by lane
    static constexpr int kResult = kO + (SPLIT ? kLZ : 0);
    static constexpr int kQ = kChunks * kWarp;
    static constexpr int kT = kQ + R * kQRow;              // sums of q per row: 8 bf16, three parts a group, then zeros
    static constexpr int kF = kT + R * 16;                 // factor per row
    static constexpr int kN = kF + R * 4;                  // positions that a row sees
    static constexpr int kM = kN + R * 4;                  // maxima [warp][row]
    static constexpr int kL = kM + kChunks * R * 4;        // sums [chunk][row]
    // in a cluster: exponents of value scales [warp][row], the chunks' maxima [chunk][row] and values of the CTA's rows
    // [chunk][item]
    static constexpr int kE = kL + kChunks * R * 4;
    static constexpr int kC = kE + (SPLIT ? kChunks * R * 4 : 0);
    static constexpr int kV = kC + (SPLIT ? kChunks * R * 4 : 0);
    static constexpr int kFlag = kV + (SPLIT ? kO / 8 * kChunks : 0);
    static constexpr int kBar = kFlag + 16;                // two barriers a warp: keys and parameters, values
    static constexpr int kBytes = kBar + kChunks * 16;
    static_assert(R * D / 4 / kCluster % (D / 4) == 0, "a CTA of a cluster joins whole rows");
    static_assert(kResult <= kWarp && kV % 16 == 0, "a warp's results fit in the place of its codes");
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

// D = A(16x16) B(16x8) + C in f16 with fp32 sums; not volatile, so that independent chains may interleave.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first of a chain: C = 0.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// D = A(16x8) B(8x8) in bf16.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%7, %7, %7, %7};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(b0), "f"(0.0f));
}

// The rows of a CTA: query rows r0 .. r_last of one kv head, row r = (token r / GH of the sequence, head r % GH).
struct Rows {
    int t0, first, GH, r0, r_last, hk;
    uint64_t magic;                              // 2^32 / GH + 1: r / GH for r * GH < 2^32
    __device__ __forceinline__ int token(int r) const { return static_cast<int>((r * magic) >> 32); }
};

// Positions that row r sees: at most max_kv, or the row would have been left out.
__device__ __forceinline__ int row_positions(const Rows &w, int r) { return w.first + w.token(r) + 1; }

// Query rows to shared memory: f16 elements scaled by a power of two, odd
// element pairs divided by 16; the sums and the factor that turn products with
// codes into scores in units of log2.
template <int D, int NB, bool SPLIT>
__device__ __forceinline__ void stage_queries(const AttnKv4Args &a, unsigned char *smem, const Rows &rows)
{
    using P = Plan<D, NB, SPLIT>;
    // all rows at once: L lanes a row, E elements a lane
    constexpr int L = kThreads / P::R, E = D / L;
    const int rl = threadIdx.x / L, at = threadIdx.x % L * E;
    const int r = rows.r0 + rl, tok = rows.token(min(r, rows.r_last));
    uint32_t w[E / 2] = {};
    if (r <= rows.r_last) {                                // idle rows are zeros
        const uint16_t *src = a.q + (rows.t0 + tok) * a.ldq + (rows.hk * rows.GH + r - tok * rows.GH) * D + at;
        if constexpr (E == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(src);
            w[0] = v.x, w[1] = v.y;
        } else {
#pragma unroll
            for (int e = 0; e < E / 8; ++e) {
                const uint4 v = reinterpret_cast<const uint4 *>(src)[e];
                w[4 * e] = v.x, w[4 * e + 1] = v.y, w[4 * e + 2] = v.z, w[4 * e + 3] = v.w;
            }
        }
    }
    float x[E], top = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        x[e] = e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
        top = fmaxf(top, fabsf(x[e]));
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // up = 2^(14 - floor(log2 top)), kept in fp32's range
    const int ex = max(-100, min(127, static_cast<int>(__float_as_uint(top) >> 23) - 127));
    const float up = pow2_int(14 - ex);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= up;
    // A group's sum in an order that does not depend on E, and so not on the form that a call takes: fours, neighbouring
    // fours, neighbours of those and so on, in the lane as long as it holds several.
    float part[E / 4];
#pragma unroll
    for (int e = 0; e < E / 4; ++e) part[e] = (x[4 * e] + x[4 * e + 1]) + (x[4 * e + 2] + x[4 * e + 3]);
#pragma unroll
    for (int o = 1; o < E / 4; o <<= 1)
#pragma unroll
        for (int e = 0; e < E / 4; e += 2 * o) part[e] += part[e + o];
    float sum = part[0];
#pragma unroll
    for (int e = 0; e < E / 4; ++e) {                      // a lane's elements begin with an even pair
        const __half2 h0 = __floats2half2_rn(x[4 * e], x[4 * e + 1]),
                      h1 = __floats2half2_rn(x[4 * e + 2] * 0.0625f, x[4 * e + 3] * 0.0625f);
        *reinterpret_cast<uint2 *>(smem + P::kQ + rl * P::kQRow + (at + 4 * e) * 2) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&h0), *reinterpret_cast<const uint32_t *>(&h1));
    }
#pragma unroll
    for (int o = 1; o < kKv4Group / E; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (at % kKv4Group == 0) {
        // three parts of 8 bits: all 24 of the sum
        uint16_t *dst = reinterpret_cast<uint16_t *>(smem + P::kT + rl * 16) + 3 * (at / kKv4Group);
        float rest = sum * 0x1p-24f;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const uint32_t part = bf16_rne_bits(rest);
            dst[i] = static_cast<uint16_t>(part);
            rest -= __uint_as_float(part << 16);
        }
        if (at == 0) {
#pragma unroll
            for (int i = 3 * P::G; i < 8; ++i) dst[i] = 0;
            // scores = factor * (products with 2^-24 c and up q)
            *reinterpret_cast<float *>(smem + P::kF + rl * 4) =
                fmaxf(fminf(a.scale * 1.4426950408889634f * 0x1p10f * pow2_int(ex), 0x1p126f), 0x1p-126f);
            *reinterpret_cast<int *>(smem + P::kN + rl * 4) = rows.first + tok + 1;
        }
    }
}

__device__ __forceinline__ unsigned long long ld_cluster_b64(uint32_t addr)
{
    unsigned long long v;
    asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// The two halves of a cluster barrier: everything before the arrival is done for those who have waited.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The fold of a block's result into a chunk's: weights of the two sides, the block's with its power of two undone,
// 2^(es - 15) but for 2^5.  The product may be subnormal, so both forms of the kernel fold with it as it is.
__device__ __forceinline__ float fold_weights(float m, float mb, int es, float &wa, float &wb)
{
    const float top = fmaxf(m, mb), ref = top == -INFINITY ? 0.0f : top;
    wa = ex2(m - ref);
    wb = ex2(mb - ref) * pow2_int(min(es, kMaxExp) - 20);
    return top;
}

constexpr float kFoldSum = 32.0f;                   // what is left of the power of two in sums of weights (exact products),
constexpr float kFoldEven = 0x1p29f;                // in products with codes, which carry 2^-24,
constexpr float kFoldOdd = 0x1p25f;                 // and 2^-20 in odd elements

__device__ __forceinline__ f2 times2(f2 v, float f) { return mul2(v, pk(f, f)); }

// a + the block's b
__device__ __forceinline__ f2 fold2(f2 a, f2 wa, f2 b, f2 wb) { return fma2(b, wb, mul2(a, wa)); }

// out[row] from the joined value v (4 elements at d) and sum.
template <int D>
__device__ __forceinline__ void write_out(const AttnKv4Args &a, int64_t at, int d, const float4 &v, float sum)
{
    const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    *reinterpret_cast<uint2 *>(a.o + at * D + d) =
        make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
}

// Adds one span's result, maximum and sum ml and 4 values x, under the row's maximum.
__device__ __forceinline__ void add_span(const float2 &ml, const float4 &x, float top, float4 &v, float &sum)
{
    const float w = ex2(ml.x - top);
    sum = __fmaf_rn(w, ml.y, sum);
    v.x = __fmaf_rn(w, x.x, v.x);
    v.y = __fmaf_rn(w, x.y, v.y);
    v.z = __fmaf_rn(w, x.z, v.z);
    v.w = __fmaf_rn(w, x.w, v.w);
}

struct SpanArgs {
    AttnKv4Args a;
    uint64_t magic;
    int row_blocks, spans;
    int count;                                   // whether the last CTA of a row block joins its spans
    int pdl;
};

// A block's value groups that are not finite (sv, r: scales and z / s of positions 2 lane and 2 lane + 1).  A weight of
// zero does not keep them from a row, so they are set to nothing for the products, and the minima's term (z, of the
// lane's columns) of the rows that see them, which joins the values of their group alone, becomes NaN.  Returns the bits
// of the largest other scale.  Rows see seen[] positions, the block's begin at pb.
template <int NB, int G>
__device__ __forceinline__ uint32_t set_aside(const int *seen, int pb, float (&sv)[2][G], float (&r)[2][G], f2 (&z)[NB][G])
{
    const int t = threadIdx.x & 3;
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < G; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool bad = __float_as_uint(sv[i][k]) >= kInfBits || !(fabsf(r[i][k]) <= kMaxRatio);
            const unsigned at = __ballot_sync(0xffffffffu, bad);
            if (bad) sv[i][k] = r[i][k] = 0.0f;
            top = max(top, __float_as_uint(sv[i][k]));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                // of the positions 2 l + i the row sees those of the first n lanes
                auto sees = [&](int row) {
                    const int n = max(0, min(32, (seen[row] - pb - i + 1) >> 1));
                    return (at & static_cast<unsigned>((1ull << n) - 1)) != 0;
                };
                float2 v = upk(z[nb][k]);
                if (sees(8 * nb + 2 * t)) v.x = __int_as_float(0x7FC00000);
                if (sees(8 * nb + 2 * t + 1)) v.y = __int_as_float(0x7FC00000);
                z[nb][k] = pk(v.x, v.y);
            }
        }
    return __reduce_max_sync(0xffffffffu, top);
}

// What a CTA finds before it knows how many rows it has.
struct Task {
    int rank, hk, rb, b, span;
    int my_pos, page;                            // the lane's 16 positions and their page
    int cu0, cu1, len;

    __device__ __forceinline__ int first() const { return len - (cu1 - cu0); }       // position of the first new token
    __device__ __forceinline__ int tokens(const Kv4View &c) const { return min(c.T, max(0, cu1)) - max(0, cu0); }
    // tokens that are not left out: those before max_q, at positions before max_kv
    __device__ __forceinline__ int live(const Kv4View &c) const { return min(min(tokens(c), c.max_q), c.max_kv - first()); }
};

// One span (SPLIT: the CTA's eighth of it) for rows block_rows rb .. of a kv head, at most 8 NB.
template <int D, int NB, bool SPLIT>
__device__ __forceinline__ void span_task(const SpanArgs &p, const Task &task, int block_rows, unsigned char *smem)
{
    using P = Plan<D, NB, SPLIT>;
    constexpr int G = P::G, W = P::kPiece / 4, BLOCKS = P::kBlocks;
    const AttnKv4Args &a = p.a;
    const Kv4View &c = a.c;
    const int rank = task.rank, rb = task.rb, b = task.b, span = task.span, my_pos = task.my_pos;
    int page = task.page;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int p0 = span * kSpan, pw = p0 + (rank * kChunks + warp) * kBlock;
    constexpr int kStep = kChunks * kBlock;
    Rows rows;
    rows.t0 = max(0, task.cu0);
    rows.GH = a.Hq / c.Hkv;
    rows.hk = task.hk;
    rows.magic = p.magic;
    rows.r0 = rb * block_rows;
    rows.first = task.first();
    const int tokens = task.tokens(c), live = task.live(c), n_rows = live * rows.GH;
    if (rb == 0 && span == 0 && rank == 0)                // the other tokens have zeros
        for (int64_t i = static_cast<int64_t>(max(0, live)) * rows.GH * (D / 4) + threadIdx.x;
             i < static_cast<int64_t>(tokens) * rows.GH * (D / 4); i += kThreads) {
            const int64_t r = i / (D / 4), tok = r / rows.GH;
            write_out<D>(a, (rows.t0 + tok) * a.Hq + rows.hk * rows.GH + r - tok * rows.GH, static_cast<int>(i % (D / 4)) * 4,
                         make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f);
        }
    if (rows.r0 >= n_rows) return;
    rows.r_last = min(n_rows, rows.r0 + P::R) - 1;
    const int n_most = row_positions(rows, rows.r_last), n_least = row_positions(rows, rows.r0);
    if (p0 >= n_most && (span > 0 || n_most > 0)) return;
    if (my_pos >= n_most) page = -1;
    const unsigned pages = __ballot_sync(0xffffffffu, page >= 0);

    unsigned char *mine = smem + warp * P::kWarp;
    const uint32_t my = smem_u32(mine);
    const int PS = 1 << c.page_shift;
    // this lane's 16 positions: where their codes begin in the page's block of the kv head, and the page's block
    const int slot = my_pos & (PS - 1);
    const unsigned char *block = kv4_block<D>(c, max(page, 0), rows.hk);
    const unsigned long long codes = reinterpret_cast<unsigned long long>(block + slot * Kv4Layout::k_row(D));
    // parameters begin p_off(PS) - slot (k_row - p_row) after the codes
    const int par_off = Kv4Layout::p_off(PS, D) - slot * (Kv4Layout::k_row(D) - Kv4Layout::p_row(D));
    // Copies of a block's keys with parameters, or of its values: 16 positions a lane, or one lane for all where a page
    // holds the whole block.  Pages that are not there are left out (what stands in their place is not used).
    const bool whole = PS >= kBlock;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + P::kBar) + 2 * warp;
    if (lane == 0) {
        mbar_init(bars, 1);
        mbar_init(bars + 1, 1);
        fence_mbarrier_init();
    }
    __syncwarp();
    const int sub = whole ? 0 : lane & 3, count = whole ? kBlock : 16;
    const bool copies = page >= 0 && (!whole || (lane & 3) == 0);
    const unsigned copy_mask = __ballot_sync(0xffffffffu, copies);
    auto copy_keys = [&](int blk) {
        if ((lane >> 2) == blk) {
            if ((lane & 3) == 0)
                mbar_arrive_expect_tx(bars, __popc((copy_mask >> (4 * blk)) & 15u) * count *
                                                (Kv4Layout::k_row(D) + Kv4Layout::p_row(D)));
            if (copies) {
                bulk_copy(my + sub * 16 * Kv4Layout::k_row(D), codes, count * Kv4Layout::k_row(D), bars);
                bulk_copy(my + 2 * P::kCodes + sub * 16 * Kv4Layout::p_row(D), codes + par_off, count * Kv4Layout::p_row(D),
                          bars);
            }
        }
    };
    auto copy_values = [&](int blk) {
        if ((lane >> 2) == blk) {
            if ((lane & 3) == 0)
                mbar_arrive_expect_tx(bars + 1, __popc((copy_mask >> (4 * blk)) & 15u) * count * Kv4Layout::k_row(D));
            if (copies)
                bulk_copy(my + P::kCodes + sub * 16 * Kv4Layout::k_row(D), codes + Kv4Layout::v_off(PS, D),
                          count * Kv4Layout::k_row(D), bars + 1);
        }
    };
    int *status = static_cast<int *>(a.ws);
    // Waits for block blk's keys (0) or values (1).  If they do not come within the limit the call's result is lost: the
    // status says so, the copies in flight on the barriers (next: the next block's keys too) get one more limit to land,
    // and if these do not either the warp issues no others and goes on, after this block, to the barriers that the other
    // warps wait at: nothing then keeps a later copy from landing in shared memory that the CTA uses again or has left.
    bool lost = false;
    auto wait = [&](int which, int blk, bool next) {
        if (!mbar_wait_bounded(bars + which, blk & 1, status)) {
            *status = DEV_TIMEOUT;
            volatile int never = 0;
            lost = !mbar_wait_bounded(bars + which, blk & 1, &never);
            if (next) mbar_wait_bounded(bars, (blk + 1) & 1, &never);
        }
        __syncwarp();
    };
    copy_keys(0);
    copy_values(0);
    stage_queries<D, NB, SPLIT>(a, smem, rows);
    unsigned char *scale = mine + 2 * P::kCodes + P::kPar, *ratio = scale + P::kScale;
    if (lane < 8) *reinterpret_cast<uint32_t *>(ratio + P::kRatio + 4 * lane) = 0;
    if (SPLIT && lane < P::R) *reinterpret_cast<int *>(smem + P::kE + (warp * P::R + lane) * 4) = 0;   // a warp may have no block
    // this lane's part of z / s as rows of V^T: row 0 the first parts, row 1 the second, no others
    const unsigned char *my_ratio = g < 2 ? ratio + g * 32 + t * 8 : ratio + P::kRatio + t * 8;
    const int ratio_step = g < 2 ? 64 : 0;
    // bytes of two parameter words for the rows of K's minima: parts of group 0 in columns 0-2, of group 1 in 3-5
    const uint32_t pick = G == 1 ? 0x3232u : t == 0 ? 0x3232u : t == 1 ? 0x7632u : 0x7676u;
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
        const int pb = pw + blk * kStep;
        if (pb >= n_most || __any_sync(0xffffffffu, lost)) break;
        const bool more = blk + 1 < BLOCKS && pb + kStep < n_most;
        // bit i: positions 16 i .. of the block are on a page; full: and every row sees the whole block
        const unsigned there = (pages >> (4 * blk)) & 15u;
        const bool full = there == 15u && pb + kBlock <= n_least;
        wait(0, blk, false);
        const unsigned char *par = mine + 2 * P::kCodes;

        // ---- the values' scales and z / s of positions 2 lane and 2 lane + 1; nothing for positions that no row sees
        uint32_t top_scale = 0;                            // bits of the block's largest
        {
            uint32_t w[2][G];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t v[2 * G];
                lds_words<8 * G>(par + (2 * lane + i) * 8 * G, v);
#pragma unroll
                for (int k = 0; k < G; ++k) w[i][k] = v[G + k];
            }
            if (!full) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (!((there >> (lane >> 3)) & 1u) || pb + 2 * lane + i >= n_most) {
#pragma unroll
                        for (int k = 0; k < G; ++k) w[i][k] = 0;
                    }
            }
            float sv[2][G], r[2][G];
#pragma unroll
            for (int k = 0; k < G; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float sc = bf16_lo(w[i][k]), zv = bf16_hi(w[i][k]), v = sc != 0.0f ? sc : 0.125f * fabsf(zv);
                    const bool some = !(v < kMinScale);    // a scale that is NaN too
                    sv[i][k] = some ? v : 0.0f;
                    r[i][k] = some ? __fdividef(zv, v) : 0.0f;
                    top_scale = max(top_scale, __float_as_uint(sv[i][k]));
                    if (!full && !(fabsf(r[i][k]) <= kMaxRatio)) top_scale = ~0u;
                }
            top_scale = __reduce_max_sync(0xffffffffu, top_scale);
            if (top_scale >= kInfBits)
                top_scale = set_aside<NB, G>(reinterpret_cast<const int *>(smem + P::kN), pb, sv, r, z);
            // position y of tile y / 16 is element 2 t + (i & 1) + 8 (i / 2) of its rows, kept as 4 t + i
            unsigned char *at = ratio + (lane >> 3) * (G * 64) + (lane & 3) * 8 + (lane & 4);
#pragma unroll
            for (int k = 0; k < G; ++k) {
                const __half2 hi = __floats2half2_rn(r[0][k], r[1][k]);
                const float2 back = __half22float2(hi);
                const __half2 lo = __floats2half2_rn(r[0][k] - back.x, r[1][k] - back.y);
                *reinterpret_cast<__half2 *>(at + k * 64) = hi;
                *reinterpret_cast<__half2 *>(at + k * 64 + 32) = lo;
            }
            if constexpr (G == 2)
                *reinterpret_cast<float4 *>(scale + lane * 16) = make_float4(sv[0][0], sv[0][G - 1], sv[1][0], sv[1][G - 1]);
            else
                *reinterpret_cast<float2 *>(scale + lane * 8) = make_float2(sv[0][0], sv[1][0]);
        }

        // ---- scores: the tiles' chains of products side by side
        float s[kTiles][NB][4];
        {
            uint32_t kw[2 * kTiles][W], kp[kTiles][2][G];    // codes; key parameters of positions g and g + 8 of a tile
#pragma unroll
            for (int i = 0; i < 2 * kTiles; ++i) lds_words<P::kPiece>(mine + (i * 32 + lane) * P::kPiece, kw[i]);
            uint32_t tq[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
                tq[nb] = *reinterpret_cast<const uint32_t *>(smem + P::kT + (8 * nb + g) * 16 + 4 * t);
#pragma unroll
            for (int tile = 0; tile < kTiles; ++tile) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const unsigned char *src = par + (16 * tile + 8 * half + g) * 8 * G;
                    if constexpr (G == 2) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(src);
                        kp[tile][half][0] = v.x;
                        kp[tile][half][G - 1] = v.y;
                    } else {
                        kp[tile][half][0] = *reinterpret_cast<const uint32_t *>(src);
                    }
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    mma_bf16(s[tile][nb], __byte_perm(kp[tile][0][0], kp[tile][0][G - 1], pick),
                             __byte_perm(kp[tile][1][0], kp[tile][1][G - 1], pick), tq[nb]);
            }
#pragma unroll
            for (int k = 0; k < G; ++k) {
                float acc[kTiles][NB][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t q[NB][2];
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            lds_words<8>(smem + P::kQ + (8 * nb + g) * P::kQRow + (64 * k + 16 * t + 8 * j + 4 * h) * 2,
                                         q[nb]);
#pragma unroll
                        for (int tile = 0; tile < kTiles; ++tile) {
                            uint32_t x0[4], x1[4];
                            code_operands(kw[2 * tile][2 * k + j], x0);
                            code_operands(kw[2 * tile + 1][2 * k + j], x1);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                if (j == 0 && h == 0)
                                    mma_first(acc[tile][nb], x0[0], x1[0], x0[1], x1[1], q[nb][0], q[nb][1]);
                                else
                                    mma(acc[tile][nb], x0[2 * h], x1[2 * h], x0[2 * h + 1], x1[2 * h + 1], q[nb][0], q[nb][1]);
                        }
                    }
#pragma unroll
                for (int tile = 0; tile < kTiles; ++tile)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float sk = __uint_as_float(kp[tile][half][k] << 16);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            float *u = s[tile][nb] + 2 * half;
                            const float *x = acc[tile][nb] + 2 * half;
                            const float2 v = upk(fma2(pk(sk, sk), pk(x[0], x[1]), pk(u[0], u[1])));
                            u[0] = v.x;
                            u[1] = v.y;
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
        // keys and parameters are read: the next block's may come
        __syncwarp();
        if (more && !lost) copy_keys(blk + 1);


        // ---- the block's maxima of scores and of value scales' exponents, per row
        float mb[NB][2];
        int es[NB][2];
        if (full) {
            // s < 2^e
            const int e_all = max(kMinExp, static_cast<int>(top_scale >> 23) - 126);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) es[nb][0] = es[nb][1] = e_all;
        } else {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) es[nb][0] = es[nb][1] = kMinExp;
#pragma unroll
            for (int tile = 0; tile < kTiles; ++tile)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t *w = reinterpret_cast<const uint32_t *>(scale + (16 * tile + 8 * half + g) * 4 * G);
                    const int e = static_cast<int>(max(w[0], w[G - 1]) >> 23) - 126;
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
                    for (int y = 4; y < 32; y <<= 1) es[nb][i] = max(es[nb][i], __shfl_xor_sync(0xffffffffu, es[nb][i], y));
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
                for (int y = 4; y < 32; y <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
                const float2 ff = upk(f[nb]);
                mb[nb][i] = top * (i ? ff.y : ff.x);       // in units of log2
            }
            const float r0 = mb[nb][0] == -INFINITY ? 0.0f : mb[nb][0], r1 = mb[nb][1] == -INFINITY ? 0.0f : mb[nb][1];
            ref[nb] = pk(static_cast<float>(15 - es[nb][0]) - r0, static_cast<float>(15 - es[nb][1]) - r1);
        }

        // ---- weights, rounded to f16 after the value's scale, as operands
        uint32_t w16[kTiles][G][NB][2];
        f2 lb[NB];
        float zb[G][NB][4];                               // rows 0 and 1 (lanes g = 0 and 1): the parts of the minima's term
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) lb[nb] = 0;
#pragma unroll
        for (int tile = 0; tile < kTiles; ++tile) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float *sv = reinterpret_cast<const float *>(scale + (16 * tile + 8 * half + g) * 4 * G);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    const float2 y = upk(fma2(pk(s[tile][nb][2 * half], s[tile][nb][2 * half + 1]), f[nb], ref[nb]));
                    const float w0 = ex2(y.x), w1 = ex2(y.y);
                    lb[nb] = add2(lb[nb], pk(w0, w1));
#pragma unroll
                    for (int k = 0; k < G; ++k) {
                        const float2 ws = upk(mul2(pk(w0, w1), pk(sv[k], sv[k])));
                        const __half2 h = __floats2half2_rn(ws.x, ws.y);
                        w16[tile][k][nb][half] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h));
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < G; ++k) {
                const uint2 r = *reinterpret_cast<const uint2 *>(my_ratio + (tile * G + k) * ratio_step);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                    if (tile == 0)
                        mma_first(zb[k][nb], r.x, 0u, r.y, 0u, w16[tile][k][nb][0], w16[tile][k][nb][1]);
                    else
                        mma(zb[k][nb], r.x, 0u, r.y, 0u, w16[tile][k][nb][0], w16[tile][k][nb][1]);
            }
        }

        // ---- the fold of sums and maxima; in a cluster, blocks are folded where all of them meet
        f2 wa[NB], wo[NB], wq[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            if constexpr (SPLIT) {
                m[nb][0] = mb[nb][0], m[nb][1] = mb[nb][1];
                if (g == 0)
                    *reinterpret_cast<int2 *>(smem + P::kE + (warp * P::R + 8 * nb + 2 * t) * 4) =
                        make_int2(es[nb][0], es[nb][1]);
                l[nb] = times2(lb[nb], kFoldSum);
#pragma unroll
                for (int k = 0; k < G; ++k)
                    z[nb][k] = fma2(pk(zb[k][nb][0], zb[k][nb][1]), pk(kFoldSum, kFoldSum), z[nb][k]);   // on 0 or NaN
            } else {
                float u[2], v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) m[nb][i] = fold_weights(m[nb][i], mb[nb][i], es[nb][i], u[i], v[i]);
                wa[nb] = pk(u[0], u[1]);
                const f2 wb = pk(v[0], v[1]);
                l[nb] = fold2(l[nb], wa[nb], times2(lb[nb], kFoldSum), wb);
#pragma unroll
                for (int k = 0; k < G; ++k)
                    z[nb][k] = fold2(z[nb][k], wa[nb], times2(pk(zb[k][nb][0], zb[k][nb][1]), kFoldSum), wb);
                wo[nb] = times2(wb, kFoldEven);
                wq[nb] = times2(wb, kFoldOdd);
            }
        }

        // ---- weighted values
        wait(1, blk, more && !lost);
        {
            uint32_t vw[2 * kTiles][W];
#pragma unroll
            for (int i = 0; i < 2 * kTiles; ++i)
                lds_words<P::kPiece>(mine + P::kCodes + (i * 4 + t) * Kv4Layout::v_pair(D) + g * P::kPiece, vw[i]);
#pragma unroll
            for (int k = 0; k < G; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float acc[2][NB][4];
#pragma unroll
                    for (int tile = 0; tile < kTiles; ++tile) {
                        uint32_t x0[4], x1[4];
                        byte_operands(vw[2 * tile][2 * k + j], x0);
                        byte_operands(vw[2 * tile + 1][2 * k + j], x1);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
                                if (tile == 0)
                                    mma_first(acc[h][nb], x0[2 * h], x0[2 * h + 1], x1[2 * h], x1[2 * h + 1],
                                              w16[tile][k][nb][0], w16[tile][k][nb][1]);
                                else
                                    mma(acc[h][nb], x0[2 * h], x0[2 * h + 1], x1[2 * h], x1[2 * h + 1], w16[tile][k][nb][0],
                                        w16[tile][k][nb][1]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            f2 *u = o[k][2 * j + h][nb];   // elements 2 h and 2 h + 1 of the word, two rows each
                            const f2 odd = pk(acc[h][nb][2], acc[h][nb][3]),
                                     even = fma2(odd, pk(-1.0f, -1.0f), pk(acc[h][nb][0], acc[h][nb][1]));
                            u[0] = SPLIT ? times2(even, kFoldEven) : fold2(u[0], wa[nb], even, wo[nb]);
                            u[1] = SPLIT ? times2(odd, kFoldOdd) : fold2(u[1], wa[nb], odd, wq[nb]);
                        }
                }
        }
        __syncwarp();
        if (more && !lost) copy_values(blk + 1);
    }
    __syncwarp();                                          // the warp's codes are read; its results take their place

    float *sm = reinterpret_cast<float *>(smem + P::kM), *sl = reinterpret_cast<float *>(smem + P::kL);
    // sums over the lanes that share a row (after the fold, lane by lane)
    auto over_lanes = [&](f2 v) {
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) v = add2(v, __shfl_xor_sync(0xffffffffu, v, i));
        return v;
    };
    float *ow = reinterpret_cast<float *>(mine);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        if (g == 0)
            *reinterpret_cast<float2 *>(sm + warp * P::R + 8 * nb + 2 * t) = make_float2(m[nb][0], m[nb][1]);
        if constexpr (SPLIT) {
            // l of every lane, [nb][lane]; z of the lanes that have some (g < 2), [nb][group][lane]
            f2 *lz = reinterpret_cast<f2 *>(mine + P::kO);
            lz[nb * 32 + lane] = l[nb];
#pragma unroll
            for (int k = 0; k < G; ++k) {
                if (g < 2) lz[(32 + 8 * k) * NB + nb * 8 + lane] = z[nb][k];
                z[nb][k] = 0;
            }
        } else {
            const f2 sum = over_lanes(l[nb]);
            if (g == 0) *reinterpret_cast<f2 *>(sl + warp * P::R + 8 * nb + 2 * t) = sum;
#pragma unroll
            for (int k = 0; k < G; ++k) z[nb][k] = over_lanes(z[nb][k]);
        }
#pragma unroll
        for (int k = 0; k < G; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 e0 = upk(o[k][2 * j][nb][0]), e1 = upk(o[k][2 * j][nb][1]), e2 = upk(o[k][2 * j + 1][nb][0]),
                             e3 = upk(o[k][2 * j + 1][nb][1]), zz = upk(z[nb][k]);
                float *dst = ow + (8 * nb + 2 * t) * D + 64 * k + 8 * g + 4 * j;
                if constexpr (SPLIT) {
                    *reinterpret_cast<float4 *>(dst) = make_float4(e0.x, e1.x, e2.x, e3.x);
                    *reinterpret_cast<float4 *>(dst + D) = make_float4(e0.y, e1.y, e2.y, e3.y);
                } else {
                    *reinterpret_cast<float4 *>(dst) = make_float4(e0.x + zz.x, e1.x + zz.x, e2.x + zz.x, e3.x + zz.x);
                    *reinterpret_cast<float4 *>(dst + D) = make_float4(e0.y + zz.y, e1.y + zz.y, e2.y + zz.y, e3.y + zz.y);
                }
            }
    }
    // a CTA's share of the rows' elements, 4 each: all of them, or an eighth
    constexpr int kItems = P::R * D / 4 / (SPLIT ? kCluster : 1);
    const float *maxima = sm;
    if constexpr (SPLIT) {
        cluster_sync_all();                                // the cluster's results are in its shared memory
        // The CTA ends with NB whole rows: 8 nb + 2 tr + i, i below.  Chunk `warp`: block j is warp `warp` of CTA j.  Sums
        // are folded lane by lane as a single warp would, then added over the lanes.  A block that no row sees has
        // maxima of -inf, and folding it in changes nothing.
        const int nbr = NB == 2 ? rank / 4 : 0, tr = NB == 2 ? rank % 4 : rank / 2;
        float *chunk_max = reinterpret_cast<float *>(smem + P::kC);
        uint32_t cta[kCluster];
        f2 mj[kChunkBlocks], ej[kChunkBlocks], lj[kChunkBlocks], zj[kChunkBlocks][G], ll = 0, zz[G];
#pragma unroll
        for (int j = 0; j < kChunkBlocks; ++j) {
            cta[j] = cluster_map(smem_u32(smem), j);
            const uint32_t lz = cta[j] + warp * P::kWarp + P::kO;
            mj[j] = ld_cluster_b64(cta[j] + P::kM + (warp * P::R + 8 * nbr + 2 * tr) * 4);
            ej[j] = ld_cluster_b64(cta[j] + P::kE + (warp * P::R + 8 * nbr + 2 * tr) * 4);
            lj[j] = ld_cluster_b64(lz + (nbr * 32 + 4 * g + tr) * 8);
#pragma unroll
            for (int k = 0; k < G; ++k)
                zj[j][k] = ld_cluster_b64(lz + ((32 + 8 * k) * NB + nbr * 8 + 4 * (g & 1) + tr) * 8);
        }
        f2 fa[kChunkBlocks], fb[kChunkBlocks];
        float mm[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < G; ++k) zz[k] = 0;
#pragma unroll
        for (int j = 0; j < kChunkBlocks; ++j) {
            const float2 x = upk(mj[j]);
            float u[2], v[2];
            mm[0] = fold_weights(mm[0], x.x, static_cast<int>(ej[j]), u[0], v[0]);
            mm[1] = fold_weights(mm[1], x.y, static_cast<int>(ej[j] >> 32), u[1], v[1]);
            fa[j] = pk(u[0], u[1]);
            fb[j] = pk(v[0], v[1]);
            ll = fold2(ll, fa[j], lj[j], fb[j]);
#pragma unroll
            for (int k = 0; k < G; ++k) zz[k] = fold2(zz[k], fa[j], zj[j][k], fb[j]);
        }
        const f2 sum = over_lanes(ll);
        if (lane == 0) {
            *reinterpret_cast<f2 *>(sl + warp * P::R + 8 * nbr + 2 * tr) = sum;
            *reinterpret_cast<float2 *>(chunk_max + warp * P::R + 8 * nbr + 2 * tr) = make_float2(mm[0], mm[1]);
        }
        float2 zr[G];
#pragma unroll
        for (int k = 0; k < G; ++k) zr[k] = upk(over_lanes(g < 2 ? zz[k] : 0ull));
        // the rows' elements of the chunk, 4 a lane
        for (int i = lane; i < kItems; i += 32) {
            const int e = rank * kItems + i, rl = e / (D / 4), d = e % (D / 4) * 4;
            const bool odd = rl & 1;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f), u[kChunkBlocks];
#pragma unroll
            for (int j = 0; j < kChunkBlocks; ++j) u[j] = ld_cluster_f4(cta[j] + warp * P::kWarp + (rl * D + d) * 4);
#pragma unroll
            for (int j = 0; j < kChunkBlocks; ++j) {
                const float2 a2 = upk(fa[j]), b2 = upk(fb[j]);
                const float wx = odd ? a2.y : a2.x, wy = odd ? b2.y : b2.x;
                v.x = __fmaf_rn(u[j].x, wy, v.x * wx);
                v.y = __fmaf_rn(u[j].y, wy, v.y * wx);
                v.z = __fmaf_rn(u[j].z, wy, v.z * wx);
                v.w = __fmaf_rn(u[j].w, wy, v.w * wx);
            }
            const float2 zk = G == 2 && d >= kKv4Group ? zr[G - 1] : zr[0];
            const float z1 = odd ? zk.y : zk.x;
            reinterpret_cast<float4 *>(smem + P::kV)[warp * kItems + i] = make_float4(v.x + z1, v.y + z1, v.z + z1, v.w + z1);
        }
        maxima = chunk_max;
        __syncwarp();
        cluster_arrive();                                  // this CTA has read what it needs of the others
    }
    __syncthreads();

    // ---- the span's chunks joined in order
    for (int i = threadIdx.x; i < kItems; i += kThreads) {
        const int e = rank * kItems + i, rl = e / (D / 4), d = e % (D / 4) * 4, r = rows.r0 + rl;
        if (r > rows.r_last) break;
        const int tok = rows.token(r), n = rows.first + tok + 1;
        if (p0 >= n && (span > 0 || n > 0)) continue;
        float mc[kChunks], top = -INFINITY, sum = 0.0f;
        float4 vc[kChunks];
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
            mc[ch] = maxima[ch * P::R + rl];
            if constexpr (SPLIT)
                vc[ch] = reinterpret_cast<const float4 *>(smem + P::kV)[ch * kItems + i];
            else
                vc[ch] = *reinterpret_cast<const float4 *>(smem + ch * P::kWarp + (rl * D + d) * 4);
            top = fmaxf(top, mc[ch]);
        }
        const float base = top == -INFINITY ? 0.0f : top;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) {
            const float w = ex2(mc[ch] - base);
            sum = __fmaf_rn(w, sl[ch * P::R + rl], sum);
            v.x = __fmaf_rn(w, vc[ch].x, v.x);
            v.y = __fmaf_rn(w, vc[ch].y, v.y);
            v.z = __fmaf_rn(w, vc[ch].z, v.z);
            v.w = __fmaf_rn(w, vc[ch].w, v.w);
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

    // ---- the last CTA of a row block, or in clusters the last of a rank (which holds whole rows), joins the spans
    if constexpr (SPLIT) {
        __syncwarp();
        cluster_wait();                                    // no CTA leaves while another reads its shared memory
    }
    if (!p.count || n_most <= kSpan) return;
    int *flag = reinterpret_cast<int *>(smem + P::kFlag);
    __syncthreads();
    if (threadIdx.x == 0) {
        int *counter = reinterpret_cast<int *>(static_cast<char *>(a.ws) + kStatusBytes) +
                       ((static_cast<int64_t>(b) * c.Hkv + rows.hk) * p.row_blocks + rb) * (SPLIT ? kCluster : 1) + rank;
        const bool last = atom_add_acq_rel_gpu(counter, 1) == (n_most + kSpan - 1) / kSpan - 1;
        if (last) *counter = 0;
        *flag = last;
    }
    __syncthreads();
    if (!*flag) return;
    for (int i = threadIdx.x; i < kItems; i += kThreads) {
        const int e = rank * kItems + i, rl = e / (D / 4), d = e % (D / 4) * 4, r = rows.r0 + rl;
        if (r > rows.r_last) break;
        const int tok = rows.token(r), n = rows.first + tok + 1;
        if (n <= kSpan) continue;
        const int64_t at = static_cast<int64_t>(rows.t0 + tok) * a.Hq + rows.hk * rows.GH + r - tok * rows.GH;
        const float *part =
            reinterpret_cast<const float *>(static_cast<char *>(a.ws) + kCounterBytes) + at * p.spans * (D + 4);
        const int C = (n + kSpan - 1) / kSpan;
        // at most kJoinSpans: their maxima and sums, and the values of eight, are on their way at once
        float2 ml[kJoinSpans];
        float4 x[8], v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kJoinSpans; ++j) {
            ml[j] = make_float2(-INFINITY, 0.0f);
            if (j < C) ml[j] = __ldcg(reinterpret_cast<const float2 *>(part + static_cast<int64_t>(j) * (D + 4)));
            if (j < 8 && j < C) x[j] = __ldcg(reinterpret_cast<const float4 *>(part + static_cast<int64_t>(j) * (D + 4) + 4 + d));
        }
#pragma unroll
        for (int j = 0; j < kJoinSpans; ++j) top = fmaxf(top, ml[j].x);
        if (top > -INFINITY) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < C) add_span(ml[j], x[j], top, v, sum);
#pragma unroll
            for (int j = 8; j < kJoinSpans; ++j)
                if (j < C)
                    add_span(ml[j], __ldcg(reinterpret_cast<const float4 *>(part + static_cast<int64_t>(j) * (D + 4) + 4 + d)),
                             top, v, sum);
        }
        write_out<D>(a, at, d, v, sum);
    }
}

// CTAs a SM: the registers decide.  16 rows of head size 128 spill at three (b 64, q 8, 4096 positions: 148 us, at
// two 140); 8 rows of it, or 16 of head size 64, wait less for one another's copies at three than at four
// (b 96, 8191: 128 and 131 us; head size 64, b 6, q 5, 40000: 50 and 53); head size 64 wants five (b 64, 8192: 33 us, at
// four 37).
template <int D, int NB, bool SPLIT>
constexpr int kCtasPerSm = D * NB > 128 && !SPLIT ? 2 : D * NB > 64 ? 3 : SPLIT ? 4 : 5;

template <int D, int NB, bool SPLIT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<D, NB, SPLIT>) attn_kv4_span_kernel(SpanArgs p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const Kv4View &c = p.a.c;
    // the spans are the slowest axis: the short last spans of a batch come last
    Task task;
    task.rank = SPLIT ? blockIdx.x % kCluster : 0;
    const int x = SPLIT ? blockIdx.x / kCluster : blockIdx.x;
    task.hk = x / p.row_blocks;
    task.rb = x - task.hk * p.row_blocks;
    task.b = blockIdx.y;
    task.span = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.pdl) pdl_wait();
    pdl_launch_dependents();

    // the warp's blocks are 4 rank + warp and every fourth after it; lane 4 j + i looks after positions 16 i .. of the
    // j-th: their page (the lengths are on their way meanwhile)
    task.my_pos = task.span * kSpan + ((task.rank + (lane >> 2)) * kChunks + warp) * kBlock + 16 * (lane & 3);
    task.page = lane < Plan<D, NB, SPLIT>::kBlocks * 4 ? kv4_page(c, task.b, task.my_pos) : -1;
    task.cu0 = __ldg(c.cu_q + task.b);
    task.cu1 = __ldg(c.cu_q + task.b + 1);
    task.len = __ldg(c.kv_len + task.b);
    if constexpr (NB == 2) {
        // a last block of at most 8 rows does not pay for 16
        if (task.live(c) * (p.a.Hq / c.Hkv) - task.rb * 16 <= 8) return span_task<D, 1, SPLIT>(p, task, 16, smem);
    }
    span_task<D, NB, SPLIT>(p, task, 8 * NB, smem);
}

// One CTA per (token, q head), where the span kernel does not join a row's
// spans itself: eight groups of D / 4 threads take runs of kJoinSpans spans in
// turn, and their sums are added in order.  (Rows of at most one run get the
// bits of the span kernel's own join: the other groups' sums are zeros.)
template <int D>
__global__ void __launch_bounds__(2 * D) attn_kv4_join_kernel(AttnKv4Args a, int spans)
{
    constexpr int L = D / 4;
    __shared__ float red[2 * D / 32];
    __shared__ float4 vs[8][L];
    __shared__ float ss[8];
    const int tid = threadIdx.x, group = tid / L, d = tid % L * 4;
    const int t = blockIdx.x / a.Hq;
    pdl_wait();
    const int b = kv4_sequence(a.c, t);
    if (b < 0) return;
    const int begin = __ldg(a.c.cu_q + b), end = __ldg(a.c.cu_q + b + 1);
    const int n = __ldg(a.c.kv_len + b) - (end - t) + 1;
    if (t - begin >= a.c.max_q || n > a.c.max_kv || n <= kSpan) return;
    const int C = (n + kSpan - 1) / kSpan;
    const float *part = reinterpret_cast<const float *>(static_cast<char *>(a.ws) + kCounterBytes) +
                        static_cast<int64_t>(blockIdx.x) * spans * (D + 4);
    float top = -INFINITY;
    for (int c = tid; c < C; c += 2 * D) top = fmaxf(top, __ldcg(part + static_cast<int64_t>(c) * (D + 4)));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    if (tid % 32 == 0) red[tid / 32] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2 * D / 32; ++w) top = fmaxf(top, red[w]);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    if (top > -INFINITY)
        for (int c = group * kJoinSpans; c < C; c += 8 * kJoinSpans)
#pragma unroll 8
            for (int j = c; j < min(C, c + kJoinSpans); ++j) {
                const float *from = part + static_cast<int64_t>(j) * (D + 4);
                add_span(__ldcg(reinterpret_cast<const float2 *>(from)), __ldcg(reinterpret_cast<const float4 *>(from + 4 + d)),
                         top, v, sum);
            }
    vs[group][tid % L] = v;
    if (d == 0) ss[group] = sum;
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int j = 1; j < 8; ++j) {
        const float4 u = vs[j][tid];
        v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        sum += ss[j];
    }
    write_out<D>(a, blockIdx.x, d, v, sum);
}

int spans_of(int max_kv) { return (max_kv + kSpan - 1) / kSpan; }

template <int D, int NB, bool SPLIT>
cudaError_t launch_span(const SpanArgs &p, cudaStream_t stream)
{
    constexpr int bytes = Plan<D, NB, SPLIT>::kBytes;
    const cudaError_t e =
        cudaFuncSetAttribute(attn_kv4_span_kernel<D, NB, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.a.c.Hkv * p.row_blocks) * (SPLIT ? kCluster : 1),
                       static_cast<unsigned>(p.a.c.B), static_cast<unsigned>(p.spans));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (SPLIT) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = kCluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (p.pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, attn_kv4_span_kernel<D, NB, SPLIT>, p);
}

template <int D, int NB>
cudaError_t launch_span(const SpanArgs &p, bool split, cudaStream_t stream)
{
    return split ? launch_span<D, NB, true>(p, stream) : launch_span<D, NB, false>(p, stream);
}

}  // namespace

size_t attention_kv4_workspace(int Hq, int D, int T, int max_kv)
{
    const int spans = spans_of(max_kv);
    return kCounterBytes + (spans == 1 ? 0 : static_cast<size_t>(T) * Hq * spans * (D + 4) * sizeof(float));
}

cudaError_t launch_attention_kv4(const AttnKv4Args &a, int D, bool pdl, cudaStream_t stream)
{
    const int GH = a.Hq / a.c.Hkv, rows = a.c.max_q * GH;
    SpanArgs p;
    p.a = a;
    p.magic = (1ull << 32) / GH + 1;
    p.spans = spans_of(a.c.max_kv);
    p.pdl = pdl ? 1 : 0;
    // 16 rows a CTA where there are as many, 8 while their clusters leave an SM at most two CTAs (b 1, 8 tokens, 2000
    // positions: 8.9 us, with 16 rows 10.2; b 1, 4 tokens, 4104, above that: 12.6, with 16 12.1).  A span a cluster while
    // all the clusters fit at once, by the CTAs a SM that the registers leave them, a span a CTA after that.  Clusters and
    // CTAs on 152 SMs, spans of 2048: 8 rows of head size 128, 64, 72, 80 and 96 spans: 12.3, 12.7, 15.5, 18.4 and 15.5 us;
    // head size 64, 72 and 80: 9.4, 13.3 and 12.3; with 16 rows, 72 and 80: 11.5, 15.3 and 14.2; 16 rows of head size 128,
    // 40, 48 and 56 spans: 13.6, 14.2, 20.7 and 19.4.
    const int64_t heads = static_cast<int64_t>(a.c.B) * a.c.Hkv;
    const bool two = rows > 8 && kCluster * heads * ((rows + 7) / 8) * p.spans > 2 * a.sms;
    p.row_blocks = two ? (rows + 15) / 16 : (rows + 7) / 8;
    const bool split = (D == 128 && two ? 3 : 2) * heads * p.row_blocks * p.spans <= a.sms;
    p.count = heads * p.row_blocks * (split ? kCluster : 1) <= kCounters && p.spans <= kJoinSpans;
    cudaError_t e;
    if (D == 64)
        e = two ? launch_span<64, 2>(p, split, stream) : launch_span<64, 1>(p, split, stream);
    else
        e = two ? launch_span<128, 2>(p, split, stream) : launch_span<128, 1>(p, split, stream);
    if (e != cudaSuccess || p.count || p.spans == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.c.T) * a.Hq);
    cfg.blockDim = dim3(2 * D);
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
