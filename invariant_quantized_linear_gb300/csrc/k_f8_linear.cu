// e4m3 linear with a scale for each 128 elements of a row of q and each
// 128 x 128 block of the weights, alone or grouped by expert:
//   y[r, n] = bf16_rne(acc),  acc = fma(d_b, RN(s_a[r, b] s_w[n / 128, b]), acc)
// over the blocks b of K in order, from acc = 0, where d_b is the tensor cores'
// fp32 sum of the block's 128 products.
//
// One order for every form.  A row's bits may not depend on the rows that share
// the call, and d_b is not an exact sum, so every form issues the same
// instructions for an element: weights are the MMA's M = 128 rows, tokens its N
// columns (16 .. 192 of them), a block is four K = 32 slices in order into an
// accumulator that starts at 0, and no form splits K.  Work is split over weight
// rows and tokens alone.
//
// Roles of a CTA (one a SM, persistent):
//   warp 0     copies weight and token tiles into a ring, one or two blocks of K a stage;
//   warp 1     allocates TMEM, issues the MMAs, a block an accumulator;
//   warps 2-3  multiply the scales of 8 blocks ahead into a table;
//   warps 4-7  where src names the token rows: fetch them;
//   the others take each accumulator out of TMEM into the fp32 sums, then store:
//              32 weight rows and all or half of the tokens a warp.
//
// Tiles.  Expert e with n_e rows has ceil(n_e / cols) token tiles.  Calls that
// are bound by the weight stream cut the weight rows into units of 16, order the
// units by expert, token tile and row, and give each CTA an equal run of them, in
// tiles of up to 128 rows that are about as high as one another: every SM streams
// the same bytes, whatever N is.  A block's MMAs take about as long however few its
// rows are, so tiles of less than some 50 rows are bound by them and not by their
// bytes (16 and 32 rows for 1 x 4096 x 4096).  Calls that are bound
// by the tensor cores have units of 128 rows, dealt in turn, so that CTAs that run
// together share weight and token tiles in L2.
//
// Every wait is bounded: a role that gives up sets the status word and all
// return.  What each has in flight is waited for before (the copies of warp 0 for 1 ms
// at most, since a stage's barrier counts other warps too), and TMEM is freed.
//
// Bound.  8 x 4096 x 24576: 20.0 us, 5.0 TB/s of weights (0.74 of the copy rate),
// the stream and a CTA's start and end.  Few rows of weights: the chain of a CTA's
// blocks, one after another (1 x 4096 x 4096: 10.0 us, of which 16 stages of two blocks
// are 5, at 610 cycles; 16 x 12288 x 64: 18.0 for 96 blocks).  Nothing in the order of
// sums asks for that: several CTAs could compute the sums of blocks side by side, and
// one join them in order.
// 2048 x 4096 x 12288: 125 us, 1,650 TFLOP/s, 0.42 of twice the bf16 rate.  A CTA has
// seven tiles of 32 blocks, about 1,000 cycles a block and 2,200 to 2,600 from a tile's
// last block to the next one's first, where the tensor cores need 384 for 128 x 192 x
// 128.  By time stamps, which add a few tens of cycles to each part: the MMA warp waits
// 540, issues for 310, loops for 160; a warp of sums waits 140, reads 550, adds the
// rest for 80, loops for 155; the copies wait 665.  So the round of the two
// accumulators that TMEM holds is the period: 310 to issue, 760 until the sums see the
// commit, 550 to read, and back.  8, 12 or 16 warps of sums: 127, 134, 134 us.  This
// width spills: 24 bytes stored and 104 loaded a thread, 160 and 208 with src.
// Each role runs as a whole warp that elects a thread for the issue, without branches
// in its loop: single-thread loops and branches around copies, MMAs or TMEM loads cost
// two to four times as much.
#include "f8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tc.cuh"

#include <cuda_bf16.h>

namespace bi {

namespace {

constexpr int kTileRows = 128;
constexpr int kAhead = 8;                 // blocks of K in a scale table
constexpr int kBlockW = kTileRows * kF8Block;
constexpr unsigned long long kDrainNs = 1000000;   // for copies in flight after a wait has given up

// T: token columns of a tile at most.  GATHER: token rows are fetched by src.
template <int T_, bool GATHER_>
struct Cfg {
    static constexpr int T = T_;
    static constexpr bool GATHER = GATHER_;
    static constexpr bool kWide = T == 192;                    // tensor cores bound the call, not the weight stream
    static constexpr int kParts = T >= 64 ? 2 : 1; // warps that share a weight row's columns
    static constexpr int kCols = T / kParts;
    static constexpr int kEpiWarp0 = GATHER ? 8 : 4;
    static constexpr int kEpiWarps = 4 * kParts;
    static constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
    static constexpr int kUnit = kWide ? 128 : 16;
    static constexpr int P = T <= 64 ? 2 : 1;                  // blocks of K a stage
    static constexpr int kBlockQ = T * kF8Block;
    static constexpr int kStage = P * (kBlockW + kBlockQ);
    static constexpr int kStages = T == 128 ? 6 : T == 64 ? 4 : 5;
    static constexpr int kAccs = kWide ? 2 : 4;                // accumulators in turn, each of P blocks
    static constexpr int kAccCols = kWide ? 256 : P * T;
    static constexpr uint32_t kTmemCols = kAccCols * kAccs;
    static constexpr int kTables = kWide ? 1 : 2;              // 128-row blocks of weights that a tile meets
    static constexpr int kScaleLd = T + 4;                     // floats between a table's rows: bank-free for its writers
    static constexpr int kTable = kAhead * kScaleLd;
    static constexpr int kScales = 2 * kTables * kTable;       // floats, two tables in turn
    // 16 warps share 65,536 registers; the sums get what the others do not need.  An increase waits, without a limit, for
    // registers of the launch that were given up: launch() checks that the compiler gave it as many.
    static constexpr bool kSplit = kWide && GATHER;
    static constexpr int kRoleRegs = 72, kFetchRegs = 56, kSumRegs = 192;
    // a stage's MMAs are waited for by its producers and by the sums: no stage comes round twice before its sums are taken
    static_assert(kStages >= kAccs, "the sums see every phase of done[]");
    static_assert(kTmemCols <= 512 && kAhead % P == 0 && kStage % 1024 == 0, "layout");
};

struct Params {
    const uint8_t *q;
    const float *s_a, *s_w;
    const int32_t *src, *offsets;
    uint16_t *y;
    int q_rows, R, E, N, K, kb, nb, cols;
    int box;           // token rows of a tile's copy, where src is null
    int vec;           // eight results may be stored together
    int *status;
    int pdl;
};

constexpr int kBarBytes = 512;

template <class C>
constexpr size_t smem_bytes(int E)
{
    static_assert(1024 + C::kStages * C::kStage + C::kScales * 4 + kBarBytes + 12 * (kMaxExperts + 1) <= 227 * 1024, "fits");
    return 1024 + C::kStages * C::kStage + C::kScales * 4 + kBarBytes + 8 * (E + 1) + 4 * (E + 1);
}

template <int V>
struct Int {
    static constexpr int value = V;
};

// Position in a ring of N buffers: a consumer waits for parity `phase`, a producer for the other.
template <int N>
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++s == N) {
            s = 0;
            phase ^= 1u;
        }
    }
};

struct Tile {
    int e;
    int row0;      // first row of y (and of src)
    int n;         // tokens
    int w0, rows;  // weight rows of the expert
    int len;       // units
};

// Where a table has column m: the four of a group of 16 that a thread's fragments hold are side by side.
__device__ __forceinline__ int place(int m) { return (m & ~15) | ((m & 6) << 1) | ((m & 8) >> 2) | (m & 1); }

// The list of units, in shared memory: first unit and first row of each expert.
struct Work {
    const long long *first;
    const int *row;
    int E, N, cols, unit;
};

__device__ __forceinline__ int expert_of(const Work &w, long long x)
{
    int lo = 0, n = w.E;
    while (n > 1) {
        const int h = n >> 1;
        if (w.first[lo + h] <= x) {
            lo += h;
            n -= h;
        } else {
            n = h;
        }
    }
    return lo;
}

// A value that all lanes have, known to be one: what is derived from it may stay in
// uniform registers, where copies, MMAs and TMEM loads take their operands from
// (2048 x 4096 x 12288 when this was the only difference: 155 us, without 162).
__device__ __forceinline__ int same(int v) { return static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(v))); }

__device__ __forceinline__ long long same(long long v) { return __shfl_sync(0xffffffffu, v, 0); }

// The tile that starts at unit x of expert t.e or a later one, ending before `end`.  Called by whole warps.
__device__ __forceinline__ void tile_at(const Work &w, long long x, long long end, Tile &t)
{
    while (w.first[t.e + 1] <= x) ++t.e;
    t.e = same(t.e);
    const int n_e = w.row[t.e + 1] - w.row[t.e];
    const int tt = (n_e + w.cols - 1) / w.cols, nu = (w.N + w.unit - 1) / w.unit, per = kTileRows / w.unit;
    const int off = static_cast<int>(x - w.first[t.e]);
    int ti, u, run;
    if (per == 1) {
        u = off / tt;                                // a weight tile's token tiles side by side
        ti = off - u * tt;
        run = 1;
    } else {
        ti = off / nu;
        u = off - ti * nu;
        const long long left = end - x;
        run = left < nu - u ? static_cast<int>(left) : nu - u;   // units up to the end of the rows or of the CTA's share,
        run = (run + (run + per - 1) / per - 1) / ((run + per - 1) / per);   // in tiles that are about as high
    }
    t.len = same(run);
    t.w0 = same(u * w.unit);
    t.rows = min(t.len * w.unit, w.N - t.w0);
    const int c = ((n_e + tt - 1) / tt + 15) & ~15;            // tokens of a tile, spread evenly
    t.row0 = same(w.row[t.e] + ti * c);
    t.n = same(min(c, n_e - ti * c));
}

// Adds the blocks of a tile, 16 NG columns of 32 rows, into acc: columns 8 j + 2 (lane % 4), + 1 of row lane / 4 + 8 i
// are in acc[8 j + 2 i], + 1.  NG is a constant because a branch around each group's TMEM loads would order them one behind
// the other (2048 x 4096 x 12288 took 290 us with them, 142 without).  table[h]: where the scales of rows 16 h on are.
template <class C, int NG>
__device__ __forceinline__ bool sum_blocks(float *acc, int blocks, const float *scales, const int (&table)[2], uint32_t from,
                                           uint64_t *done, uint64_t *acc_empty, uint64_t *sc_full, uint64_t *sc_empty,
                                           Ring<C::kStages> &ring, Ring<C::kAccs> &accs, Ring<2> &tabs, volatile int *abort_flag)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int g = 0; g < 16 * NG; ++g) acc[g] = 0.0f;
    bool ready = false;                              // the next accumulator has been seen to be full
    // NB blocks of an accumulator, whose scales start at sc
    auto unit = [&](auto nb, const float *sc) {
        constexpr int NB = decltype(nb)::value;
        const int a = accs.s;
        // warp-uniform: the TMEM loads below are warp-collective
        if (!__all_sync(0xffffffffu, ready || mbar_wait_short(&done[ring.s], ring.phase, abort_flag))) return false;
        ring.next();
        accs.next();
        tc::fence_after();
        // 16 columns are on their way from TMEM while the 16 before them are added
        uint32_t d[2][16];
        auto fetch = [&](int i) {
            const uint32_t at = from + a * C::kAccCols + i / (NG > 0 ? NG : 1) * C::T + 16 * (i % (NG > 0 ? NG : 1));
            tc::ld16_frag(at, d[i & 1]);
            tc::ld16_frag(at + (16u << 16), d[i & 1] + 8);
        };
        if (NG > 0) fetch(0);
#pragma unroll
        for (int u = 0; u < NG * NB; ++u) {
            const int g = u % (NG > 0 ? NG : 1);
            const float *f0 = sc + u / (NG > 0 ? NG : 1) * C::kScaleLd + 16 * g;
            const float4 lo = *reinterpret_cast<const float4 *>(f0 + table[0]);
            const float4 hi = C::kTables == 2 ? *reinterpret_cast<const float4 *>(f0 + table[1]) : lo;
            tc::wait_ld();
            if (u + 1 < NG * NB) {
                fetch(u + 1);
            } else {
                // the accumulator is in registers: the next one is looked at while it is added
                tc::fence_before();
                if (lane == 0) mbar_arrive(&acc_empty[a]);
                ready = mbar_test_wait(&done[ring.s], ring.phase);
            }
            const uint32_t(&v)[16] = d[u & 1];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 &f = i < 2 ? lo : hi;
                    const int r = 8 * (i >> 1) + 4 * j + 2 * (i & 1);
                    float *s = acc + 2 * (8 * g + 4 * j + i);
                    s[0] = __fmaf_rn(__uint_as_float(v[r]), j ? f.z : f.x, s[0]);
                    s[1] = __fmaf_rn(__uint_as_float(v[r + 1]), j ? f.w : f.y, s[1]);
                }
        }
        if (NG == 0 && lane == 0) mbar_arrive(&acc_empty[a]);
        return true;
    };
    for (int k0 = 0; k0 < blocks; k0 += kAhead) {
        if (!__all_sync(0xffffffffu, mbar_wait_short(&sc_full[tabs.s], tabs.phase, abort_flag))) return false;
        const float *sc = scales + tabs.s * C::kTables * C::kTable;
        const int n = min(kAhead, blocks - k0);
        int i = 0;
        for (; i + C::P <= n; i += C::P)
            if (!unit(Int<C::P>(), sc + i * C::kScaleLd)) return false;
        if (i < n && !unit(Int<1>(), sc + i * C::kScaleLd)) return false;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_empty[tabs.s]);
        tabs.next();
    }
    return true;
}

// The same for `groups` groups, at most NG.
template <class C, int NG, typename... Rest>
__device__ __forceinline__ bool sum_any(int groups, Rest &&...rest)
{
    if constexpr (NG > 0) {
        if (groups < NG) return sum_any<C, NG - 1>(groups, rest...);
    }
    return sum_blocks<C, NG>(rest...);
}

// Stores 16 NG columns (tokens from c0 on) of the weight rows r0 .. r0 + 31 of a tile.  Eight tokens at a time are
// transposed: lane i then has token i / 4 and the weight rows 8 j + 2 (i % 4), + 1 in word j; where rows of y allow it,
// the four lanes of a token exchange words so that each stores 16 bytes (64 side by side a token).  Bit g of `nowhere`:
// src sends the g-th of a lane's tokens nowhere.
template <class C, int NG>
__device__ __forceinline__ void store_tile(const float *acc, const Params &p, const Tile &t, int c0, int r0, uint32_t nowhere)
{
    const int lane = threadIdx.x & 31, quad = lane & 3;
    const bool wide = p.vec && r0 + 32 <= t.rows;
    uint16_t *y = p.y + static_cast<long long>(t.row0 + c0 + (lane >> 2)) * p.N + t.w0 + r0;
    constexpr int kBatch = NG % 2 == 0 ? 4 : 2;      // groups of 8 tokens whose exchanges overlap
#pragma unroll
    for (int g0 = 0; g0 < 2 * NG; g0 += kBatch) {
        uint32_t w[kBatch][4];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 o = __floats2bfloat162_rn(acc[8 * (g0 + b) + 2 * i], acc[8 * (g0 + b) + 2 * i + 1]);
                w[b][i] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&o));
            }
        if (C::GATHER) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (nowhere >> (g0 + b) & 1) w[b][0] = w[b][1] = w[b][2] = w[b][3] = 0;
        }
        if (wide) {
            // words 4 x 4 of the quad, transposed: pairs of lanes exchange pairs of words, then single ones
            const bool b1 = quad & 1, b2 = quad & 2;
            uint32_t a[kBatch][4];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const uint32_t s0 = __shfl_xor_sync(0xffffffffu, b2 ? w[b][0] : w[b][2], 2);
                const uint32_t s1 = __shfl_xor_sync(0xffffffffu, b2 ? w[b][1] : w[b][3], 2);
                a[b][0] = b2 ? s0 : w[b][0];
                a[b][1] = b2 ? s1 : w[b][1];
                a[b][2] = b2 ? w[b][2] : s0;
                a[b][3] = b2 ? w[b][3] : s1;
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const uint32_t x0 = __shfl_xor_sync(0xffffffffu, b1 ? a[b][0] : a[b][1], 1);
                const uint32_t x1 = __shfl_xor_sync(0xffffffffu, b1 ? a[b][2] : a[b][3], 1);
                const uint4 o = make_uint4(b1 ? x0 : a[b][0], b1 ? a[b][1] : x0, b1 ? x1 : a[b][2], b1 ? a[b][3] : x1);
                const int m = 8 * (g0 + b);
                if (c0 + m + (lane >> 2) < t.n) *reinterpret_cast<uint4 *>(y + m * static_cast<long long>(p.N) + 8 * quad) = o;
            }
        } else {
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = 8 * i + 2 * quad, m = 8 * (g0 + b);
                    if (c0 + m + (lane >> 2) >= t.n) continue;
                    uint16_t *at = y + m * static_cast<long long>(p.N) + n;
                    if (r0 + n < t.rows) at[0] = static_cast<uint16_t>(w[b][i]);
                    if (r0 + n + 1 < t.rows) at[1] = static_cast<uint16_t>(w[b][i] >> 16);
                }
        }
    }
}

template <class C, int NG, typename... Rest>
__device__ __forceinline__ void store_any(int groups, const Rest &...rest)
{
    if constexpr (NG > 0) {
        if (groups < NG) return store_any<C, NG - 1>(groups, rest...);
        store_tile<C, NG>(rest...);
    }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    linear_f8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_w16,
                     const __grid_constant__ CUtensorMap map_q, Params p)
{
    constexpr int T = C::T;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *scales = reinterpret_cast<float *>(smem + C::kStages * C::kStage);
    uint64_t *full = reinterpret_cast<uint64_t *>(scales + C::kScales);   // copies landed
    uint64_t *done = full + C::kStages;                                   // MMAs complete: stage free, accumulator full
    uint64_t *acc_empty = done + C::kStages;                              // taken out
    uint64_t *sc_full = acc_empty + C::kAccs;                             // [2] table written
    uint64_t *sc_empty = sc_full + 2;                                     // [2] read
    uint64_t *drain = sc_empty + 2;                                       // all MMAs complete
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert((2 * C::kStages + C::kAccs + 4 + 1) * 8 + 8 <= kBarBytes, "barriers fit");
    long long *first = reinterpret_cast<long long *>(full + kBarBytes / 8);
    int *row = reinterpret_cast<int *>(first + p.E + 1);

    const int warp = warp_index(), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], C::GATHER ? 5 : 1);   // the weights' copies, and four warps' rows
            mbar_init(&done[s], 1);
        }
        for (int a = 0; a < C::kAccs; ++a) mbar_init(&acc_empty[a], C::kEpiWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sc_full[i], 2);
            mbar_init(&sc_empty[i], C::kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) tc::tmem_alloc(tmem_slot, C::kTmemCols);
    if (p.pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    if (warp == 2) {
        // rows and units of the experts; offsets that are out of order or range leave experts empty
        const int nu = (p.N + C::kUnit - 1) / C::kUnit;
        int top = 0;
        long long units = 0;
        if (lane == 0) row[0] = p.offsets ? max(0, min(p.R, __ldg(p.offsets))) : 0;
        __syncwarp();
        top = row[0];
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int end = top;
            if (e < p.E) end = p.offsets ? max(top, min(p.R, __ldg(p.offsets + e + 1))) : p.R;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end = max(end, v);
            }
            int begin = __shfl_up_sync(0xffffffffu, end, 1);
            if (lane == 0) begin = top;
            const long long mine = static_cast<long long>((end - begin + p.cols - 1) / p.cols) * nu;
            long long sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (e < p.E) {
                first[e] = units + sum - mine;
                row[e + 1] = end;
            }
            units += __shfl_sync(0xffffffffu, sum, 31);
            top = __shfl_sync(0xffffffffu, end, 31);
        }
        if (lane == 0) first[p.E] = units;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = static_cast<uint32_t>(same(static_cast<int>(*tmem_slot)));
    const Work work{first, row, p.E, p.N, p.cols, C::kUnit};
    const long long total = same(first[p.E]), b = blockIdx.x, G = gridDim.x;
    // this CTA's units: a run of them, or every G-th
    const long long x0 = same(C::kWide ? b : total * b / G), x1 = same(C::kWide ? total : total * (b + 1) / G);
    const int e0 = same(x0 < x1 ? expert_of(work, x0) : 0);
    auto next = [&](long long x, const Tile &t) { return C::kWide ? x + G : x + t.len; };
    auto end_of = [&](long long x) { return C::kWide ? x + 1 : x1; };

    auto fail = [&]() {
        if (!*abort_flag) {
            *abort_flag = 1;
            atomicExch(p.status, DEV_TIMEOUT);
        }
    };

    if (warp < 4) {
        if (C::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRoleRegs));
        if (warp == 0) {
            // ------------------------------------------------ copies
            Ring<C::kStages> ring;
            bool ok = true, wrapped = false;
            const uint64_t pol_w = policy_evict_first(), pol_q = policy_evict_last();
            if (lane == 0) {
                prefetch_tensormap(&map_w);
                prefetch_tensormap(&map_w16);
                if (!C::GATHER) prefetch_tensormap(&map_q);
            }
            Tile t;
            t.e = e0;
            for (long long x = x0; ok && x < x1; x = next(x, t)) {
                tile_at(work, x, end_of(x), t);
                const int wy = t.e * p.N + t.w0;
                const uint32_t bytes_q = C::GATHER ? 0 : p.box * kF8Block;
                // NW copies of 16 weight rows, or (8) one of 128; no branch but the waits'
                auto stages = [&](auto nw) {
                    constexpr int NW = decltype(nw)::value;
                    const uint32_t bytes = NW * 16 * kF8Block + bytes_q;
                    auto copy = [&](int s, int b, int k) {
                        uint8_t *sw = smem + s * C::kStage + b * kBlockW;
                        [[maybe_unused]] uint8_t *sq = smem + s * C::kStage + C::P * kBlockW + b * C::kBlockQ;
                        if constexpr (NW == 8) {
                            tma_load_2d(sw, &map_w, &full[s], k, wy, pol_w);
                        } else {
#pragma unroll
                            for (int i = 0; i < NW; ++i) tma_load_2d(sw + i * 2048, &map_w16, &full[s], k, wy + i * 16, pol_w);
                        }
                        if constexpr (!C::GATHER) tma_load_2d(sq, &map_q, &full[s], k, t.row0, pol_q);
                    };
                    int kb = 0;
                    for (; kb + C::P <= p.kb; kb += C::P) {
                        const int s = ring.s;
                        ok = __all_sync(0xffffffffu, mbar_wait_short(&done[s], ring.phase ^ 1u, abort_flag));
                        if (!ok) return;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&full[s], bytes * C::P);
#pragma unroll
                            for (int b = 0; b < C::P; ++b) copy(s, b, (kb + b) * kF8Block);
                        }
                        __syncwarp();
                        ring.next();
                        wrapped |= ring.s == 0;
                    }
                    if (kb < p.kb) {                             // the last block of an odd number
                        const int s = ring.s;
                        ok = __all_sync(0xffffffffu, mbar_wait_short(&done[s], ring.phase ^ 1u, abort_flag));
                        if (!ok) return;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&full[s], bytes);
                            copy(s, 0, kb * kF8Block);
                        }
                        __syncwarp();
                        ring.next();
                        wrapped |= ring.s == 0;
                    }
                };
                switch (t.rows > 112 ? 8 : (t.rows + 15) >> 4) {
                case 1: stages(Int<1>()); break;
                case 2: stages(Int<2>()); break;
                case 3: stages(Int<3>()); break;
                case 4: stages(Int<4>()); break;
                case 5: stages(Int<5>()); break;
                case 6: stages(Int<6>()); break;
                case 7: stages(Int<7>()); break;
                default: stages(Int<8>());
                }
            }
            if (!ok) fail();
            // Every copy that was issued lands before the CTA can exit.  After a failure the rows by src may never be handed
            // over, and a stage's barrier not turn: kDrainNs in all then.
            unsigned long long t0 = 0;
            for (int s = 0; s < C::kStages; ++s) {
                if (s >= ring.s && !wrapped) continue;
                const uint32_t parity = s < ring.s ? ring.phase : ring.phase ^ 1u;
                while (!mbar_try_wait(&full[s], parity)) {
                    const unsigned long long t = global_timer_ns();
                    if (t0 == 0) t0 = t;
                    if (t - t0 > (*abort_flag ? kDrainNs : kWaitLimitNs)) break;
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------ MMAs
            Ring<C::kStages> ring;
            Ring<C::kAccs> accs;
            bool ok = true, sound = true;
            const uint64_t dw0 = tc::sdesc_kmajor_sw128(smem_u32(smem));
            const uint64_t dq0 = tc::sdesc_kmajor_sw128(smem_u32(smem) + C::P * kBlockW);
            Tile t;
            t.e = e0;
            for (long long x = x0; ok && x < x1; x = next(x, t)) {
                tile_at(work, x, end_of(x), t);
                // rows of the stage beyond the tile's hold old bytes: their sums are never looked at
                const uint32_t idesc = tc::idesc_e4m3_f32(kTileRows, (t.n + 15) & ~15);
                auto block = [&](int s, int a, int b) {
                    const uint64_t at = static_cast<uint32_t>(s * (C::kStage >> 4));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_e4m3_ss(tmem + a * C::kAccCols + b * T, dw0 + at + b * (kBlockW >> 4) + 2 * k,
                                        dq0 + at + b * (C::kBlockQ >> 4) + 2 * k, idesc, k > 0 ? 1u : 0u);
                };
                auto stage = [&](auto nb) {
                    const int a = accs.s, s = ring.s;
                    // Half the lanes look at each barrier: one look's latency for both.  After a wait that gave up nothing is
                    // issued or committed any more: `done` would let a producer arrive at a barrier whose phase is still
                    // open.  The loop goes on to the tile's end without a way out (16 x 12288 x 64: 18.0 us so, 19.6 with
                    // a branch out of it), a microsecond a block.
                    uint64_t *bar = lane & 1 ? &full[s] : &acc_empty[a];
                    const bool there = mbar_wait_short(bar, lane & 1 ? ring.phase : accs.phase ^ 1u, abort_flag);
                    if (!there) fail();
                    sound &= __all_sync(0xffffffffu, there);
                    tc::fence_after();
                    if (elect_one() & sound) {
#pragma unroll
                        for (int b = 0; b < decltype(nb)::value; ++b) block(s, a, b);
                        tc::commit(&done[s]);
                    }
                    ring.next();
                    accs.next();
                };
                int kb = 0;
                // two stages a turn where the chain of MMAs is the call (185 x 8 of 48 experts with T = 64: 36.8 us so,
                // 34.9 one by one; 2048 x 4096 x 12288 142 and 127)
                if constexpr (T <= 32) {
                    for (; kb + 2 * C::P <= p.kb; kb += 2 * C::P) {
                        stage(Int<C::P>());
                        stage(Int<C::P>());
                    }
                }
                for (; kb + C::P <= p.kb; kb += C::P) stage(Int<C::P>());
                if (kb < p.kb) stage(Int<1>());
                __syncwarp();
                ok = !__any_sync(0xffffffffu, *abort_flag);
            }
            // the same thread as above: commit counts what its thread issued
            if (elect_one()) {
                tc::commit(drain);
                volatile int never = 0;
                mbar_wait_bounded(drain, 0, &never);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------ scales
            // lane: block lane % 8 of the table, tokens m1, m1 + 8, ...; kBatch of them on their way at once
            Ring<2> tabs;
            bool ok = true;
            Tile t;
            t.e = e0;
            constexpr int kBatch = T / 8;
            const int i = lane & 7, m1 = (lane >> 3) + 4 * (warp - 2);
            for (long long x = x0; ok && x < x1; x = next(x, t)) {
                tile_at(work, x, end_of(x), t);
                const int cols = (t.n + 15) & ~15;
                const float *sw = p.s_w + (static_cast<long long>(t.e) * p.nb + t.w0 / kF8Block) * p.kb;
                const bool two = C::kTables == 2 && t.w0 / kF8Block != (t.w0 + t.rows - 1) / kF8Block;
                for (int k0 = 0; k0 < p.kb; k0 += kAhead) {
                    ok = __all_sync(0xffffffffu, mbar_wait_short(&sc_empty[tabs.s], tabs.phase ^ 1u, abort_flag));
                    if (!ok) {
                        fail();
                        break;
                    }
                    float *table = scales + tabs.s * C::kTables * C::kTable + i * C::kScaleLd;
                    const int k = min(k0 + i, p.kb - 1);         // entries beyond the last block are not looked at
                    const float f0 = __ldg(sw + k), f1 = two ? __ldg(sw + p.kb + k) : 0.0f;
                    for (int m0 = m1; m0 < cols; m0 += 8 * kBatch) {
                        int r[kBatch];
                        float v[kBatch];
#pragma unroll
                        for (int u = 0; u < kBatch; ++u) {
                            r[u] = t.row0 + min(m0 + 8 * u, t.n - 1);
                            if (C::GATHER) r[u] = __ldg(p.src + r[u]);
                            if (static_cast<unsigned>(r[u]) >= static_cast<unsigned>(p.q_rows)) r[u] = 0;
                        }
#pragma unroll
                        for (int u = 0; u < kBatch; ++u) v[u] = __ldg(p.s_a + static_cast<long long>(r[u]) * p.kb + k);
#pragma unroll
                        for (int u = 0; u < kBatch; ++u)
                            if (m0 + 8 * u < cols) {
                                const int at = place(m0 + 8 * u);
                                table[at] = __fmul_rn(v[u], f0);
                                if (two) table[C::kTable + at] = __fmul_rn(v[u], f1);
                            }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sc_full[tabs.s]);
                    tabs.next();
                }
            }
        }
    } else if (warp < C::kEpiWarp0) {
        // ------------------------------------------------ token rows by src
        // Four rows an instruction, a lane 16 bytes: rows 16 i + 4 (warp % 4) + lane / 8.  A stage is handed over when
        // its copies have landed, kDepth - 1 stages later.  (Gathers of four rows by TMA took 32 cycles each, 1,530 a
        // block of 192.)
        if (C::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kFetchRegs));
        constexpr int kDepth = C::kStages - 1;
        const int quarter = warp & 3, r4 = 4 * quarter + (lane >> 3), chunk = lane & 7;
        const uint32_t to = smem_u32(smem) + C::P * kBlockW + r4 * 128 + ((chunk ^ (r4 & 7)) << 4);
        Ring<C::kStages> ring, landed;
        int flying = 0;
        bool ok = true;
        auto hand_over = [&]() {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[landed.s]);
            landed.next();
            --flying;
        };
        Tile t;
        t.e = e0;
        for (long long x = x0; ok && x < x1; x = next(x, t)) {
            tile_at(work, x, end_of(x), t);
            int row[T / 16];
#pragma unroll
            for (int i = 0; i < T / 16; ++i) {
                const int r = __ldg(p.src + t.row0 + min(16 * i + r4, t.n - 1));
                row[i] = static_cast<unsigned>(r) < static_cast<unsigned>(p.q_rows) ? r : 0;
            }
            for (int kb = 0; kb < p.kb; kb += C::P) {
                ok = __all_sync(0xffffffffu, mbar_wait_short(&done[ring.s], ring.phase ^ 1u, abort_flag));
                if (!ok) break;
#pragma unroll
                for (int b = 0; b < C::P; ++b) {
                    const int k = (kb + b) * kF8Block + 16 * chunk;
                    const int there = k < p.K ? 16 : 0;      // zeros behind the last element
                    const uint32_t at = to + ring.s * C::kStage + b * C::kBlockQ;
                    const uint8_t *from = p.q + (there ? k : 0);
#pragma unroll
                    for (int i = 0; i < T / 16; ++i)
                        if (16 * i < t.n) cp_async16(at + i * 2048, from + static_cast<long long>(row[i]) * p.K, there);
                }
                cp_async_commit();
                ring.next();
                if (++flying == kDepth) {
                    cp_async_wait<kDepth - 1>();
                    hand_over();
                }
            }
        }
        if (!ok) fail();
        cp_async_wait<0>();
        while (flying > 0) hand_over();
    } else {
        // ------------------------------------------------ sums and results
        if (C::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSumRegs));
        const int qd = warp & 3, part = (warp - C::kEpiWarp0) >> 2;
        Ring<C::kStages> ring;
        Ring<C::kAccs> accs;
        Ring<2> tabs;
        bool ok = true;
        Tile t;
        t.e = e0;
        for (long long x = x0; ok && x < x1; x = next(x, t)) {
            tile_at(work, x, end_of(x), t);
            const int cols = (t.n + 15) & ~15;
            const int share = (cols / C::kParts + 15) & ~15;
            const int c0 = part * share, nc = max(0, min(share, cols - c0));
            // the table of rows 32 qd + 16 h on (16 rows lie in one block of the weights)
            int table[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 32 * qd + 16 * h;
                table[h] = C::kTables == 2 && r < t.rows && (t.w0 + r) / kF8Block != t.w0 / kF8Block ? C::kTable : 0;
            }
            uint32_t nowhere = 0;                            // read here: the loads' latency passes behind the first block
            if (C::GATHER) {
#pragma unroll
                for (int g = 0; g < C::kCols / 8; ++g) {
                    const int r = __ldg(p.src + t.row0 + min(c0 + 8 * g + (lane >> 2), t.n - 1));
                    if (static_cast<unsigned>(r) >= static_cast<unsigned>(p.q_rows)) nowhere |= 1u << g;
                }
            }
            float acc[C::kCols];
            const float *sc = scales + c0 + 4 * (lane & 3);
            const uint32_t from = tmem + (static_cast<uint32_t>(32 * qd) << 16) + c0;
            ok = sum_any<C, C::kCols / 16>((nc + 15) >> 4, acc, p.kb, sc, table, from, done, acc_empty, sc_full, sc_empty, ring,
                                           accs, tabs, abort_flag);
            if (!ok) {
                fail();
                break;
            }
            store_any<C, C::kCols / 16>((nc + 15) >> 4, acc, p, t, c0, 32 * qd, nowhere);
        }
    }
    __syncwarp();
    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <class C>
cudaError_t launch(const F8LinearArgs &a, bool pdl, cudaStream_t stream)
{
    const size_t smem = smem_bytes<C>(a.E);
    // A few hundred ns of host time, and right on every device.  The opt-in is the kernel's, not the call's, so it is always
    // the largest call's: a smaller one would take it from a call that another thread is about to launch.
    cudaError_t e = cudaFuncSetAttribute(linear_f8_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem_bytes<C>(kMaxExperts)));
    if (e != cudaSuccess) return e;
    if constexpr (C::kSplit) {
        static const int regs = [] {
            cudaFuncAttributes f = {};
            return cudaFuncGetAttributes(&f, linear_f8_kernel<C>) == cudaSuccess ? f.numRegs : 0;
        }();
        if (regs * C::kThreads < 32 * (4 * C::kRoleRegs + 4 * C::kFetchRegs + C::kEpiWarps * C::kSumRegs))
            return cudaErrorLaunchOutOfResources;
    }
    Params p;
    p.q = a.q;
    p.s_a = a.s_a;
    p.s_w = a.s_w;
    p.src = a.src;
    p.offsets = a.offsets;
    p.y = a.y;
    p.q_rows = a.q_rows;
    p.R = a.R;
    p.E = a.E;
    p.N = a.N;
    p.K = a.K;
    p.kb = f8_blocks(a.K);
    p.nb = f8_blocks(a.N);
    p.cols = a.plan.cols;
    p.box = a.box;
    p.vec = a.N % 8 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15u) == 0 ? 1 : 0;
    p.status = a.status;
    p.pdl = pdl ? 1 : 0;
    // units at most: each expert's last token tile may be a part of one
    const long long tiles = a.R / a.plan.cols + (a.E < a.R ? a.E : a.R);
    const long long units = tiles * ((a.N + C::kUnit - 1) / C::kUnit);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units < a.sms ? units : a.sms));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, linear_f8_kernel<C>, a.map_w, a.map_w16, a.map_q, p);
}

}  // namespace

F8Plan f8_plan(int rows, int experts, int N, int sms)
{
    const int busy = experts < rows ? experts : rows;
    const int mean = (rows + busy - 1) / busy;
    const long long need = experts == 1 ? rows : 2LL * mean < rows ? 2 * mean : rows;
    for (int T = 16; T <= 64; T *= 2)
        if (need <= T) return {T, T};
    const long long tall = (N + kTileRows - 1) / kTileRows;
    if (mean <= 128 || busy * tall * ((mean + 191) / 192) < sms) return {128, 128};
    if (experts > 1) return {192, 192};
    // fewest tensor cycles: waves of tiles, each as long as its columns
    int best = 192;
    long long least = 1LL << 62;
    for (int cols = 192; cols > 128; cols -= 16) {
        const long long tiles = tall * ((rows + cols - 1) / cols), cost = (tiles + sms - 1) / sms * cols;
        if (cost < least) {
            least = cost;
            best = cols;
        }
    }
    return {192, best};
}

template <int T>
static cudaError_t launch_any(const F8LinearArgs &a, bool pdl, cudaStream_t stream)
{
    return a.src ? launch<Cfg<T, true>>(a, pdl, stream) : launch<Cfg<T, false>>(a, pdl, stream);
}

cudaError_t launch_linear_f8(const F8LinearArgs &a, bool pdl, cudaStream_t stream)
{
    switch (a.plan.T) {
    case 16: return launch_any<16>(a, pdl, stream);
    case 32: return launch_any<32>(a, pdl, stream);
    case 64: return launch_any<64>(a, pdl, stream);
    case 128: return launch_any<128>(a, pdl, stream);
    default: return launch_any<192>(a, pdl, stream);
    }
}

}  // namespace bi
