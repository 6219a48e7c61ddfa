// e4m3 linear with a scale for each 128 elements of a row of q and each
// 128 x 128 block of the weights, alone or grouped by expert:
//   y[r, n] = bf16_rne(acc),  acc = fma(d_b, RN(s_a[r, b] s_w[n / 128, b]), acc)
// over the blocks b of K in order, from acc = 0, where d_b is the tensor cores'
// fp32 sum of the block's 128 products.
//
// One order for every form.  A row's bits may not depend on the rows that share
// the call, and d_b is not an exact sum, so every form issues the same
// instructions for an element: weights are the MMA's M = 128 rows, tokens its N
// columns (16 .. 256 of them), a block is four K = 32 slices in order into an
// accumulator that starts at 0, and no form splits K.  Work is split over weight
// rows and tokens alone.
//
// Roles of a CTA (one a SM, persistent):
//   warp 0     copies weight and token tiles into a ring, one block of K a stage;
//              token rows that src names are gathered four at a time;
//   warp 1     allocates TMEM, issues the MMAs, a block an accumulator;
//   warp 2     multiplies the scales of 8 blocks ahead into a table;
//   warps 4 on a weight row a thread (TMEM lane), up to 128 tokens: take each
//              accumulator out of TMEM into the fp32 sums, then store.
//
// Tiles.  Expert e with n_e rows has ceil(n_e / cols) token tiles.  Calls that
// are bound by the weight stream cut the weight rows into units of 16, order the
// units by expert, 128-row chunk, token tile and row, and give each CTA an equal
// run of them: every SM streams the same bytes, whatever N is, and a chunk's
// token tiles follow one another on one SM.  Calls that are bound by the tensor
// cores have units of 128 rows, dealt in turn, so that CTAs that run together
// share weight and token tiles in L2.
//
// Every wait is bounded: a role that gives up sets the status word and all
// return; copies in flight are waited for and TMEM is freed.
#include "f8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tc.cuh"

#include <cuda_bf16.h>

namespace bi {

namespace {

constexpr int kTileRows = 128;
constexpr int kAhead = 8;                 // blocks of K in a scale table
constexpr int kEpiWarp0 = 4;
constexpr int kStageW = kTileRows * kF8Block;

template <int T>
struct Cfg {
    static constexpr int kHalves = T == 256 ? 2 : 1;           // epilogue threads a weight row
    static constexpr int kCols = T / kHalves;
    static constexpr int kEpiWarps = 4 * kHalves;
    static constexpr int kThreads = (kEpiWarp0 + kEpiWarps) * 32;
    static constexpr int kUnit = T == 256 ? 128 : 16;
    static constexpr bool kInTurn = T == 256;
    static constexpr int kStage = kStageW + T * kF8Block;
    static constexpr int kStages = T == 256 ? 4 : T == 128 ? 6 : T == 64 ? 8 : 10;
    static constexpr int kAccs = T == 256 ? 2 : T == 128 ? 4 : 8;
    static constexpr uint32_t kTmemCols = T * kAccs;
    static constexpr int kTables = T == 256 ? 1 : 2;           // 128-row blocks of weights that a tile meets
    static constexpr int kScaleLd = T + 4;                     // floats between a table's rows: bank-free for its writers
    static constexpr int kTable = kAhead * kScaleLd;
    static constexpr int kScales = 2 * kTables * kTable;       // floats, two tables in turn
};

struct Params {
    const float *s_a, *s_w;
    const int32_t *src, *offsets;
    uint16_t *y;
    int q_rows, R, E, N, K, kb, nb, cols;
    int *status;
    int pdl;
};

template <int T>
size_t smem_bytes(int E)
{
    using C = Cfg<T>;
    return 1024 + C::kStages * C::kStage + C::kScales * 4 + 512 + 8 * (E + 1) + 4 * (E + 1);
}

struct Tile {
    int e;
    int row0;      // first row of y (and of src)
    int n;         // tokens
    int w0, rows;  // weight rows of the expert
    int len;       // units
};

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

// The tile that starts at unit x of expert t.e or a later one, ending before `end`.
__device__ __forceinline__ void tile_at(const Work &w, long long x, long long end, Tile &t)
{
    while (w.first[t.e + 1] <= x) ++t.e;
    const int n_e = w.row[t.e + 1] - w.row[t.e];
    const int tt = (n_e + w.cols - 1) / w.cols, nu = (w.N + w.unit - 1) / w.unit, per = kTileRows / w.unit;
    const long long off = x - w.first[t.e];
    const int chunk = static_cast<int>(off / (per * tt));
    const int rem = static_cast<int>(off - static_cast<long long>(chunk) * per * tt);
    const int run = min(per, nu - chunk * per);
    const int ti = rem / run, u = rem - ti * run;
    const long long left = end - x;
    t.len = left < run - u ? static_cast<int>(left) : run - u;
    t.w0 = (chunk * per + u) * w.unit;
    t.rows = min(t.len * w.unit, w.N - t.w0);
    const int c = ((n_e + tt - 1) / tt + 15) & ~15;            // tokens of a tile, spread evenly
    t.row0 = w.row[t.e] + ti * c;
    t.n = min(c, n_e - ti * c);
}

template <int T>
__global__ void __launch_bounds__(Cfg<T>::kThreads, 1)
    linear_f8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_w16,
                     const __grid_constant__ CUtensorMap map_q, Params p)
{
    using C = Cfg<T>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *scales = reinterpret_cast<float *>(smem + C::kStages * C::kStage);
    uint64_t *full = reinterpret_cast<uint64_t *>(scales + C::kScales);   // copies landed
    uint64_t *empty = full + C::kStages;                                  // MMAs done reading
    uint64_t *acc_full = empty + C::kStages;                              // block summed
    uint64_t *acc_empty = acc_full + C::kAccs;                            // taken out
    uint64_t *sc_full = acc_empty + C::kAccs;                             // [2] table written
    uint64_t *sc_empty = sc_full + 2;                                     // [2] read
    uint64_t *drain = sc_empty + 2;                                       // all MMAs complete
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    static_assert((2 * C::kStages + 2 * C::kAccs + 4 + 1) * 8 + 8 <= 512, "barriers fit");
    long long *first = reinterpret_cast<long long *>(full + 64);
    int *row = reinterpret_cast<int *>(first + p.E + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < C::kAccs; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], C::kEpiWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sc_full[i], 1);
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
    const uint32_t tmem = *tmem_slot;
    const Work work{first, row, p.E, p.N, p.cols, C::kUnit};
    const long long total = first[p.E], b = blockIdx.x, G = gridDim.x;
    // this CTA's units: a run of them, or every G-th
    const long long x0 = C::kInTurn ? b : total * b / G, x1 = C::kInTurn ? total : total * (b + 1) / G;
    const int e0 = x0 < x1 ? expert_of(work, x0) : 0;
    auto next = [&](long long x, const Tile &t) { return C::kInTurn ? x + G : x + t.len; };
    auto end_of = [&](long long x) { return C::kInTurn ? x + 1 : x1; };

    auto fail = [&]() {
        if (!*abort_flag) {
            *abort_flag = 1;
            atomicExch(p.status, DEV_TIMEOUT);
        }
    };

    if (warp == 0) {
        // ------------------------------------------------ copies
        if (lane == 0) {
            prefetch_tensormap(&map_w);
            prefetch_tensormap(&map_w16);
            prefetch_tensormap(&map_q);
        }
        const uint64_t pol_w = policy_evict_first(), pol_q = policy_evict_last();
        long long j = 0;
        bool ok = true;
        Tile t;
        t.e = e0;
        for (long long x = x0; ok && x < x1; x = next(x, t)) {
            tile_at(work, x, end_of(x), t);
            const int cols = (t.n + 15) & ~15, nw = (t.rows + 15) >> 4;
            const int wy = t.e * p.N + t.w0;
            const uint32_t bytes = nw * 2048 + cols * kF8Block;
            int idx[(T + 127) / 128][4];
            if (p.src) {
#pragma unroll
                for (int i = 0; i < (T + 127) / 128; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int m = 4 * (lane + 32 * i) + k;
                        const int r = m < t.n ? __ldg(p.src + t.row0 + m) : 0;
                        idx[i][k] = static_cast<unsigned>(r) < static_cast<unsigned>(p.q_rows) ? r : 0;
                    }
            }
            for (int kb = 0; kb < p.kb; ++kb, ++j) {
                const int s = static_cast<int>(j % C::kStages);
                if (j >= C::kStages)
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&empty[s], static_cast<uint32_t>(j / C::kStages - 1) & 1u,
                                                                   abort_flag));
                if (!ok) {
                    fail();
                    break;
                }
                uint8_t *sw = smem + s * C::kStage, *sq = sw + kStageW;
                if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
                __syncwarp();
                const int k = kb * kF8Block;
                if (nw == 8) {
                    if (lane == 0) tma_load_2d(sw, &map_w, &full[s], k, wy, pol_w);
                } else if (lane < nw) {
                    tma_load_2d(sw + lane * 2048, &map_w16, &full[s], k, wy + lane * 16, pol_w);
                }
                if (p.src) {
#pragma unroll
                    for (int i = 0; i < (T + 127) / 128; ++i)
                        if (4 * (lane + 32 * i) < cols)
                            tma_gather4(sq + (lane + 32 * i) * 512, &map_q, &full[s], k, idx[i], pol_q);
                } else if (16 * lane < cols) {
                    tma_load_2d(sq + lane * 2048, &map_q, &full[s], k, t.row0 + 16 * lane, pol_q);
                }
            }
        }
        // every copy that was issued lands before the CTA can exit
        volatile int never = 0;
        for (long long jj = j > C::kStages ? j - C::kStages : 0; jj < j; ++jj)
            mbar_wait_bounded(&full[jj % C::kStages], static_cast<uint32_t>(jj / C::kStages) & 1u, &never);
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs
        long long j = 0;
        bool ok = true;
        Tile t;
        t.e = e0;
        for (long long x = x0; ok && x < x1; x = next(x, t)) {
            tile_at(work, x, end_of(x), t);
            // rows of the stage beyond the tile's hold old bytes: their sums are never looked at
            const uint32_t idesc = tc::idesc_e4m3_f32(kTileRows, (t.n + 15) & ~15);
            for (int kb = 0; kb < p.kb; ++kb, ++j) {
                const int a = static_cast<int>(j % C::kAccs), s = static_cast<int>(j % C::kStages);
                if (j >= C::kAccs)
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&acc_empty[a], static_cast<uint32_t>(j / C::kAccs - 1) & 1u,
                                                                   abort_flag));
                if (ok)
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait_bounded(&full[s], static_cast<uint32_t>(j / C::kStages) & 1u, abort_flag));
                if (!ok) break;
                tc::fence_after();
                if (lane == 0) {
                    const uint32_t sw = smem_u32(smem + s * C::kStage), sq = sw + kStageW;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_e4m3_ss(tmem + a * T, tc::sdesc_kmajor_sw128(sw + 32 * k), tc::sdesc_kmajor_sw128(sq + 32 * k),
                                        idesc, k > 0 ? 1u : 0u);
                    tc::commit(&empty[s]);
                    tc::commit(&acc_full[a]);
                }
                __syncwarp();
            }
        }
        if (!ok) fail();
        tc::fence_before();
        if (lane == 0) tc::commit(drain);
        __syncwarp();
        volatile int never = 0;
        mbar_wait_bounded(drain, 0, &never);
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ scales
        // lane: block lane % 8 of the table, tokens lane / 8, + 4, ...
        long long c = 0;
        bool ok = true;
        Tile t;
        t.e = e0;
        const int i = lane & 7, m1 = lane >> 3;
        for (long long x = x0; ok && x < x1; x = next(x, t)) {
            tile_at(work, x, end_of(x), t);
            const int cols = (t.n + 15) & ~15;
            const float *sw = p.s_w + (static_cast<long long>(t.e) * p.nb + t.w0 / kF8Block) * p.kb;
            const bool two = C::kTables == 2 && t.w0 / kF8Block != (t.w0 + t.rows - 1) / kF8Block;
            for (int k0 = 0; k0 < p.kb; k0 += kAhead, ++c) {
                const int s = static_cast<int>(c & 1);
                if (c >= 2)
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait_bounded(&sc_empty[s], static_cast<uint32_t>((c >> 1) - 1) & 1u, abort_flag));
                if (!ok) {
                    fail();
                    break;
                }
                float *table = scales + s * C::kTables * C::kTable + i * C::kScaleLd;
                const bool in = k0 + i < p.kb;
                const float f0 = in ? __ldg(sw + k0 + i) : 0.0f, f1 = in && two ? __ldg(sw + p.kb + k0 + i) : 0.0f;
#pragma unroll 4
                for (int m = m1; m < cols; m += 4) {
                    float v = 0.0f;
                    if (in && m < t.n) {
                        int r = t.row0 + m;
                        if (p.src) r = __ldg(p.src + r);
                        if (static_cast<unsigned>(r) < static_cast<unsigned>(p.q_rows))
                            v = __ldg(p.s_a + static_cast<long long>(r) * p.kb + k0 + i);
                    }
                    table[m] = __fmul_rn(v, f0);
                    if (two) table[C::kTable + m] = __fmul_rn(v, f1);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[s]);
            }
        }
    } else if (warp >= kEpiWarp0) {
        // ------------------------------------------------ sums and results
        const int qd = warp & 3, half = (warp - kEpiWarp0) >> 2;
        long long j = 0, c = 0;
        bool ok = true;
        Tile t;
        t.e = e0;
        for (long long x = x0; ok && x < x1; x = next(x, t)) {
            tile_at(work, x, end_of(x), t);
            const int cols = (t.n + 15) & ~15;
            const int share = C::kHalves == 2 ? (cols / 2 + 15) & ~15 : cols;
            const int c0 = half * share, nc = min(share, cols - c0);
            const int mine = 32 * qd + lane;
            const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * qd) << 16) + c0;
            const int table = C::kTables == 2 && (t.w0 + mine) / kF8Block != t.w0 / kF8Block && mine < t.rows ? C::kTable : 0;
            f2 acc[C::kCols / 2];
#pragma unroll
            for (int g = 0; g < C::kCols / 2; ++g) acc[g] = 0;
            for (int kb = 0; kb < p.kb; ++kb, ++j) {
                const int a = static_cast<int>(j % C::kAccs), s = static_cast<int>(c & 1);
                if (kb % kAhead == 0)
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sc_full[s], static_cast<uint32_t>(c >> 1) & 1u, abort_flag));
                // warp-uniform: the TMEM loads below are warp-collective
                if (ok)
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait_bounded(&acc_full[a], static_cast<uint32_t>(j / C::kAccs) & 1u, abort_flag));
                if (!ok) {
                    fail();
                    break;
                }
                tc::fence_after();
                const float *sc = scales + s * C::kTables * C::kTable + table + (kb % kAhead) * C::kScaleLd + c0;
#pragma unroll
                for (int g = 0; g < C::kCols / 16; ++g) {
                    if (16 * g < nc) {
                        uint32_t d[16];
                        tc::ld16(lane_addr + a * T + 16 * g, d);
                        float4 f[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[i] = *reinterpret_cast<const float4 *>(sc + 16 * g + 4 * i);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            acc[8 * g + 2 * i] = fma2(pk(__uint_as_float(d[4 * i]), __uint_as_float(d[4 * i + 1])),
                                                      pk(f[i].x, f[i].y), acc[8 * g + 2 * i]);
                            acc[8 * g + 2 * i + 1] = fma2(pk(__uint_as_float(d[4 * i + 2]), __uint_as_float(d[4 * i + 3])),
                                                          pk(f[i].z, f[i].w), acc[8 * g + 2 * i + 1]);
                        }
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[a]);
                if (kb % kAhead == kAhead - 1 || kb == p.kb - 1) {
                    if (lane == 0) mbar_arrive(&sc_empty[s]);
                    ++c;
                }
            }
            if (!ok) break;
            if (mine < t.rows) {
                const int n = min(nc, t.n - c0);
                uint16_t *y = p.y + static_cast<long long>(t.row0 + c0) * p.N + t.w0 + mine;
#pragma unroll
                for (int g = 0; g < C::kCols; ++g) {
                    if (g < n) {
                        const float2 v = upk(acc[g / 2]);
                        float o = (g & 1) ? v.y : v.x;
                        // a row that src sends nowhere
                        if (p.src && static_cast<unsigned>(__ldg(p.src + t.row0 + c0 + g)) >= static_cast<unsigned>(p.q_rows)) o = 0.0f;
                        y[static_cast<long long>(g) * p.N] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
                    }
                }
            }
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

template <int T>
cudaError_t launch(const F8LinearArgs &a, bool pdl, cudaStream_t stream)
{
    using C = Cfg<T>;
    const size_t smem = smem_bytes<T>(a.E);
    // a few hundred ns of host time, and right on every device
    cudaError_t e = cudaFuncSetAttribute(linear_f8_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    Params p;
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
    return cudaLaunchKernelEx(&cfg, linear_f8_kernel<T>, a.map_w, a.map_w16, a.map_q, p);
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
    if (mean <= 128 || busy * tall * ((mean + 255) / 256) < sms) return {128, 128};
    if (experts > 1) return {256, 256};
    // fewest tensor cycles: waves of tiles, each as long as its columns
    int best = 256;
    long long least = 1LL << 62;
    for (int cols = 256; cols >= 144; cols -= 16) {
        const long long tiles = tall * ((rows + cols - 1) / cols), cost = (tiles + sms - 1) / sms * cols;
        if (cost < least) {
            least = cost;
            best = cols;
        }
    }
    return {256, best};
}

cudaError_t launch_linear_f8(const F8LinearArgs &a, bool pdl, cudaStream_t stream)
{
    switch (a.plan.T) {
    case 16: return launch<16>(a, pdl, stream);
    case 32: return launch<32>(a, pdl, stream);
    case 64: return launch<64>(a, pdl, stream);
    case 128: return launch<128>(a, pdl, stream);
    default: return launch<256>(a, pdl, stream);
    }
}

}  // namespace bi
