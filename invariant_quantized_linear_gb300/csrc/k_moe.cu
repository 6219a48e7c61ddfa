// Mixture of experts: the router's selection with the order of rows by expert,
// and the weighted sum of the experts' rows.
//
// Selection.  A warp a token; the k largest logits come out one at a time, the
// largest by one reduction over the warp and the lowest id that has it by another.
// Order.  A token takes an expert once, so in a chunk of tokens the row of (token,
// expert) behind the expert's first is the number of earlier tokens that took it: a
// count of bits in a mask of the chunk's tokens, kept for each expert in shared
// memory.  No atomic's order enters a result.
// One CTA does a call of one chunk.  Longer calls write each chunk's counts, and a
// second launch adds the counts of the chunks before its own.
//
// Bound: latency.  8192 x 128 logits are 2 MB, 0.5 us at the copy rate; the two launches
// take 12.7 us: eight picks of two reductions each for two tokens a warp, the counts of
// 128 chunks, the rows.  5 x 64: 3.7 us.  The sum of 8 rows of 4096 for 4096 tokens:
// 57.5 us, 5.8 TB/s (0.86 of the copy rate), HBM.
#include "f8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "row_ops.cuh"

namespace bi {

namespace {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kChunk = 64;                        // tokens of a chunk, where that gives at most kMostChunks
constexpr int kMostChunks = 152;                  // the SMs; a constant, as the counts' workspace is sized without a device
constexpr size_t kPlainSmem = 47 * 1024;          // dynamic shared memory that needs no opt-in, the static share beside it

int chunk_tokens(int M)
{
    const int c = (M + kMostChunks - 1) / kMostChunks;
    return c <= kChunk ? kChunk : (c + 31) / 32 * 32;
}

// Larger floats have larger keys; -0 and 0 the same.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x == 0.0f ? 0.0f : x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

constexpr uint32_t kNone = 0x007FFFFFu;           // key of -inf: allowed by no one

// A token's logits, expert lane + 32 i, as keys: NaN as -inf, +inf as the largest finite value.
template <int EP>
__device__ __forceinline__ void load_keys(const RouteArgs &a, int64_t m, uint32_t (&key)[EP])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < EP; ++i) {
        const int e = lane + 32 * i;
        float x = -INFINITY;
        if (e < a.E)
            x = a.half ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(a.logits)[m * a.ldl + e]) << 16)
                       : static_cast<const float *>(a.logits)[m * a.ldl + e];
        key[i] = x != x ? kNone : key_of(fminf(x, 3.402823466e38f));
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The selection of token m: lane j < k has its j-th expert (-1: none) and weight.
template <int EP>
__device__ __forceinline__ void select(const RouteArgs &a, int64_t m, int &id, float &weight)
{
    const int lane = threadIdx.x & 31;
    uint32_t key[EP];
    load_keys(a, m, key);
    float whole = 0.0f, high = 0.0f;
    if (a.score == BI_ROUTE_SOFTMAX) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < EP; ++i) top = max(top, key[i]);
        top = __reduce_max_sync(0xffffffffu, top);
        high = top == kNone ? 0.0f : value_of(top);
        if (!a.renorm) {
#pragma unroll
            for (int i = 0; i < EP; ++i)
                if (lane + 32 * i < a.E) whole = __fadd_rn(whole, expf(__fsub_rn(value_of(key[i]), high)));
            whole = warp_sum(whole);
        }
    }
    id = -1;
    float x = -INFINITY;
    for (int j = 0; j < a.k; ++j) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < EP; ++i) top = max(top, key[i]);
        top = __reduce_max_sync(0xffffffffu, top);
        if (top <= kNone) break;
        int at = 1 << 30;
#pragma unroll
        for (int i = EP - 1; i >= 0; --i)
            if (key[i] == top) at = lane + 32 * i;
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < EP; ++i)
            if (lane + 32 * i == at) key[i] = 0;
        if (lane == j) {
            id = at;
            x = value_of(top);
        }
    }
    weight = 0.0f;
    if (a.score == BI_ROUTE_SOFTMAX) {
        if (id >= 0) weight = expf(__fsub_rn(x, high));
    } else {
        // exp(x - low) / (1 + exp(x)) for x <= 0: with renorm all are taken exp(low) apart, low the largest x below 0, so that
        // their quotients stay where the sigmoids themselves leave fp32
        const float low = a.renorm ? fminf(__shfl_sync(0xffffffffu, x, 0), 0.0f) : 0.0f;
        if (id >= 0)
            weight = x > 0.0f ? __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x)))
                              : __fdiv_rn(expf(__fsub_rn(x, low)), __fadd_rn(1.0f, expf(x)));
        whole = 1.0f;
    }
    if (a.renorm) whole = warp_sum(weight);
    weight = __fmul_rn(__fdiv_rn(weight, whole > 0.0f ? whole : 1.0f), a.scale);
}

// Exclusive prefix of v over the CTA's threads, and the sum of all.
__device__ __forceinline__ int block_prefix(int v, int *sums, int &all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int u = lane < kRouteWarps ? sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, u, o);
            if (lane >= o) u += w;
        }
        sums[lane] = u;
    }
    __syncthreads();
    all = sums[kRouteWarps - 1];
    return s - v + (warp > 0 ? sums[warp - 1] : 0);
}

// Rows of the chunk's slots, from the masks and each expert's first row in this chunk.
__device__ __forceinline__ void place(const RouteArgs &a, int first, int tokens, int words, const uint32_t *mask, const int *base)
{
    for (int i = threadIdx.x; i < tokens * a.k; i += kRouteThreads) {
        const int t = i / a.k;
        const int64_t slot = static_cast<int64_t>(first) * a.k + i;
        const int e = a.ids[slot];
        int r = -1;
        if (e >= 0) {
            const uint32_t *w = mask + e * words;
            r = base[e] + __popc(w[t >> 5] & ((1u << (t & 31)) - 1));
            for (int j = 0; j < t >> 5; ++j) r += __popc(w[j]);
            a.src[r] = first + t;
        }
        a.pos[slot] = r;
    }
}

// The chunk's masks from its ids.
__device__ __forceinline__ void mark(const RouteArgs &a, int first, int tokens, int words, uint32_t *mask)
{
    for (int i = threadIdx.x; i < tokens * a.k; i += kRouteThreads) {
        const int t = i / a.k, e = a.ids[static_cast<int64_t>(first) * a.k + i];
        if (e >= 0) atomicOr(mask + e * words + (t >> 5), 1u << (t & 31));
    }
}

// Selection; then, of a call of one chunk, everything, else the chunk's counts.
template <int EP>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteArgs a, int chunk, int pdl)
{
    extern __shared__ uint32_t mask[];                   // [E][words], then int [E] first rows
    __shared__ int sums[32];
    const int words = chunk / 32;
    int *base = reinterpret_cast<int *>(mask + a.E * words);
    for (int i = threadIdx.x; i < a.E * words; i += kRouteThreads) mask[i] = 0;
    if (gridDim.x > 1) pdl_launch_dependents();          // the second launch waits for this one's end before it reads
    if (pdl) pdl_wait();
    __syncthreads();
    const int first = blockIdx.x * chunk, tokens = min(chunk, a.M - first), lane = threadIdx.x & 31;
    for (int t = threadIdx.x >> 5; t < tokens; t += kRouteWarps) {
        int id;
        float w;
        const int64_t m = first + t;
        select<EP>(a, m, id, w);
        if (lane < a.k) {
            a.ids[m * a.k + lane] = id;
            a.weights[m * a.k + lane] = w;
            if (id >= 0) atomicOr(mask + id * words + (t >> 5), 1u << (t & 31));
        }
    }
    __syncthreads();
    int n = 0;
    const int e = threadIdx.x;
    if (e < a.E)
        for (int j = 0; j < words; ++j) n += __popc(mask[e * words + j]);
    if (gridDim.x > 1) {
        if (e < a.E) static_cast<int *>(a.ws)[static_cast<int64_t>(blockIdx.x) * a.E + e] = n;
        return;
    }
    int all;
    const int at = block_prefix(n, sums, all);
    if (e < a.E) {
        base[e] = at;
        a.offsets[e] = at;
    }
    if (e == 0) a.offsets[a.E] = all;
    __syncthreads();
    place(a, first, tokens, words, mask, base);
    for (int r = all + threadIdx.x; r < a.M * a.k; r += kRouteThreads) a.src[r] = -1;
    pdl_launch_dependents();
}

__global__ void __launch_bounds__(kRouteThreads) route_rows_kernel(RouteArgs a, int chunk)
{
    extern __shared__ uint32_t mask[];
    __shared__ int sums[32];
    const int words = chunk / 32;
    int *base = reinterpret_cast<int *>(mask + a.E * words), *before = base + a.E, *whole = before + a.E;
    for (int i = threadIdx.x; i < a.E * words; i += kRouteThreads) mask[i] = 0;
    for (int i = threadIdx.x; i < 2 * a.E; i += kRouteThreads) before[i] = 0;
    pdl_wait();
    __syncthreads();
    const int first = blockIdx.x * chunk, tokens = min(chunk, a.M - first);
    mark(a, first, tokens, words, mask);
    // counts of the chunks before this one and of all: threads share an expert's column
    const int share = kRouteThreads / a.E > 0 ? kRouteThreads / a.E : 1, part = threadIdx.x / a.E, e = threadIdx.x - part * a.E;
    if (part < share) {
        int mine = 0, all = 0;
        const int *counts = static_cast<const int *>(a.ws) + e;
#pragma unroll 8
        for (int c = part; c < static_cast<int>(gridDim.x); c += share) {
            const int n = __ldcg(counts + static_cast<int64_t>(c) * a.E);
            all += n;
            if (c < static_cast<int>(blockIdx.x)) mine += n;
        }
        atomicAdd(before + e, mine);                     // whole numbers: any order
        atomicAdd(whole + e, all);
    }
    __syncthreads();
    int total;
    const int at = block_prefix(threadIdx.x < a.E ? whole[threadIdx.x] : 0, sums, total);
    if (threadIdx.x < a.E) {
        base[threadIdx.x] = at + before[threadIdx.x];
        if (blockIdx.x == 0) a.offsets[threadIdx.x] = at;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = total;
    __syncthreads();
    place(a, first, tokens, words, mask, base);
    for (int64_t r = total + static_cast<int64_t>(blockIdx.x) * kRouteThreads + threadIdx.x; r < static_cast<int64_t>(a.M) * a.k;
         r += static_cast<int64_t>(gridDim.x) * kRouteThreads)
        a.src[r] = -1;
    pdl_launch_dependents();
}

// Dynamic shared memory of a call: the masks of a chunk's tokens and three numbers an expert.
size_t route_smem(int chunk, int E) { return static_cast<size_t>(E) * (chunk / 32) * 4 + 3 * static_cast<size_t>(E) * 4; }

template <int EP>
cudaError_t route(const RouteArgs &a, bool pdl, cudaStream_t stream)
{
    const int chunk = chunk_tokens(a.M), chunks = (a.M + chunk - 1) / chunk;
    const size_t smem = route_smem(chunk, a.E);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(chunks));
    cfg.blockDim = dim3(kRouteThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    cudaError_t e = cudaSuccess;
    // Without an opt-in a kernel has 48 KB, its static share among them.  The opt-in is the kernel's, not the call's, so
    // it is always the largest call's: a smaller one would take it from a call of another thread.
    if (smem > kPlainSmem) {
        const int most = static_cast<int>(route_smem(chunk_tokens(kMaxTokens), kMaxExperts));
        e = cudaFuncSetAttribute(route_kernel<EP>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(route_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    e = cudaLaunchKernelEx(&cfg, route_kernel<EP>, a, chunk, pdl ? 1 : 0);
    if (e != cudaSuccess || chunks == 1) return e;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_rows_kernel, a, chunk);
}

// ------------------------------------------------------------ weighted sum

constexpr int kSumThreads = 256;

// Eight columns a thread (VEC), or one.  Rows of a token are added in the order of its experts, each by one fma.
template <bool VEC>
__global__ void __launch_bounds__(kSumThreads) combine_kernel(CombineArgs a, int per_row, long long work, int pdl)
{
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    constexpr int W = VEC ? 8 : 1;
    const long long at = static_cast<long long>(blockIdx.x) * kSumThreads + threadIdx.x;
    if (at >= work) return;
    const long long m = at / per_row;
    const int n = static_cast<int>(at - m * per_row) * W;
    float sum[W];
#pragma unroll
    for (int i = 0; i < W; ++i) sum[i] = 0.0f;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
        uint4 x[8];
        float w[8];
        bool there[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            there[j] = false;
            w[j] = 0.0f;
            if (j0 + j < a.k) {
                const int r = __ldg(a.pos + m * a.k + j0 + j);
                there[j] = static_cast<unsigned>(r) < static_cast<unsigned>(a.R);
                if (there[j]) {
                    w[j] = __ldg(a.weights + m * a.k + j0 + j);
                    const uint16_t *p = a.rows + static_cast<long long>(r) * a.N + n;
                    if (VEC) x[j] = __ldcs(reinterpret_cast<const uint4 *>(p));
                    else x[j].x = __ldcs(p);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (there[j]) {
                const uint32_t v[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                for (int i = 0; i < W; ++i) sum[i] = __fmaf_rn(w[j], (i & 1) ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]), sum[i]);
            }
    }
    const long long out = m * a.N + n;
    if (VEC) {
        if (a.base) {
            const uint4 b = __ldcs(reinterpret_cast<const uint4 *>(a.base + out));
            const uint32_t v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < W; ++i) sum[i] = __fadd_rn((i & 1) ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]), sum[i]);
        }
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(sum[(2 * i) % W], sum[(2 * i + 1) % W]);
        *reinterpret_cast<uint4 *>(a.y + out) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
        if (a.base) sum[0] = __fadd_rn(bf16_lo(a.base[out]), sum[0]);
        a.y[out] = static_cast<uint16_t>(bf16_rne_bits(sum[0]));
    }
}

}  // namespace

size_t moe_route_workspace(int M, int E)
{
    const int c = chunk_tokens(M), chunks = (M + c - 1) / c;
    return (static_cast<size_t>(chunks) * E * 4 + 255) / 256 * 256;
}

cudaError_t launch_moe_route(const RouteArgs &a, bool pdl, cudaStream_t stream)
{
    if (a.E <= 32) return route<1>(a, pdl, stream);
    if (a.E <= 64) return route<2>(a, pdl, stream);
    if (a.E <= 128) return route<4>(a, pdl, stream);
    if (a.E <= 256) return route<8>(a, pdl, stream);
    return route<32>(a, pdl, stream);
}

cudaError_t launch_moe_combine(const CombineArgs &a, bool pdl, cudaStream_t stream)
{
    auto aligned16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    const bool vec = a.N % 8 == 0 && aligned16(a.rows) && aligned16(a.y) && (!a.base || aligned16(a.base));
    const int per_row = vec ? a.N / 8 : a.N;
    const long long work = static_cast<long long>(a.M) * per_row;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((work + kSumThreads - 1) / kSumThreads));
    cfg.blockDim = dim3(kSumThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return vec ? cudaLaunchKernelEx(&cfg, combine_kernel<true>, a, per_row, work, pdl ? 1 : 0)
               : cudaLaunchKernelEx(&cfg, combine_kernel<false>, a, per_row, work, pdl ? 1 : 0);
}

}  // namespace bi
