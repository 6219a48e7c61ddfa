// Penalties, biases and grammar masks on logits, with the argmax.
//
// One CTA per (vocabulary slice, row).  The CTA counts the row's history ids
// that fall into its slice in shared memory (integer adds, so the order of the
// threads does not matter), then streams the slice once.  The slices' largest
// values meet in a 64-bit key per row, (ordered value, ~index), by atomicMax;
// the last CTA of a row writes the argmax and restores the row's words to zero.
//
// Bound: HBM; 2 bytes read, 4 written and 1/8 of mask per logit.  A history is
// read once per slice, from L2 after the first.
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

namespace bi {

namespace {

constexpr int kSlice = 4096;
constexpr int kLogitsThreads = 256;

struct RowKey {
    unsigned long long key;
    int done;
    int pad;
};

// Monotone map of a float that is not NaN to an unsigned integer above 0 (-inf: 0x007FFFFF + 1 > 0).
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__global__ void __launch_bounds__(kLogitsThreads) logits_kernel(LogitsArgs a, int pdl)
{
    __shared__ uint32_t held[kSlice];    // bit 31: in the history; the rest: times generated
    __shared__ uint32_t biased[kSlice];  // 1 + index of the last bias for the element
    __shared__ unsigned long long best;
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const int row = blockIdx.y, v0 = blockIdx.x * kSlice, tid = threadIdx.x;
    const int n = min(kSlice, a.V - v0);
    const bool hist = a.r.ids != nullptr, bias = a.r.bias_ids != nullptr && a.r.n_bias > 0;
    if (tid == 0) best = 0;
    if (hist)
        for (int i = tid; i < kSlice; i += kLogitsThreads) held[i] = 0;
    if (bias)
        for (int i = tid; i < kSlice; i += kLogitsThreads) biased[i] = 0;
    __syncthreads();
    if (hist) {
        const int mid = a.r.mid[row], end = a.r.end[row];
        for (int i = a.r.begin[row] + tid; i < end; i += kLogitsThreads) {
            const int id = a.r.ids[i];
            if (id >= v0 && id - v0 < n) {
                atomicOr(&held[id - v0], 0x80000000u);
                if (i >= mid) atomicAdd(&held[id - v0], 1u);
            }
        }
    }
    if (bias)
        for (int i = tid; i < a.r.n_bias; i += kLogitsThreads) {
            const int id = a.r.bias_ids[static_cast<int64_t>(row) * a.r.n_bias + i];
            if (id >= v0 && id - v0 < n) atomicMax(&biased[id - v0], static_cast<uint32_t>(i + 1));
        }
    __syncthreads();
    const float rep = a.r.repetition ? a.r.repetition[row] : 1.0f;
    const float pres = a.r.presence ? a.r.presence[row] : 0.0f;
    const float freq = a.r.frequency ? a.r.frequency[row] : 0.0f;
    unsigned long long key = 0;
    for (int i = tid; i < n; i += kLogitsThreads) {
        const int v = v0 + i;
        float x = __uint_as_float(static_cast<uint32_t>(a.logits[row * a.ldl + v]) << 16);
        if (hist && held[i]) {
            x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
            const uint32_t c = held[i] & 0x7FFFFFFFu;
            if (c) x = __fsub_rn(__fsub_rn(x, __fmul_rn(freq, static_cast<float>(c))), pres);
        }
        if (bias && biased[i]) x = __fadd_rn(x, a.r.bias[static_cast<int64_t>(row) * a.r.n_bias + biased[i] - 1]);
        if (a.r.mask && !((a.r.mask[row * a.r.ld_mask + (v >> 5)] >> (v & 31)) & 1u)) x = -INFINITY;
        if (a.out) a.out[row * a.ldo + v] = x;
        if (x > -INFINITY) {
            if (x == 0.0f) x = 0.0f;                 // -0 and +0 tie
            const unsigned long long k =
                (static_cast<unsigned long long>(ordered(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(v));
            key = k > key ? k : key;
        }
    }
    if (!a.argmax) return;
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
        key = k > key ? k : key;
    }
    if ((tid & 31) == 0) atomicMax(&best, key);
    __syncthreads();
    if (tid == 0) {
        RowKey *r = static_cast<RowKey *>(a.ws) + row;
        if (best) atomicMax(&r->key, best);
        if (atom_add_acq_rel_gpu(&r->done, 1) == static_cast<int>(gridDim.x) - 1) {
            const unsigned long long k = atomicExch(&r->key, 0ull);
            a.argmax[row] = k ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(k)) : -1;
            r->done = 0;
        }
    }
}

}  // namespace

size_t logits_workspace(int M) { return sizeof(RowKey) * static_cast<size_t>(M); }

cudaError_t launch_logits_process(const LogitsArgs &a, bool pdl, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.V + kSlice - 1) / kSlice), static_cast<unsigned>(a.M));
    cfg.blockDim = dim3(kLogitsThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, logits_kernel, a, pdl ? 1 : 0);
}

}  // namespace bi
