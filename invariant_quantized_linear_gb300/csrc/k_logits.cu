// Penalties, biases and grammar masks on logits, with the argmax.
//
// One CTA per (vocabulary slice, row).  The CTA counts the row's history ids
// that fall into its slice in shared memory (integer adds, so the order of the
// threads does not matter) and lists the elements that it meets; their logits
// are on their way meanwhile.  The slice is then streamed once, four elements a
// thread, leaving the listed ones out of the maximum, and these are done
// afterwards, one a thread: a text's few hundred tokens touch nearly every
// group of 128 elements, and penalties in the stream would cost it twice its
// time.  The slices' largest values meet in a 64-bit key per row, (ordered
// value, ~index), by atomicMax; the last CTA of a row writes the argmax and
// restores the row's words to zero.
//
// Bound: HBM; 2 bytes read, 4 written and 1/8 of mask per logit.  A history is
// read once per slice, from L2 after the first.  Rows of an odd vocabulary start
// anywhere: slices are cut so that a thread's four results are one aligned
// store, and its four logits come out of two aligned loads.
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

namespace bi {

namespace {

constexpr int kLogitsThreads = 256;

struct RowKey {
    unsigned long long key;
    int done;
    int pad;
};

// Monotone map of a float that is not NaN to an unsigned integer (above 0 for all but the lowest).
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// A row's candidate: larger for a larger value, then for a lower index; 0 for -inf and NaN.
__device__ __forceinline__ unsigned long long key_of(float x, int v)
{
    // + 0: -0 and +0 tie
    return x > -INFINITY ? (static_cast<unsigned long long>(ordered(x + 0.0f)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(v))
                         : 0ull;
}

// x[i] = max(x[i], v) for a 16-bit element, by exchanges of the word that holds it.
__device__ __forceinline__ void max_u16(uint16_t *x, int i, uint32_t v)
{
    uint32_t *word = reinterpret_cast<uint32_t *>(x) + i / 2;
    const int sh = 16 * (i & 1);
    uint32_t old = *word;
    while (((old >> sh) & 0xFFFFu) < v) {                  // each failed exchange means that another lane's went through
        const uint32_t seen = atomicCAS(word, old, (old & ~(0xFFFFu << sh)) | (v << sh));
        if (seen == old) break;
        old = seen;
    }
}

// N elements a thread, four at a time; the slice is 256 N elements.
template <int N>
__global__ void __launch_bounds__(kLogitsThreads) logits_kernel(LogitsArgs a, int pdl)
{
    constexpr int kSlice = kLogitsThreads * N, kSteps = N / 4;
    extern __shared__ __align__(16) uint32_t smem[];
    uint32_t *held = smem;               // bit 31: in the history, bit 30: has a bias; the rest: times generated
    uint16_t *listed = reinterpret_cast<uint16_t *>(smem + kSlice);   // the elements with any of these
    uint16_t *biased = listed + kSlice;  // 1 + index of the last bias for the element
    __shared__ unsigned long long best;
    __shared__ int n_listed;
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const int row = blockIdx.y, tid = threadIdx.x;
    const uint16_t *x = a.logits + row * a.ldl;
    float *out = a.out ? a.out + row * a.ldo : nullptr;
    // element v is number v + shift of the row's slices: numbers that are multiples of 4 are aligned for the store, or,
    // without one, for the load
    const int shift = out ? static_cast<int>((reinterpret_cast<uintptr_t>(out) >> 2) & 3u)
                          : static_cast<int>((reinterpret_cast<uintptr_t>(x) >> 1) & 3u);
    const int v0 = static_cast<int>(blockIdx.x) * kSlice - shift;
    // the four logits begin `off` elements into an aligned group of four
    const int off = static_cast<int>(((reinterpret_cast<uintptr_t>(x) >> 1) + 4 - shift) & 3u);
    uint2 lo[kSteps], hi[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int v = v0 + 4 * (tid + i * kLogitsThreads) - off;
        const bool inner = v >= 0 && v + (off ? 8 : 4) <= a.V;
        lo[i] = hi[i] = make_uint2(0u, 0u);
        if (inner) {
            lo[i] = __ldcs(reinterpret_cast<const uint2 *>(x + v));
            if (off) hi[i] = __ldcs(reinterpret_cast<const uint2 *>(x + v + 4));
        }
    }
    // and the mask's words; a row's first group of four may begin before it
    const uint32_t *mask = a.r.mask ? a.r.mask + row * a.r.ld_mask : nullptr;
    uint32_t m_lo[kSteps], m_hi[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int v = v0 + 4 * (tid + i * kLogitsThreads), m = max(v, 0);
        m_lo[i] = m_hi[i] = ~0u;
        if (mask && m < a.V) {
            m_lo[i] = __ldg(mask + (m >> 5));
            m_hi[i] = (m & 31) > 28 ? __ldg(mask + (min(m + 3, a.V - 1) >> 5)) : 0u;
        }
    }
    const bool hist = a.r.ids != nullptr, bias = a.r.bias_ids != nullptr, some = hist || bias;
    const int end = hist ? a.r.end[row] : 0, mid = hist ? a.r.mid[row] : 0, begin = hist ? a.r.begin[row] : 0;
    const float rep = a.r.repetition ? a.r.repetition[row] : 1.0f;
    const float pres = a.r.presence ? a.r.presence[row] : 0.0f;
    const float freq = a.r.frequency ? a.r.frequency[row] : 0.0f;
    if (tid == 0) {
        best = 0;
        n_listed = 0;
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        if (some) reinterpret_cast<uint4 *>(held)[tid + i * kLogitsThreads] = make_uint4(0u, 0u, 0u, 0u);
        if (bias) reinterpret_cast<uint2 *>(biased)[tid + i * kLogitsThreads] = make_uint2(0u, 0u);
    }
    __syncthreads();
    // ids of the slice: v0 <= id < v0 + kSlice, and 0 <= id < V
    const int first = max(v0, 0), past = min(v0 + kSlice, a.V);
    if (hist) {
#pragma unroll 4
        for (int i = begin + tid; i < end; i += kLogitsThreads) {
            const int id = __ldg(a.r.ids + i);
            if (id >= first && id < past) {
                if (atomicOr(&held[id - v0], 0x80000000u) == 0u) listed[atomicAdd(&n_listed, 1)] = static_cast<uint16_t>(id - v0);
                if (i >= mid) atomicAdd(&held[id - v0], 1u);
            }
        }
    }
    if (bias) {
        __syncthreads();                                   // an element is listed by whoever finds its word zero
        for (int i = tid; i < a.r.n_bias; i += kLogitsThreads) {
            const int id = __ldg(a.r.bias_ids + static_cast<int64_t>(row) * a.r.n_bias + i);
            if (id >= first && id < past) {
                if (atomicOr(&held[id - v0], 0x40000000u) == 0u) listed[atomicAdd(&n_listed, 1)] = static_cast<uint16_t>(id - v0);
                max_u16(biased, id - v0, static_cast<uint32_t>(i + 1));
            }
        }
    }
    __syncthreads();

    float top = -INFINITY;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int k = tid + i * kLogitsThreads, v = v0 + 4 * k;
        if (v + 4 <= 0 || v >= a.V) continue;
        float y[4];
        if (v - off >= 0 && v - off + (off ? 8 : 4) <= a.V) {
            // elements off .. off + 3 of the eight
            const uint32_t w[4] = {lo[i].x, lo[i].y, hi[i].x, hi[i].y};
            const uint32_t p = off & 2 ? w[1] : w[0], q = off & 2 ? w[2] : w[1], r = off & 2 ? w[3] : w[2];
            const uint32_t z0 = off & 1 ? __byte_perm(p, q, 0x5432) : p, z1 = off & 1 ? __byte_perm(q, r, 0x5432) : q;
            y[0] = bf16_lo(z0), y[1] = bf16_hi(z0), y[2] = bf16_lo(z1), y[3] = bf16_hi(z1);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = v + e >= 0 && v + e < a.V ? __uint_as_float(static_cast<uint32_t>(x[v + e]) << 16) : -INFINITY;
        }
        if (mask) {
            const int m = max(v, 0);
            const uint32_t bits = __funnelshift_r(m_lo[i], m_hi[i], m & 31) << (m - v);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = (bits >> e) & 1u ? y[e] : -INFINITY;
        }
        if (out) {
            if (v >= 0 && v + 4 <= a.V) {
                __stcs(reinterpret_cast<float4 *>(out + v), make_float4(y[0], y[1], y[2], y[3]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (v + e >= 0 && v + e < a.V) out[v + e] = y[e];
            }
        }
        if (some) {
            const uint4 c = reinterpret_cast<const uint4 *>(held)[k];
            if (c.x | c.y | c.z | c.w) {
                y[0] = c.x ? -INFINITY : y[0];
                y[1] = c.y ? -INFINITY : y[1];
                y[2] = c.z ? -INFINITY : y[2];
                y[3] = c.w ? -INFINITY : y[3];
            }
        }
        const float most = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
        if (most > top) {                                  // rare after a few; the lowest element of the largest value
            top = most;
            at = v + (y[0] == most ? 0 : y[1] == most ? 1 : y[2] == most ? 2 : 3);
        }
    }
    unsigned long long key = key_of(top, at);
    if (some) {
        __syncthreads();                                   // the stream's stores come before these
        for (int i = tid; i < n_listed; i += kLogitsThreads) {
            const int k = listed[i], v = v0 + k;
            const uint32_t c = held[k], n = c & 0x3FFFFFFFu;
            float z = __uint_as_float(static_cast<uint32_t>(x[v]) << 16);
            if (c & 0x80000000u) z = z > 0.0f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
            if (n) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, static_cast<float>(n))), pres);
            if (c & 0x40000000u) z = __fadd_rn(z, __ldg(a.r.bias + static_cast<int64_t>(row) * a.r.n_bias + biased[k] - 1));
            if (mask && !((__ldg(mask + (v >> 5)) >> (v & 31)) & 1u)) z = -INFINITY;
            if (out) out[v] = z;
            const unsigned long long kz = key_of(z, v);
            key = kz > key ? kz : key;
        }
    }
    if (!a.argmax) return;
#pragma unroll
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

template <int N>
cudaError_t launch(const LogitsArgs &a, bool pdl, cudaStream_t stream)
{
    constexpr int slice = kLogitsThreads * N;
    // room for the history's counts and the biases, as far as there are such
    const int bytes = a.r.bias_ids ? 8 * slice : a.r.ids ? 6 * slice : 0;
    if (bytes + 1024 > 48 * 1024) {                        // with the kernel's own, more than any launch may have
        const cudaError_t e = cudaFuncSetAttribute(logits_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * slice);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    // up to 3 elements of shift
    cfg.gridDim = dim3(static_cast<unsigned>((a.V + 3 + slice - 1) / slice), static_cast<unsigned>(a.M));
    cfg.blockDim = dim3(kLogitsThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, logits_kernel<N>, a, pdl ? 1 : 0);
}

}  // namespace

size_t logits_workspace(int M) { return sizeof(RowKey) * static_cast<size_t>(M); }

cudaError_t launch_logits_process(const LogitsArgs &a, int sms, bool pdl, cudaStream_t stream)
{
    // short slices while the long ones would leave SMs idle: each slice reads the row's history again
    return static_cast<int64_t>(a.M) * ((a.V + 8191) / 8192) < 2 * sms ? launch<8>(a, pdl, stream) : launch<32>(a, pdl, stream);
}

}  // namespace bi
