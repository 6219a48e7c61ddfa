// Penalties, biases and grammar masks on logits, with the argmax.
//
// One CTA per (vocabulary slice, row).  It marks the row's history ids and biases
// that fall into the slice in a bit map, ranks the marks, and counts the ids at
// their ranks (integer adds, so the order of the threads does not matter), all
// in shared memory; the slice's logits are on their way to L2 meanwhile.  The
// slice is then streamed, four elements a thread; marked elements go with the
// forbidden ones there, so that they do not enter the maximum, and are done
// afterwards, one a thread, their logits asked for before the stream: a text's
// few hundred tokens touch nearly every group of 128 elements, and penalties in
// the stream would cost it twice its time.  The largest values meet in a 64-bit
// key per row, (ordered value, ~index), by atomicMax; the last CTA of a row
// writes the argmax and restores the row's words to zero.
//
// Bound: HBM; 2 bytes read, 4 written and 1/8 of mask per logit: 400 rows of
// 128259 take 48 us without rules, 6.4 TB/s.  A history is read once per slice,
// from L2 after the first, and its four barriers and two looks are what the
// stream of other CTAs hides in part only: 84 us with histories of 3000, biases
// and masks (3.7 TB/s), 70 when only the argmax is asked for (2 bytes a logit: 16 us
// of copies).  5 rows of 151936: 7.1 us.  Measured and not kept: the
// slices of a row as a cluster that sorts the history once (104 us), ids taken
// in turn by a warp's lanes (84, small calls slower), CTAs of 128 or 512 threads
// (89, 88), slices as long as balanced waves allow (85).  Rows of an odd vocabulary start
// anywhere: slices are cut so that a thread's four results are one aligned
// store, and its four logits come out of two aligned loads.
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

#include <type_traits>

namespace bi {

namespace {

constexpr int kLogitsThreads = 256;
constexpr int kLogitsCtas = 4;           // CTAs a SM that the registers are to allow
constexpr int kIds = 3;                  // groups of four history ids of a thread in flight

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

// A row as the kernel sees it.  Element v is number v + shift of the row's
// slices: numbers that are multiples of 4 are aligned for the store, or, without
// one, for the load.
struct Row {
    const uint16_t *x;
    float *out;
    const uint32_t *mask;
    int V, off;                          // the four logits of a group begin `off` elements into an aligned four

    __device__ __forceinline__ bool inner(int v) const { return v >= off && v - off + (off ? 8 : 4) <= V; }
};

// Four logits from v on, EDGE: as far as there are such (-inf else).
template <bool EDGE>
__device__ __forceinline__ void four(const Row &r, int v, const uint2 &lo, const uint2 &hi, float (&y)[4])
{
    if (EDGE && !r.inner(v)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = v + e >= 0 && v + e < r.V ? __uint_as_float(static_cast<uint32_t>(r.x[v + e]) << 16) : -INFINITY;
        return;
    }
    const bool up = r.off & 2;
    const uint32_t p = up ? lo.y : lo.x, q = up ? hi.x : lo.y, s = up ? hi.y : hi.x;
    const int sh = 16 * (r.off & 1);
    const uint32_t z0 = __funnelshift_r(p, q, sh), z1 = __funnelshift_r(q, s, sh);
    y[0] = bf16_lo(z0), y[1] = bf16_hi(z0), y[2] = bf16_lo(z1), y[3] = bf16_hi(z1);
}

// Bit e of the mask words that hold elements v .. v + 3 (a row's first group may begin before it).
__device__ __forceinline__ uint32_t mask_bits(uint32_t lo, uint32_t hi, int v)
{
    const int m = max(v, 0);
    return __funnelshift_r(lo, hi, m & 31) << (m - v);
}

constexpr int kMarks = 4096;             // marked elements of a slice done at once
constexpr int kMet = 2048;               // history ids of a slice that are kept between the two passes over them

// Shared memory for a slice of `slice` elements.
struct LogitsPlan {
    int rank, held, listed, biased, met, bytes;
    __host__ __device__ constexpr LogitsPlan(int slice)
        : rank(slice / 8), held(rank + slice / 16), listed(held + 4 * kMarks), biased(listed + 2 * kMarks),
          met(biased + 2 * kMarks), bytes(met + 2 * kMet)
    {
    }
};

// STEPS groups of four elements a thread, BATCH of them in flight; the slice is 1024 STEPS elements.
template <int STEPS, int BATCH>
__global__ void __launch_bounds__(kLogitsThreads, kLogitsCtas) logits_kernel(LogitsArgs a, int pdl)
{
    constexpr int kStep = 4 * kLogitsThreads, kSlice = kStep * STEPS, kWords = kSlice / 32;
    constexpr LogitsPlan P(kSlice);
    extern __shared__ __align__(16) unsigned char smem[];
    uint32_t *marked = reinterpret_cast<uint32_t *>(smem);            // a bit an element
    uint16_t *rank = reinterpret_cast<uint16_t *>(smem + P.rank);     // marks before each word
    // of the marked elements, by rank: times generated, bit 31: in the prompt, bit 30: has a bias; which; its last bias + 1
    uint32_t *held = reinterpret_cast<uint32_t *>(smem + P.held);
    uint16_t *listed = reinterpret_cast<uint16_t *>(smem + P.listed), *biased = reinterpret_cast<uint16_t *>(smem + P.biased);
    // the history's ids in the slice, in any order: element, bit 15: generated; as many as there is room for
    uint16_t *met = reinterpret_cast<uint16_t *>(smem + P.met);
    __shared__ int n_met;
    __shared__ unsigned long long best;
    __shared__ int warp_marks[kLogitsThreads / 32];
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const bool hist = a.r.ids != nullptr, bias = a.r.bias_ids != nullptr, some = hist || bias;
    const int end = hist ? a.r.end[row] : 0, mid = hist ? a.r.mid[row] : 0, begin = hist ? a.r.begin[row] : 0;
    Row r;
    r.x = a.logits + row * a.ldl;
    r.out = a.out ? a.out + row * a.ldo : nullptr;
    r.mask = a.r.mask ? a.r.mask + row * a.r.ld_mask : nullptr;
    r.V = a.V;
    const int shift = r.out ? static_cast<int>((reinterpret_cast<uintptr_t>(r.out) >> 2) & 3u)
                            : static_cast<int>((reinterpret_cast<uintptr_t>(r.x) >> 1) & 3u);
    r.off = static_cast<int>(((reinterpret_cast<uintptr_t>(r.x) >> 1) + 4 - shift) & 3u);
    const int v0 = static_cast<int>(blockIdx.x) * kSlice - shift;
    // whether some group of a batch is not whole: at a row's ends
    auto edge = [&](int step) {
        const int v = v0 + step * kStep;
        return v < 4 || v + BATCH * kStep + 8 > a.V;
    };
    // a batch of the slice's logits and mask words
    const int own0 = v0 + 4 * tid;                         // the thread's groups begin here and every kStep elements
    const uint16_t *const px = r.x + (own0 - r.off);
    const uint32_t *const pm = r.mask ? r.mask + (own0 >> 5) : nullptr;
    const int next = ((own0 + 3) >> 5) - (own0 >> 5);      // a group may lie in two words
    uint2 lo[BATCH], hi[BATCH];
    uint32_t m_lo[BATCH], m_hi[BATCH];
    auto load = [&](int step) {
        const bool whole = !edge(step);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int at = (step + i) * kStep, v = own0 + at;
            hi[i] = make_uint2(0u, 0u);
            m_lo[i] = m_hi[i] = ~0u;
            if (whole) {
                lo[i] = __ldcs(reinterpret_cast<const uint2 *>(px + at));
                if (r.off) hi[i] = __ldcs(reinterpret_cast<const uint2 *>(px + at + 4));
                if (pm) {
                    m_lo[i] = __ldg(pm + at / 32);
                    if (v0 & 3) m_hi[i] = __ldg(pm + at / 32 + next);
                }
            } else {
                lo[i] = make_uint2(0u, 0u);
                if (r.inner(v)) {
                    lo[i] = __ldcs(reinterpret_cast<const uint2 *>(px + at));
                    if (r.off) hi[i] = __ldcs(reinterpret_cast<const uint2 *>(px + at + 4));
                }
                if (pm && v < a.V) {
                    m_lo[i] = __ldg(r.mask + (max(v, 0) >> 5));
                    m_hi[i] = __ldg(r.mask + (min(max(v, 0) + 3, a.V - 1) >> 5));
                }
            }
        }
    };
    load(0);
    if (STEPS > BATCH) {                                   // the rest into L2 while the history is looked at: a line a thread
        const int v = v0 + tid * (kSlice / kLogitsThreads);
        if (v >= 0 && v < a.V) asm volatile("prefetch.global.L2 [%0];" ::"l"(r.x + v));
    }
    const float rep = a.r.repetition ? a.r.repetition[row] : 1.0f;
    const float pres = a.r.presence ? a.r.presence[row] : 0.0f;
    const float freq = a.r.frequency ? a.r.frequency[row] : 0.0f;
    if (tid == 0) best = 0, n_met = 0;

    // the slice's ids: v0 <= id < v0 + kSlice, and 0 <= id < V
    const int first = max(v0, 0), past = min(v0 + kSlice, a.V);
    const unsigned n_ids = past > first ? past - first : 0;
    // f(i, element of the slice) for the history's: aligned fours from vb to ve, at most three ids before and after them
    const int head = hist ? static_cast<int>((0u - static_cast<unsigned>(reinterpret_cast<uintptr_t>(a.r.ids + begin) >> 2)) & 3u) : 0;
    const int vb = min(begin + head, max(begin, end)), ve = vb + (max(end - vb, 0) & ~3);
    auto load_ids = [&](int i0, int4 (&id)[kIds]) {
#pragma unroll
        for (int j = 0; j < kIds; ++j) {
            const int i = i0 + 4 * j * kLogitsThreads;
            id[j] = i < ve ? __ldg(reinterpret_cast<const int4 *>(a.r.ids + i)) : make_int4(-1, -1, -1, -1);
        }
    };
    int4 ids[kIds];                                        // the first, on their way while the marks are cleared
    if (hist) load_ids(vb + 4 * tid, ids);
    const int bias0 = bias && tid < a.r.n_bias ? __ldg(a.r.bias_ids + static_cast<int64_t>(row) * a.r.n_bias + tid) : -1;
    auto history = [&](auto f, bool loaded) {
        auto one = [&](int i, int id) {
            if (static_cast<unsigned>(id) - first < n_ids) f(i, id - v0);
        };
        if (tid < vb - begin) one(begin + tid, __ldg(a.r.ids + begin + tid));
        if (tid < end - ve) one(ve + tid, __ldg(a.r.ids + ve + tid));
        for (int i0 = vb + 4 * tid; i0 < ve; i0 += 4 * kIds * kLogitsThreads) {
            if (!loaded) load_ids(i0, ids);                // loads first: a mark in between would hold up the next
            loaded = false;
#pragma unroll
            for (int j = 0; j < kIds; ++j) {
                const int i = i0 + 4 * j * kLogitsThreads;
                one(i, ids[j].x);
                one(i + 1, ids[j].y);
                one(i + 2, ids[j].z);
                one(i + 3, ids[j].w);
            }
        }
    };
    auto biases = [&](auto f) {
        for (int i = tid; i < a.r.n_bias; i += kLogitsThreads) {
            const int id = i == tid ? bias0 : __ldg(a.r.bias_ids + static_cast<int64_t>(row) * a.r.n_bias + i);
            if (id >= first && id < past) f(i, id - v0);
        }
    };
    int n = 0;                                             // marked elements
    if (some) {
        for (int i = tid; i < kWords / 4; i += kLogitsThreads)
            reinterpret_cast<uint4 *>(marked)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        auto mark = [&](int, int k) { atomicOr(&marked[k >> 5], 1u << (k & 31)); };
        if (hist)
            history([&](int i, int k) {
                atomicOr(&marked[k >> 5], 1u << (k & 31));
                const int at = atomicAdd(&n_met, 1);
                if (at < kMet) met[at] = static_cast<uint16_t>(k | (i >= mid ? 0x8000 : 0));
            }, true);
        if (bias) biases(mark);
        __syncthreads();
        // ranks: a run of words a thread, over the warp, over the warps
        constexpr int kRun = (kWords + kLogitsThreads - 1) / kLogitsThreads;
        int c = 0;
#pragma unroll
        for (int j = 0; j < kRun; ++j)
            if (tid * kRun + j < kWords) c += __popc(marked[tid * kRun + j]);
        int sum = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        if (lane == 31) warp_marks[tid >> 5] = sum;
        __syncthreads();
        int at = sum - c;
#pragma unroll
        for (int w = 0; w < kLogitsThreads / 32; ++w) {
            if (w < tid >> 5) at += warp_marks[w];
            n += warp_marks[w];
        }
#pragma unroll
        for (int j = 0; j < kRun; ++j)
            if (tid * kRun + j < kWords) {
                rank[tid * kRun + j] = static_cast<uint16_t>(at);
                at += __popc(marked[tid * kRun + j]);
            }
    }
    // counts, list and biases of the marked elements of ranks from .. from + kMarks - 1
    auto collect = [&](int from) {
        const int here = min(n - from, kMarks);
        for (int i = tid; i < here; i += kLogitsThreads) {
            held[i] = 0u;
            biased[i] = 0;
        }
        __syncthreads();
        auto slot = [&](int k) {
            const uint32_t w = marked[k >> 5];
            return rank[k >> 5] + __popc(w & ((1u << (k & 31)) - 1u)) - from;
        };
        if (hist) {
            auto count = [&](bool generated, int k) {
                const int s = slot(k);
                if (s < 0 || s >= kMarks) return;
                if (generated) atomicAdd(&held[s], 1u);
                else atomicOr(&held[s], 0x80000000u);
                listed[s] = static_cast<uint16_t>(k);
            };
            const int m = n_met;
            if (m <= kMet) {
                for (int i = tid; i < m; i += kLogitsThreads) count(met[i] & 0x8000u, met[i] & 0x7FFF);
            } else {
                history([&](int i, int k) { count(i >= mid, k); }, false);
            }
        }
        if (bias)
            biases([&](int i, int k) {
                const int s = slot(k);
                if (s < 0 || s >= kMarks) return;
                atomicOr(&held[s], 0x40000000u);
                max_u16(biased, s, static_cast<uint32_t>(i + 1));
                listed[s] = static_cast<uint16_t>(k);
            });
        __syncthreads();
        return here;
    };
    int here = 0, k_own = 0;
    uint32_t x_own = 0, m_own = ~0u;
    auto own = [&](int i) {
        k_own = listed[i];
        x_own = r.x[v0 + k_own];
        if (r.mask) m_own = __ldg(r.mask + ((v0 + k_own) >> 5));
    };
    if (n > 0) {
        here = collect(0);
        if (tid < here) own(tid);                          // the thread's first, on its way during the stream
    }

    float top = -INFINITY;
    int top_at = 0;
    // one step; EDGE: of a batch with groups that are not whole
    float *const po = r.out + own0;                        // used where r.out is given
    const uint32_t *const my_marks = marked + (tid >> 3);
    const int mark_shift = 4 * (tid & 7);
    auto one_step = [&](int i, int number, auto is_edge) {
        constexpr bool EDGE = decltype(is_edge)::value;
        const int v = own0 + number * kStep;
        if (EDGE && (v + 4 <= 0 || v >= a.V)) return;
        float y[4];
        four<EDGE>(r, v, lo[i], hi[i], y);
        uint32_t bits = EDGE ? mask_bits(m_lo[i], m_hi[i], v) : __funnelshift_r(m_lo[i], m_hi[i], own0);   // by own0 % 32
        if (some) bits &= ~(my_marks[number * (kStep / 32)] >> mark_shift);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = bits & (1u << e) ? y[e] : -INFINITY;
        if (r.out) {
            if (!EDGE || (v >= 0 && v + 4 <= a.V)) {
                __stcs(reinterpret_cast<float4 *>(po + number * kStep), make_float4(y[0], y[1], y[2], y[3]));
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (v + e >= 0 && v + e < a.V) r.out[v + e] = y[e];
            }
        }
        const float most = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
        const int at = v + (y[0] == most ? 0 : y[1] == most ? 1 : y[2] == most ? 2 : 3);
        top_at = most > top ? at : top_at;
        top = fmaxf(top, most);
    };
#pragma unroll 1
    for (int s = 0; s < STEPS; s += BATCH) {
        if (edge(s)) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) one_step(i, s + i, std::true_type());
        } else {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) one_step(i, s + i, std::false_type());
        }
        if (s + BATCH < STEPS) load(s + BATCH);
    }
    unsigned long long key = key_of(top, top_at);
    if (n > 0) {
        __syncthreads();                                   // the stream's stores come before these
        for (int from = 0;;) {
            for (int i = tid; i < here; i += kLogitsThreads) {
                if (i != tid || from > 0) own(i);
                const int v = v0 + k_own;
                const uint32_t c = held[i], times = c & 0x3FFFFFFFu;
                float z = __uint_as_float(x_own << 16);
                if ((c & 0x80000000u) || times) z = z > 0.0f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
                if (times) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, static_cast<float>(times))), pres);
                if (c & 0x40000000u)
                    z = __fadd_rn(z, __ldg(a.r.bias + static_cast<int64_t>(row) * a.r.n_bias + biased[i] - 1));
                if (!((m_own >> (v & 31)) & 1u)) z = -INFINITY;
                if (r.out) r.out[v] = z;
                const unsigned long long kz = key_of(z, v);
                key = kz > key ? kz : key;
            }
            from += kMarks;
            if (from >= n) break;
            __syncthreads();
            here = collect(from);
        }
    }
    if (!a.argmax) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long k = __shfl_xor_sync(0xffffffffu, key, o);
        key = k > key ? k : key;
    }
    __syncthreads();                                       // best is zero
    if (lane == 0) atomicMax(&best, key);
    __syncthreads();
    if (tid == 0) {
        RowKey *rk = static_cast<RowKey *>(a.ws) + row;
        if (best) atomicMax(&rk->key, best);
        if (atom_add_acq_rel_gpu(&rk->done, 1) == static_cast<int>(gridDim.x) - 1) {
            const unsigned long long k = atomicExch(&rk->key, 0ull);
            a.argmax[row] = k ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(k)) : -1;
            rk->done = 0;
        }
    }
}

template <int STEPS, int BATCH>
cudaError_t launch(const LogitsArgs &a, bool pdl, cudaStream_t stream)
{
    constexpr int slice = 4 * kLogitsThreads * STEPS;
    constexpr LogitsPlan plan(slice);
    static_assert(slice <= 32768 && plan.bytes + 1024 <= 48 * 1024, "15-bit places, and no more than any launch may have");
    cudaLaunchConfig_t cfg = {};
    // up to 3 elements of shift
    cfg.gridDim = dim3(static_cast<unsigned>((a.V + 3 + slice - 1) / slice), static_cast<unsigned>(a.M));
    cfg.blockDim = dim3(kLogitsThreads);
    cfg.dynamicSmemBytes = a.r.ids || a.r.bias_ids ? plan.bytes : 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, logits_kernel<STEPS, BATCH>, a, pdl ? 1 : 0);
}

}  // namespace

size_t logits_workspace(int M) { return sizeof(RowKey) * static_cast<size_t>(M); }

cudaError_t launch_logits_process(const LogitsArgs &a, int sms, bool pdl, cudaStream_t stream)
{
    // The shortest slices of which the SMs hold all at once: each slice reads the row's history again.  (Histories of
    // 1000: 5 x 151936 6.7, 7.6, 8.2 and 9.6 us with slices of 2048, 4096, 8192 and 16384; 12 x 128259 10.7, 8.4, 9.0 and
    // 10.2; 24 x 128259 16.0, 12.6, 10.9 and 12.0; 150 x 32003 23.6, 16.4, 13.3 and 12.7.)
    auto fits = [&](int slice) { return static_cast<int64_t>(a.M) * ((a.V + slice - 1) / slice) <= kLogitsCtas * sms; };
    return fits(2048)   ? launch<2, 2>(a, pdl, stream)
           : fits(4096) ? launch<4, 4>(a, pdl, stream)
           : fits(8192) ? launch<8, 4>(a, pdl, stream)
                        : launch<16, 4>(a, pdl, stream);
}

}  // namespace bi
