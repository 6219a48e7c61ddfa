// Launch interface of the decoder-step operators (k_norm.cu, k_kv4.cu,
// k_attn_kv4.cu, k_logits.cu) for the C ABI (bi_step.cu), and the 4-bit
// cache's layout as the kernels see it.
#pragma once

#include "bi.h"

#include <cuda_runtime.h>
#include <stdint.h>

namespace bi {

struct NormArgs {
    const uint16_t *h, *y, *w;   // y may be null
    uint16_t *h_out;             // null when y is
    int64_t ldh, ldy, ldo;
    float eps;
    int M, K;
    int8_t *q;
    float *s_a;
};

cudaError_t launch_rmsnorm_quantize(const NormArgs &a, int sms, bool pdl, cudaStream_t stream);

// ------------------------------------------------------------ 4-bit cache

constexpr int kKv4Group = 64;                        // elements that share a scale and a minimum

// Offsets of one kv head's block of a page (P positions, head size D).
struct Kv4Layout {
    __host__ __device__ static constexpr int k_row(int D) { return D / 2; }                     // bytes of a position's key codes
    __host__ __device__ static constexpr int v_pair(int D) { return D; }                        // bytes of a position pair's value codes
    __host__ __device__ static constexpr int p_row(int D) { return 8 * (D / kKv4Group); }       // bytes of a position's parameters
    __host__ __device__ static constexpr int v_off(int P, int D) { return P * (D / 2); }
    __host__ __device__ static constexpr int p_off(int P, int D) { return P * D; }
    __host__ __device__ static constexpr int block(int P, int D) { return P * D + P * p_row(D); }
};

// The cache and the batch by value, for kernels.
struct Kv4View {
    unsigned char *pool;
    int64_t page_stride;
    int num_pages, page_shift, Hkv;
    const int32_t *cu_q, *kv_len, *pages;
    int64_t ld_pages;
    int B, T, max_q, max_kv;
};

struct RopeAppendArgs {
    Kv4View c;
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv;
    int Hq;
    const uint16_t *q_norm, *k_norm;
    float eps;
    const float2 *rope;
    int n_pos, rot;
    uint16_t *q_out;
};

cudaError_t launch_rope_table(const double *inv_freq, int n_freq, float amp, int n_pos, float2 *rope,
                              cudaStream_t stream);
// D is 64 or 128
cudaError_t launch_rope_append_kv4(const RopeAppendArgs &a, int D, bool interleaved, int sms, bool pdl,
                                   cudaStream_t stream);
cudaError_t launch_kv4_gather(const Kv4View &c, int D, uint16_t *k_out, uint16_t *v_out, int sms, cudaStream_t stream);

struct AttnKv4Args {
    Kv4View c;
    const uint16_t *q;
    int64_t ldq;
    int Hq;
    float scale;
    uint16_t *o;
    void *ws;
    int sms;
};

size_t attention_kv4_workspace(int Hq, int D, int T, int max_kv);
cudaError_t launch_attention_kv4(const AttnKv4Args &a, int D, bool pdl, cudaStream_t stream);

struct LogitsArgs {
    bi_logits_rules r;
    const uint16_t *logits;
    int64_t ldl, ldo;
    int M, V;
    float *out;
    int32_t *argmax;
    void *ws;
};

size_t logits_workspace(int M);
cudaError_t launch_logits_process(const LogitsArgs &a, int sms, bool pdl, cudaStream_t stream);

// ------------------------------------------------------------ device helpers

#ifdef __CUDACC__
// The sequence of token row t: the largest b with cu_q[b] <= t, searched by
// the whole warp 32 ways at a time (two rounds of loads up to 1024 sequences).
// Returns -1 for a row past the last sequence's.
__device__ __forceinline__ int kv4_sequence(const Kv4View &c, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = c.B;                             // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool le = lane * step < n && __ldg(c.cu_q + i) <= t;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        if (m == 0) return -1;                       // cu_q[lo] > t: not a valid table
        const int top = 31 - __clz(m);
        n = min(step, n - top * step);
        lo += top * step;
    }
    return __ldg(c.cu_q + lo + 1) > t && __ldg(c.cu_q + lo) <= t ? lo : -1;
}

// Page of position p of sequence b, or -1 when it lies outside the table or the pool.
__device__ __forceinline__ int kv4_page(const Kv4View &c, int b, int p)
{
    const int i = p >> c.page_shift;
    if (p < 0 || i >= c.ld_pages) return -1;
    const int page = __ldg(c.pages + static_cast<int64_t>(b) * c.ld_pages + i);
    return static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages) ? page : -1;
}

// A token row's sequence, position and page; page < 0: leave it out.
struct Kv4Token {
    int b, pos, page;
};

__device__ __forceinline__ Kv4Token kv4_token(const Kv4View &c, int t)
{
    Kv4Token k{-1, -1, -1};
    k.b = kv4_sequence(c, t);
    if (k.b < 0) return k;
    const int begin = __ldg(c.cu_q + k.b), end = __ldg(c.cu_q + k.b + 1);
    if (t - begin >= c.max_q) return k;
    k.pos = __ldg(c.kv_len + k.b) - (end - t);
    if (k.pos >= 0 && k.pos < c.max_kv) k.page = kv4_page(c, k.b, k.pos);
    return k;
}

template <int D>
__device__ __forceinline__ unsigned char *kv4_block(const Kv4View &c, int page, int head)
{
    return c.pool + static_cast<int64_t>(page) * c.page_stride + static_cast<int64_t>(head) * Kv4Layout::block(1 << c.page_shift, D);
}
#endif

}  // namespace bi
