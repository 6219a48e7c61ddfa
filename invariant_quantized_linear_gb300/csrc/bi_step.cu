// C ABI of the decoder-step operators: argument validation and dispatch.
// Declarations and the contract of every entry point are in include/bi.h.
#include "bi.h"
#include "host_common.h"
#include "kernels.cuh"
#include "step.cuh"

#include <algorithm>
#include <cuda_runtime.h>
#include <math.h>

namespace {

using bi::host::aligned16;
using bi::host::aligned4;
using bi::host::check_k;
using bi::host::device_info;
using bi::host::from_cuda;
using bi::host::overlaps;

constexpr int kMaxHeads = 1024;
constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxPositions = 1 << 22;
constexpr int kMaxAttnRows = 1 << 22;   // query rows of a sequence and kv head
constexpr int kMaxVocab = 1 << 24;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// log2 of a supported page size, or -1
int page_shift(int page_size)
{
    switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    }
    return -1;
}

bool head_size_ok(int D) { return D == 64 || D == 128; }

bi_status check_cache(const bi_kv4_cache *c)
{
    if (!c || !c->pool || c->num_pages < 1 || c->Hkv < 1 || c->Hkv > kMaxHeads || !head_size_ok(c->D) ||
        page_shift(c->page_size) < 0)
        return BI_ERR_INVALID_ARG;
    if (c->page_stride < static_cast<int64_t>(c->Hkv) * bi::Kv4Layout::block(c->page_size, c->D))
        return BI_ERR_INVALID_ARG;
    if (!aligned16(c->pool) || (c->page_stride % 16) != 0) return BI_ERR_ALIGNMENT;
    return BI_OK;
}

bi_status check_batch(const bi_kv4_batch *b)
{
    if (!b || !b->cu_q || !b->kv_len || !b->pages || b->ld_pages < 1 || b->B < 1 || b->B > 65535 || b->T < 1 ||
        b->T > kMaxTokens || b->max_q < 1 || b->max_q > 65535 || b->max_kv < 1 || b->max_kv > kMaxPositions)
        return BI_ERR_INVALID_ARG;
    if (!aligned4(b->cu_q) || !aligned4(b->kv_len) || !aligned4(b->pages)) return BI_ERR_ALIGNMENT;
    return BI_OK;
}

bi::Kv4View view(const bi_kv4_cache *c, const bi_kv4_batch *b)
{
    bi::Kv4View v;
    v.pool = static_cast<unsigned char *>(c->pool);
    v.page_stride = c->page_stride;
    v.num_pages = c->num_pages;
    v.page_shift = page_shift(c->page_size);
    v.Hkv = c->Hkv;
    v.cu_q = b->cu_q;
    v.kv_len = b->kv_len;
    v.pages = b->pages;
    v.ld_pages = b->ld_pages;
    v.B = b->B;
    v.T = b->T;
    v.max_q = b->max_q;
    v.max_kv = b->max_kv;
    return v;
}

size_t rows_bytes(int64_t rows, int64_t ld, int64_t width, size_t esz)
{
    return static_cast<size_t>((rows - 1) * ld + width) * esz;
}

// Bytes from p on; none where p is null or n is 0.
struct Span {
    const void *p;
    size_t n;
    bool meets(const Span &o) const { return p && o.p && n && o.n && overlaps(p, n, o.p, o.n); }
};

bool finite_at_least(float x, float least) { return x >= least && x <= 3.402823466e38f; }

}  // namespace

extern "C" {

bi_status bi_rmsnorm_quantize(const uint16_t *h, int64_t ldh, const uint16_t *y, int64_t ldy, const uint16_t *w,
                              float eps, int M, int K, uint16_t *h_out, int64_t ldo, int8_t *q, float *s_a,
                              unsigned flags, bi_stream_t stream)
{
    if (!h || !w || !q || !s_a || (y == nullptr) != (h_out == nullptr) || M < 1 || M > 65535 || ldh < K ||
        (y && (ldy < K || ldo < K)) || !finite_at_least(eps, 0.0f))
        return BI_ERR_INVALID_ARG;
    bi_status st = check_k(K);
    if (st != BI_OK) return st;
    if (!aligned16(h) || !aligned16(w) || !aligned16(q) || !aligned4(s_a) || (ldh % 8) != 0 ||
        (y && (!aligned16(y) || !aligned16(h_out) || (ldy % 8) != 0 || (ldo % 8) != 0)))
        return BI_ERR_ALIGNMENT;
    const size_t hb = rows_bytes(M, ldh, K, 2), qb = static_cast<size_t>(M) * K, sb = 4u * static_cast<size_t>(M);
    if (overlaps(q, qb, h, hb) || overlaps(s_a, sb, h, hb) || overlaps(q, qb, s_a, sb) || overlaps(q, qb, w, 2u * K) ||
        overlaps(s_a, sb, w, 2u * K))
        return BI_ERR_INVALID_ARG;
    if (y) {
        const size_t yb = rows_bytes(M, ldy, K, 2), ob = rows_bytes(M, ldo, K, 2);
        const bool in_place = h_out == h && ldo == ldh;
        if ((!in_place && overlaps(h_out, ob, h, hb)) || overlaps(h_out, ob, y, yb) || overlaps(h_out, ob, w, 2u * K) ||
            overlaps(q, qb, y, yb) || overlaps(s_a, sb, y, yb) || overlaps(q, qb, h_out, ob) || overlaps(s_a, sb, h_out, ob))
            return BI_ERR_INVALID_ARG;
    }
    int sms = 0;
    st = device_info(&sms);
    if (st != BI_OK) return st;
    bi::NormArgs a;
    a.h = h;
    a.y = y;
    a.w = w;
    a.h_out = h_out;
    a.ldh = ldh;
    a.ldy = ldy;
    a.ldo = ldo;
    a.eps = eps;
    a.M = M;
    a.K = K;
    a.q = q;
    a.s_a = s_a;
    return from_cuda(bi::launch_rmsnorm_quantize(a, sms, (flags & BI_FLAG_PDL) != 0, stream));
}

size_t bi_kv4_block_bytes(int page_size, int D)
{
    if (page_shift(page_size) < 0 || !head_size_ok(D)) return 0;
    return static_cast<size_t>(bi::Kv4Layout::block(page_size, D));
}

bi_status bi_rope_table(const double *inv_freq, int n_freq, float amp, int n_pos, float *rope, bi_stream_t stream)
{
    if (!inv_freq || !rope || n_freq < 1 || n_freq > 65536 || n_pos < 1 || n_pos > kMaxPositions ||
        !finite_at_least(fabsf(amp), 0.0f))
        return BI_ERR_INVALID_ARG;
    if (!aligned(inv_freq, 8) || !aligned(rope, 8)) return BI_ERR_ALIGNMENT;
    const bi_status st = device_info(nullptr);
    if (st != BI_OK) return st;
    return from_cuda(bi::launch_rope_table(inv_freq, n_freq, amp, n_pos, reinterpret_cast<float2 *>(rope), stream));
}

bi_status bi_rope_append_kv4(const uint16_t *q, int64_t ldq, int Hq, const uint16_t *k, int64_t ldk, const uint16_t *v,
                             int64_t ldv, const uint16_t *q_norm, const uint16_t *k_norm, float eps, const float *rope,
                             int n_pos, int rot, int layout, uint16_t *q_out, const bi_kv4_cache *cache,
                             const bi_kv4_batch *batch, unsigned flags, bi_stream_t stream)
{
    bi_status st = check_cache(cache);
    if (st != BI_OK) return st;
    st = check_batch(batch);
    if (st != BI_OK) return st;
    const int64_t D = cache->D, T = batch->T, wq = Hq * D, wk = cache->Hkv * D;
    if (!q || !k || !v || !q_out || !rope || Hq < 1 || Hq > kMaxHeads || ldq < wq || ldk < wk || ldv < wk || n_pos < 1 ||
        rot < 0 || rot > D || (rot % (layout == BI_ROPE_HALF ? 8 : 4)) != 0 ||
        (layout != BI_ROPE_HALF && layout != BI_ROPE_INTERLEAVED) ||
        !finite_at_least(eps, 0.0f))
        return BI_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(rope) ||
        (q_norm && !aligned16(q_norm)) || (k_norm && !aligned16(k_norm)) || (ldq % 8) != 0 || (ldk % 8) != 0 ||
        (ldv % 8) != 0)
        return BI_ERR_ALIGNMENT;
    const size_t ob = static_cast<size_t>(T * wq) * 2;
    if (overlaps(q_out, ob, q, rows_bytes(T, ldq, wq, 2)) || overlaps(q_out, ob, k, rows_bytes(T, ldk, wk, 2)) ||
        overlaps(q_out, ob, v, rows_bytes(T, ldv, wk, 2)))
        return BI_ERR_INVALID_ARG;
    int sms = 0;
    st = device_info(&sms);
    if (st != BI_OK) return st;
    bi::RopeAppendArgs a;
    a.c = view(cache, batch);
    a.q = q;
    a.k = k;
    a.v = v;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.Hq = Hq;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    a.rope = reinterpret_cast<const float2 *>(rope);
    a.n_pos = n_pos;
    a.rot = rot;
    a.q_out = q_out;
    return from_cuda(bi::launch_rope_append_kv4(a, cache->D, layout == BI_ROPE_INTERLEAVED, sms,
                                                (flags & BI_FLAG_PDL) != 0, stream));
}

bi_status bi_kv4_gather(const bi_kv4_cache *cache, const bi_kv4_batch *batch, uint16_t *k_out, uint16_t *v_out,
                        bi_stream_t stream)
{
    bi_status st = check_cache(cache);
    if (st != BI_OK) return st;
    st = check_batch(batch);
    if (st != BI_OK) return st;
    if (!k_out || !v_out) return BI_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out)) return BI_ERR_ALIGNMENT;
    const size_t nb = static_cast<size_t>(batch->T) * cache->Hkv * cache->D * 2;
    if (overlaps(k_out, nb, v_out, nb)) return BI_ERR_INVALID_ARG;
    int sms = 0;
    st = device_info(&sms);
    if (st != BI_OK) return st;
    return from_cuda(bi::launch_kv4_gather(view(cache, batch), cache->D, k_out, v_out, sms, stream));
}

size_t bi_attention_kv4_workspace_size(int Hq, const bi_kv4_cache *cache, const bi_kv4_batch *batch)
{
    if (!cache || !batch || Hq < 1 || Hq > kMaxHeads || cache->Hkv < 1 || cache->Hkv > kMaxHeads || Hq % cache->Hkv != 0 ||
        !head_size_ok(cache->D) || batch->B < 1 || batch->B > 65535 || batch->T < 1 || batch->T > kMaxTokens ||
        batch->max_q < 1 || batch->max_q > 65535 || batch->max_kv < 1 || batch->max_kv > kMaxPositions)
        return 0;
    // at least what bi_workspace_status asks for
    return std::max(bi::kWsBytes, bi::attention_kv4_workspace(Hq, cache->D, batch->T, batch->max_kv));
}

bi_status bi_attention_kv4(const uint16_t *q, int64_t ldq, int Hq, const bi_kv4_cache *cache, const bi_kv4_batch *batch,
                           float scale, uint16_t *o, void *ws, size_t ws_bytes, unsigned flags, bi_stream_t stream)
{
    bi_status st = check_cache(cache);
    if (st != BI_OK) return st;
    st = check_batch(batch);
    if (st != BI_OK) return st;
    const int64_t wq = static_cast<int64_t>(Hq) * cache->D;
    if (static_cast<int64_t>(batch->max_q) * (Hq / cache->Hkv) > kMaxAttnRows) return BI_ERR_INVALID_ARG;
    if (!q || !o || Hq < 1 || Hq > kMaxHeads || Hq % cache->Hkv != 0 || ldq < wq || !(scale > 0.0f) ||
        !finite_at_least(scale, 0.0f))
        return BI_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || (ldq % 8) != 0) return BI_ERR_ALIGNMENT;
    if (overlaps(o, static_cast<size_t>(batch->T) * wq * 2, q, rows_bytes(batch->T, ldq, wq, 2))) return BI_ERR_INVALID_ARG;
    const size_t need = bi_attention_kv4_workspace_size(Hq, cache, batch);
    if (need == 0) return BI_ERR_INVALID_ARG;
    if (!ws || ws_bytes < need || !aligned16(ws)) return BI_ERR_WORKSPACE;
    if (overlaps(ws, need, q, rows_bytes(batch->T, ldq, wq, 2)) || overlaps(ws, need, o, static_cast<size_t>(batch->T) * wq * 2))
        return BI_ERR_INVALID_ARG;
    bi::AttnKv4Args a;
    st = device_info(&a.sms);
    if (st != BI_OK) return st;
    a.c = view(cache, batch);
    a.q = q;
    a.ldq = ldq;
    a.Hq = Hq;
    a.scale = scale;
    a.o = o;
    a.ws = ws;
    return from_cuda(bi::launch_attention_kv4(a, cache->D, (flags & BI_FLAG_PDL) != 0, stream));
}

size_t bi_logits_workspace_size(int M) { return M < 1 || M > 65535 ? 0 : bi::logits_workspace(M); }

bi_status bi_logits_process(const uint16_t *logits, int64_t ldl, int M, int V, const bi_logits_rules *rules, float *out,
                            int64_t ldo, int32_t *argmax, void *ws, size_t ws_bytes, unsigned flags, bi_stream_t stream)
{
    if (!logits || !rules || M < 1 || M > 65535 || V < 1 || V > kMaxVocab || ldl < V || (!out && !argmax) ||
        (out && ldo < V))
        return BI_ERR_INVALID_ARG;
    const bi_logits_rules &r = *rules;
    if ((r.ids && (!r.begin || !r.mid || !r.end)) || r.n_bias < 0 || r.n_bias > 65535 ||
        (r.n_bias > 0 && (!r.bias_ids || !r.bias)) || (r.mask && r.ld_mask < (V + 31) / 32))
        return BI_ERR_INVALID_ARG;
    if (!aligned(logits, 2) || !aligned4(out) || !aligned4(argmax) || !aligned4(r.ids) || !aligned4(r.begin) ||
        !aligned4(r.mid) || !aligned4(r.end) || !aligned4(r.repetition) || !aligned4(r.presence) ||
        !aligned4(r.frequency) || !aligned4(r.bias_ids) || !aligned4(r.bias) || !aligned4(r.mask))
        return BI_ERR_ALIGNMENT;
    if (!ws || ws_bytes < bi::logits_workspace(M) || !aligned16(ws)) return BI_ERR_WORKSPACE;
    // what is written overlaps nothing; the extent of ids is the device's to know
    const size_t per_row = 4 * static_cast<size_t>(M), per_bias = per_row * static_cast<size_t>(r.n_bias);
    const Span written[] = {{out, out ? rows_bytes(M, ldo, V, 4) : 0}, {argmax, per_row}, {ws, bi::logits_workspace(M)}};
    const Span read[] = {{logits, rows_bytes(M, ldl, V, 2)},
                         {r.ids ? r.begin : nullptr, per_row},
                         {r.ids ? r.mid : nullptr, per_row},
                         {r.ids ? r.end : nullptr, per_row},
                         {r.repetition, per_row},
                         {r.presence, per_row},
                         {r.frequency, per_row},
                         {r.bias_ids, per_bias},
                         {r.n_bias > 0 ? r.bias : nullptr, per_bias},
                         {r.mask, r.mask ? rows_bytes(M, r.ld_mask, (V + 31) / 32, 4) : 0}};
    for (const Span &w : written) {
        for (const Span &x : read)
            if (w.meets(x)) return BI_ERR_INVALID_ARG;
        for (const Span &x : written)
            if (&w < &x && w.meets(x)) return BI_ERR_INVALID_ARG;
    }
    int sms = 0;
    const bi_status st = device_info(&sms);
    if (st != BI_OK) return st;
    bi::LogitsArgs a;
    a.r = r;
    if (r.n_bias == 0) a.r.bias_ids = nullptr;
    a.logits = logits;
    a.ldl = ldl;
    a.ldo = ldo;
    a.M = M;
    a.V = V;
    a.out = out;
    a.argmax = argmax;
    a.ws = ws;
    return from_cuda(bi::launch_logits_process(a, sms, (flags & BI_FLAG_PDL) != 0, stream));
}

}  // extern "C"
