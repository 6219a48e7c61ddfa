// C ABI of the e4m3 linears and the mixture of experts: argument validation and
// dispatch.  Declarations and the contract of every entry point are in include/bi.h.
#include "bi.h"
#include "f8.cuh"
#include "host_common.h"
#include "kernels.cuh"

#include <cuda_runtime.h>

namespace {

using bi::host::aligned16;
using bi::host::aligned4;
using bi::host::device_info;
using bi::host::from_cuda;
using bi::host::overlaps;
using bi::kMaxTokens;

constexpr int kMaxRows = 1 << 20;
constexpr int kMaxK = 1 << 20;
constexpr int kMaxCols = 1 << 24;

bool aligned2(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

bool k_ok(int K) { return K >= 16 && K % 16 == 0 && K <= kMaxK; }

size_t bytes(int64_t rows, int64_t cols, size_t esz) { return static_cast<size_t>(rows) * static_cast<size_t>(cols) * esz; }

size_t strided(int64_t rows, int64_t ld, int64_t cols, size_t esz) { return static_cast<size_t>((rows - 1) * ld + cols) * esz; }

// Bytes from p on; none where p is null or n is 0.
struct Span {
    const void *p;
    size_t n;
    bool meets(const Span &o) const { return p && o.p && n && o.n && overlaps(p, n, o.p, o.n); }
};

// No written span meets another span.
template <size_t W, size_t R>
bool apart(const Span (&written)[W], const Span (&read)[R])
{
    for (size_t i = 0; i < W; ++i) {
        for (const Span &x : read)
            if (written[i].meets(x)) return false;
        for (size_t j = i + 1; j < W; ++j)
            if (written[i].meets(written[j])) return false;
    }
    return true;
}

bi_status quantize(const uint16_t *x, int64_t ldx, int M, int K, int gate, uint8_t *q, float *s_a, unsigned flags,
                   bi_stream_t stream)
{
    const int64_t width = gate < 0 ? K : 2 * static_cast<int64_t>(K);
    if (!x || !q || !s_a || M < 1 || M > kMaxRows || !k_ok(K) || ldx < width ||
        static_cast<int64_t>(M) * bi::f8_blocks(K) > 0x7FFFFFFF)
        return BI_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(q) || !aligned4(s_a) || ldx % 8 != 0) return BI_ERR_ALIGNMENT;
    const Span written[] = {{q, bytes(M, K, 1)}, {s_a, bytes(M, bi::f8_blocks(K), 4)}};
    const Span read[] = {{x, strided(M, ldx, width, 2)}};
    if (!apart(written, read)) return BI_ERR_INVALID_ARG;
    int sms = 0;
    const bi_status st = device_info(&sms);
    if (st != BI_OK) return st;
    bi::F8QuantArgs a;
    a.x = x;
    a.ldx = ldx;
    a.M = M;
    a.K = K;
    a.gate = gate;
    a.q = q;
    a.s = s_a;
    return from_cuda(bi::launch_quantize_f8(a, sms, (flags & BI_FLAG_PDL) != 0, stream));
}

// 2-D tensor of bytes [rows, cols], boxes of 128 columns and box_rows rows.
bi_status encode(CUtensorMap *map, const void *base, long long rows, int cols, int box_rows, bool stream_once)
{
    return bi::host::encode_int8_2d(map, base, rows, cols, bi::kF8Block, box_rows, stream_once);
}

bi_status linear(const uint8_t *q, const float *s_a, int q_rows, int K, const int32_t *src, int R, const int32_t *offsets, int E,
                 const uint8_t *w, const float *s_w, int N, uint16_t *y, void *ws, size_t ws_bytes, unsigned flags,
                 bi_stream_t stream)
{
    if (!q || !s_a || !w || !s_w || !y || q_rows < 1 || q_rows > kMaxRows || R < 1 || R > kMaxRows || E < 1 ||
        E > bi::kMaxExperts || N < 1 || N > kMaxCols || static_cast<int64_t>(E) * N > 0x7FFFFFFF || !k_ok(K))
        return BI_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(w) || !aligned4(s_a) || !aligned4(s_w) || !aligned2(y) || (src && !aligned4(src)) ||
        (offsets && !aligned4(offsets)))
        return BI_ERR_ALIGNMENT;
    if (!ws || ws_bytes < bi_f8_workspace_size() || !aligned16(ws)) return BI_ERR_WORKSPACE;
    const int kb = bi::f8_blocks(K);
    const Span written[] = {{y, bytes(R, N, 2)}, {ws, bi_f8_workspace_size()}};
    const Span read[] = {{q, bytes(q_rows, K, 1)},
                         {s_a, bytes(q_rows, kb, 4)},
                         {src, bytes(R, 1, 4)},
                         {offsets, bytes(E + 1, 1, 4)},
                         {w, bytes(static_cast<int64_t>(E) * N, K, 1)},
                         {s_w, bytes(static_cast<int64_t>(E) * bi::f8_blocks(N), kb, 4)}};
    if (!apart(written, read)) return BI_ERR_INVALID_ARG;
    bi::F8LinearArgs a;
    bi_status st = device_info(&a.sms);
    if (st != BI_OK) return st;
    a.plan = bi::f8_plan(R, E, N, a.sms);
    // rows of the copy of a tile's tokens: with one expert all tiles but the last have as many
    const int tiles = (R + a.plan.cols - 1) / a.plan.cols;
    a.box = !offsets ? ((R + tiles - 1) / tiles + 15) / 16 * 16 : a.plan.T;
    const long long w_rows = static_cast<long long>(E) * N;
    st = encode(&a.map_w, w, w_rows, K, 128, true);
    if (st == BI_OK) st = encode(&a.map_w16, w, w_rows, K, 16, true);
    if (st == BI_OK && !src) st = encode(&a.map_q, q, q_rows, K, a.box, false);
    if (st != BI_OK) return st;
    a.q = q;
    a.s_a = s_a;
    a.s_w = s_w;
    a.src = src;
    a.offsets = offsets;
    a.y = y;
    a.q_rows = q_rows;
    a.R = R;
    a.E = E;
    a.N = N;
    a.K = K;
    a.status = bi::workspace_view(ws).status;
    return from_cuda(bi::launch_linear_f8(a, (flags & BI_FLAG_PDL) != 0, stream));
}

}  // namespace

extern "C" {

bi_status bi_quantize_act_f8(const uint16_t *x, int64_t ldx, int M, int K, uint8_t *q, float *s_a, unsigned flags,
                             bi_stream_t stream)
{
    return quantize(x, ldx, M, K, -1, q, s_a, flags, stream);
}

bi_status bi_gated_quantize_f8(const uint16_t *gu, int64_t ldgu, int M, int K, int gate, uint8_t *q, float *s_a, unsigned flags,
                               bi_stream_t stream)
{
    if (gate != BI_GATE_RELU && gate != BI_GATE_SILU) return BI_ERR_INVALID_ARG;
    return quantize(gu, ldgu, M, K, gate, q, s_a, flags, stream);
}

bi_status bi_quantize_weight_f8(const float *w, int64_t ldw, int N, int K, uint8_t *w_q, float *s_w, bi_stream_t stream)
{
    if (!w || !w_q || !s_w || N < 1 || N > kMaxCols || !k_ok(K) || ldw < K) return BI_ERR_INVALID_ARG;
    if (!aligned16(w) || !aligned16(w_q) || !aligned4(s_w) || ldw % 4 != 0) return BI_ERR_ALIGNMENT;
    const Span written[] = {{w_q, bytes(N, K, 1)}, {s_w, bytes(bi::f8_blocks(N), bi::f8_blocks(K), 4)}};
    const Span read[] = {{w, strided(N, ldw, K, 4)}};
    if (!apart(written, read)) return BI_ERR_INVALID_ARG;
    const bi_status st = device_info(nullptr);
    if (st != BI_OK) return st;
    return from_cuda(bi::launch_quantize_weight_f8(w, ldw, N, K, w_q, s_w, stream));
}

size_t bi_f8_workspace_size(void) { return bi::kWsBytes; }

bi_status bi_linear_f8(const uint8_t *q, const float *s_a, int M, int K, const uint8_t *w, const float *s_w, int N, uint16_t *y,
                       void *ws, size_t ws_bytes, unsigned flags, bi_stream_t stream)
{
    return linear(q, s_a, M, K, nullptr, M, nullptr, 1, w, s_w, N, y, ws, ws_bytes, flags, stream);
}

bi_status bi_linear_f8_grouped(const uint8_t *q, const float *s_a, int q_rows, int K, const int32_t *src, int R,
                               const int32_t *offsets, int E, const uint8_t *w, const float *s_w, int N, uint16_t *y, void *ws,
                               size_t ws_bytes, unsigned flags, bi_stream_t stream)
{
    if (!offsets || (!src && q_rows < R)) return BI_ERR_INVALID_ARG;
    return linear(q, s_a, q_rows, K, src, R, offsets, E, w, s_w, N, y, ws, ws_bytes, flags, stream);
}

size_t bi_moe_route_workspace_size(int M, int E)
{
    return M < 1 || M > kMaxTokens || E < 1 || E > bi::kMaxExperts ? 0 : bi::moe_route_workspace(M, E);
}

bi_status bi_moe_route(const void *logits, int64_t ldl, int type, int M, int E, int k, int score, int renorm, float scale,
                       int32_t *ids, float *weights, int32_t *offsets, int32_t *src, int32_t *pos, void *ws, size_t ws_bytes,
                       unsigned flags, bi_stream_t stream)
{
    if (!logits || !ids || !weights || !offsets || !src || !pos || M < 1 || M > kMaxTokens || E < 1 || E > bi::kMaxExperts ||
        k < 1 || k > bi::kMaxTopK || k > E || ldl < E || (type != BI_TYPE_F32 && type != BI_TYPE_BF16) ||
        (score != BI_ROUTE_SOFTMAX && score != BI_ROUTE_SIGMOID) || !(scale >= -3.402823466e38f && scale <= 3.402823466e38f))
        return BI_ERR_INVALID_ARG;
    if (!(type == BI_TYPE_F32 ? aligned4(logits) : aligned2(logits)) || !aligned4(ids) || !aligned4(weights) ||
        !aligned4(offsets) || !aligned4(src) || !aligned4(pos))
        return BI_ERR_ALIGNMENT;
    if (!ws || ws_bytes < bi::moe_route_workspace(M, E) || !aligned16(ws)) return BI_ERR_WORKSPACE;
    const size_t slots = bytes(M, k, 4);
    const Span written[] = {{ids, slots}, {weights, slots}, {offsets, bytes(E + 1, 1, 4)}, {src, slots}, {pos, slots},
                            {ws, bi::moe_route_workspace(M, E)}};
    const Span read[] = {{logits, strided(M, ldl, E, type == BI_TYPE_F32 ? 4 : 2)}};
    if (!apart(written, read)) return BI_ERR_INVALID_ARG;
    const bi_status st = device_info(nullptr);
    if (st != BI_OK) return st;
    bi::RouteArgs a;
    a.logits = logits;
    a.ldl = ldl;
    a.half = type == BI_TYPE_BF16;
    a.M = M;
    a.E = E;
    a.k = k;
    a.score = score;
    a.renorm = renorm != 0;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.src = src;
    a.pos = pos;
    a.ws = ws;
    return from_cuda(bi::launch_moe_route(a, (flags & BI_FLAG_PDL) != 0, stream));
}

bi_status bi_moe_combine(const uint16_t *rows, int R, const int32_t *pos, const float *weights, int M, int k, int N,
                         const uint16_t *base, uint16_t *y, unsigned flags, bi_stream_t stream)
{
    if (!rows || !pos || !weights || !y || R < 1 || R > kMaxRows * 2 || M < 1 || M > kMaxTokens || k < 1 || k > bi::kMaxTopK ||
        N < 1 || N > kMaxCols)
        return BI_ERR_INVALID_ARG;
    if (!aligned2(rows) || !aligned4(pos) || !aligned4(weights) || (base && !aligned2(base)) || !aligned2(y))
        return BI_ERR_ALIGNMENT;
    const Span written[] = {{y, bytes(M, N, 2)}};
    const Span read[] = {{rows, bytes(R, N, 2)}, {pos, bytes(M, k, 4)}, {weights, bytes(M, k, 4)},
                         {base == y ? nullptr : base, bytes(M, N, 2)}};
    if (!apart(written, read)) return BI_ERR_INVALID_ARG;
    const bi_status st = device_info(nullptr);
    if (st != BI_OK) return st;
    bi::CombineArgs a;
    a.rows = rows;
    a.R = R;
    a.pos = pos;
    a.weights = weights;
    a.base = base;
    a.y = y;
    a.M = M;
    a.k = k;
    a.N = N;
    return from_cuda(bi::launch_moe_combine(a, (flags & BI_FLAG_PDL) != 0, stream));
}

}  // extern "C"
