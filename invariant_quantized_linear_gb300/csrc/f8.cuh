// Launch interface of the e4m3 linears and the mixture of experts
// (k_f8_quant.cu, k_f8_linear.cu, k_moe.cu) for the C ABI (bi_f8.cu).
#pragma once

#include "bi.h"

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace bi {

constexpr int kF8Block = 128;       // elements of a row (and of a weight's column) that share a scale
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kMaxTokens = 65535;   // of the routing and the weighted sum

inline int f8_blocks(int n) { return (n + kF8Block - 1) / kF8Block; }

// K values of x or, with gate >= 0 (a bi_gate), of act(x[:, :K]) * x[:, K:2K].
struct F8QuantArgs {
    const uint16_t *x;
    int64_t ldx;
    int M, K;
    int gate;
    uint8_t *q;
    float *s;
};

cudaError_t launch_quantize_f8(const F8QuantArgs &a, int sms, bool pdl, cudaStream_t stream);
cudaError_t launch_quantize_weight_f8(const float *w, int64_t ldw, int N, int K, uint8_t *w_q, float *s_w,
                                      cudaStream_t stream);

// Token columns of a tile: how a call is split into tiles (see f8_plan).
struct F8Plan {
    int T;            // most token columns of a tile: 16, 32, 64, 128 or 192
    int cols;         // tokens a tile is filled to (a multiple of 16, <= T)
};

F8Plan f8_plan(int rows, int experts, int N, int sms);

struct F8LinearArgs {
    CUtensorMap map_w;          // w [E N, K], box 128 B x 128 rows
    CUtensorMap map_w16;        // the same, 16 rows
    CUtensorMap map_q;          // q [rows of q, K], box 128 B x `box` rows; not set where src is given
    int box;
    const uint8_t *q;
    const float *s_a, *s_w;
    const int32_t *src;         // row of q for each row of y, or null: the same row
    const int32_t *offsets;     // [E + 1] rows of each expert, or null: one weight matrix, all rows
    uint16_t *y;
    int q_rows;                 // rows of q
    int R;                      // rows of y
    int E, N, K;
    int *status;
    F8Plan plan;
    int sms;
};

cudaError_t launch_linear_f8(const F8LinearArgs &a, bool pdl, cudaStream_t stream);

struct RouteArgs {
    const void *logits;
    int64_t ldl;
    bool half;                  // bf16 logits, else fp32
    int M, E, k;
    int score;                  // a bi_route_score
    bool renorm;
    float scale;
    int32_t *ids;
    float *weights;
    int32_t *offsets, *src, *pos;
    void *ws;
};

size_t moe_route_workspace(int M, int E);
cudaError_t launch_moe_route(const RouteArgs &a, bool pdl, cudaStream_t stream);

struct CombineArgs {
    const uint16_t *rows;
    int R;
    const int32_t *pos;
    const float *weights;
    const uint16_t *base;       // may be null
    uint16_t *y;
    int M, k, N;
};

cudaError_t launch_moe_combine(const CombineArgs &a, bool pdl, cudaStream_t stream);

}  // namespace bi
