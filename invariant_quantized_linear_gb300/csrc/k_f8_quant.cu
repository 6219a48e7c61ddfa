// Quantisation to e4m3 with a scale for each 128 elements of a row, of bf16 rows
// as they are or behind the gated product, and of fp32 weights with a scale for
// each block of 128 x 128.
//
// A block's scale is RN(amax / 448), 448 being the largest e4m3 value, and a code
// is the e4m3 rounding of RN(x / scale).  The gated product stays in fp32: it is
// never written, so nothing asks for a bf16 rounding of it.
//
// Bound: HBM; 3 bytes an element read and written, 5 behind the gate.  Half a warp
// takes a block, 8 elements (16 bytes) a lane, so that the block's largest is four
// shuffles away and its elements stay in registers.  8192 x 12288 behind silu: 101 us,
// 5.0 TB/s (0.74 of the copy rate); behind relu 91; as it is 74, 4.1 TB/s.  The plain
// form moves 3/5 of the bytes in 3/4 of the time, so instructions show beside the
// stream; a division that each thread does no more took 10 us of it.  8192 x 4096 as it
// is: 24.9 us.  One row of 4096: 1.9 us, a launch and one read's latency.
#include "f8.cuh"
#include "ptx.cuh"
#include "row_ops.cuh"

namespace bi {

namespace {

constexpr int kThreads = 256;
constexpr float kTop = 448.0f;

// two e4m3 codes, lo in the low byte; values beyond 448 become 448, NaN stays NaN
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The scale of a block whose largest magnitude is amax: a quotient that
// underflows to zero (as for a block of zeros) is taken as 1.
__device__ __forceinline__ float scale_of(float amax)
{
    const float s = __fdiv_rn(amax, kTop);
    return s == 0.0f ? 1.0f : s;
}

// Codes of 8 elements.  RN(t / s) by quotient_rn where that is the IEEE quotient
// for every quotient that does not round to code 0.
__device__ __forceinline__ uint2 codes8(const float (&t)[8], float s, bool plain, float inv)
{
    float v[8];
    if (plain) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = copysignf(quotient_rn(t[e], s, inv), t[e]);   // its zeros have lost their sign
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fdiv_rn(t[e], s);
    }
    return make_uint2(e4m3x2(v[0], v[1]) | (e4m3x2(v[2], v[3]) << 16), e4m3x2(v[4], v[5]) | (e4m3x2(v[6], v[7]) << 16));
}

// act(g) u in fp32.  silu by the hardware's exponential and reciprocal: relative
// error below (|g| + 8) 2^-23, far below a code's 2^-4.  Both flush what is not a
// normal number, and 1 / (1 + exp(-g)) is none from g = -87.4 on, where g times it
// still is.  LOW: for g below kLowGate the exponential is taken as 2^-64 of itself
// (the 1 beside it is nothing there, either way) and the product scaled back, which
// holds to g = -131; for other g the bits are the same as without LOW.
constexpr float kLowGate = -80.0f;

template <int GATE, bool LOW>
__device__ __forceinline__ float gated(float g, float u)
{
    if (GATE == BI_GATE_RELU) return __fmul_rn(relu_pos(g), u);
    const bool low = LOW && g < kLowGate;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmaf_rn(g, -1.4426950408889634f, low ? -64.0f : -0.0f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, e)));
    const float t = __fmul_rn(__fmul_rn(g, r), u);
    return low ? __fmul_rn(t, 0x1p-64f) : t;
}

// GATE -1: x as it is.  Blocks are counted in 32 bits: their division by kb in 64 cost 7 us of 106 (8192 x 12288 behind
// silu) and 10 of 84 (as it is).  Returns the largest of this thread's gates as whole numbers, 16 bits each: the negative one farthest from 0, if any.
template <int GATE, int AHEAD, bool LOW>
__device__ __forceinline__ uint32_t quantize_blocks(const F8QuantArgs &a, unsigned kb, unsigned blocks)
{
    uint32_t lowest = 0;
    const int sub = threadIdx.x & 15;
    const unsigned step = gridDim.x * (kThreads / 16);
    for (unsigned at = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);; at += AHEAD * step) {
        // the two halves of a warp leave together: they share the shuffles
        if (__all_sync(0xffffffffu, at >= blocks)) break;
        uint4 x[AHEAD], up[AHEAD];
        long long row[AHEAD];
        int col[AHEAD];
        bool there[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const unsigned b = at + i * step, r = b / kb;
            row[i] = r;
            col[i] = static_cast<int>(b - r * kb) * kF8Block + sub * 8;
            there[i] = b < blocks && col[i] < a.K;
            x[i] = up[i] = make_uint4(0, 0, 0, 0);
            if (there[i]) {
                const uint16_t *p = a.x + row[i] * a.ldx + col[i];
                x[i] = __ldcs(reinterpret_cast<const uint4 *>(p));
                if (GATE >= 0) up[i] = __ldcs(reinterpret_cast<const uint4 *>(p + a.K));
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            const uint32_t v[4] = {up[i].x, up[i].y, up[i].z, up[i].w};
            if (GATE == BI_GATE_SILU && !LOW) lowest = __vimax3_u16x2(__vimax3_u16x2(lowest, w[0], w[1]), w[2], w[3]);
            float t[8];
            uint32_t top = 0;   // bits of the largest magnitude: NaN is above infinity, and is kept
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[e] = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
                if (GATE >= 0) t[e] = gated<GATE, LOW>(t[e], (e & 1) ? bf16_hi(v[e >> 1]) : bf16_lo(v[e >> 1]));
                top = max(top, __float_as_uint(t[e]) & 0x7FFFFFFFu);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float s = scale_of(__uint_as_float(top));
            const bool plain = s >= kQuotientMinScale && s <= 0x1p64f;
            if (!there[i]) continue;
            *reinterpret_cast<uint2 *>(a.q + row[i] * a.K + col[i]) = codes8(t, s, plain, __fdiv_rn(1.0f, s));
            if (sub == 0) a.s[row[i] * kb + col[i] / kF8Block] = s;
        }
    }
    return lowest;
}

// The warp's blocks once more, for gates below kLowGate.  Not inlined: its registers would be the kernel's (8 us more).
template <int GATE>
__device__ __noinline__ void quantize_low(const F8QuantArgs &a, unsigned kb, unsigned blocks)
{
    quantize_blocks<GATE, 1, true>(a, kb, blocks);
}

// Gates that low are rare.  A warp that has met one goes over its blocks a second time: 101 us for 8192 x 12288 without any
// (99 if they were not looked for), 121 with one a row.  With the counts in 64 bits, when this took 109: a choice for each
// element 120, a branch for each block 111.
template <int GATE, int AHEAD>
__global__ void __launch_bounds__(kThreads) quantize_f8_kernel(F8QuantArgs a, unsigned kb, unsigned blocks, int pdl)
{
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const uint32_t lowest = quantize_blocks<GATE, AHEAD, false>(a, kb, blocks);
    if (GATE == BI_GATE_SILU) {
        constexpr uint32_t kBits = 0xC2A0;                           // kLowGate as bf16
        if (__any_sync(0xffffffffu, (lowest >> 16) > kBits || (lowest & 0xFFFF) > kBits)) quantize_low<GATE>(a, kb, blocks);
    }
}

// One CTA a block of 128 x 128: its largest magnitude, then its codes (the second reading comes from L1 or L2).
__global__ void __launch_bounds__(kThreads) quantize_weight_f8_kernel(const float *__restrict__ w, int64_t ldw, int N, int K,
                                                                      uint8_t *__restrict__ q, float *__restrict__ s_w)
{
    __shared__ uint32_t tops[kThreads / 32];
    const int kb = gridDim.x;
    const long long n0 = static_cast<long long>(blockIdx.y) * kF8Block;
    const int k0 = blockIdx.x * kF8Block;
    const int rows = static_cast<int>(min(static_cast<long long>(kF8Block), N - n0)), lane = threadIdx.x & 31;
    const int k = k0 + 4 * lane;
    uint32_t top = 0;
    if (k < K)
        for (int r = threadIdx.x >> 5; r < rows; r += kThreads / 32) {
            const float4 v = *reinterpret_cast<const float4 *>(w + (n0 + r) * ldw + k);
            top = max(max(top, __float_as_uint(v.x) & 0x7FFFFFFFu), __float_as_uint(v.y) & 0x7FFFFFFFu);
            top = max(max(top, __float_as_uint(v.z) & 0x7FFFFFFFu), __float_as_uint(v.w) & 0x7FFFFFFFu);
        }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, tops[i]);
    const float s = scale_of(__uint_as_float(top));
    if (threadIdx.x == 0) s_w[static_cast<long long>(blockIdx.y) * kb + blockIdx.x] = s;
    if (k >= K) return;
    for (int r = threadIdx.x >> 5; r < rows; r += kThreads / 32) {
        const float4 v = *reinterpret_cast<const float4 *>(w + (n0 + r) * ldw + k);
        const uint32_t c = e4m3x2(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s)) | (e4m3x2(__fdiv_rn(v.z, s), __fdiv_rn(v.w, s)) << 16);
        *reinterpret_cast<uint32_t *>(q + (n0 + r) * K + k) = c;
    }
}

template <int GATE, int AHEAD>
cudaError_t launch(const F8QuantArgs &a, unsigned grid, unsigned kb, unsigned blocks, bool pdl, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, quantize_f8_kernel<GATE, AHEAD>, a, kb, blocks, pdl ? 1 : 0);
}

template <int AHEAD>
cudaError_t launch(const F8QuantArgs &a, unsigned grid, unsigned kb, unsigned blocks, bool pdl, cudaStream_t stream)
{
    if (a.gate < 0) return launch<-1, AHEAD>(a, grid, kb, blocks, pdl, stream);
    if (a.gate == BI_GATE_RELU) return launch<BI_GATE_RELU, AHEAD>(a, grid, kb, blocks, pdl, stream);
    return launch<BI_GATE_SILU, AHEAD>(a, grid, kb, blocks, pdl, stream);
}

}  // namespace

cudaError_t launch_quantize_f8(const F8QuantArgs &a, int sms, bool pdl, cudaStream_t stream)
{
    // Up to eight CTAs a SM a block of 128 a half warp; longer calls read two ahead.
    const unsigned kb = f8_blocks(a.K), blocks = a.M * kb, ctas = (blocks + kThreads / 16 - 1) / (kThreads / 16);
    if (ctas <= 8u * sms) return launch<1>(a, ctas, kb, blocks, pdl, stream);
    const unsigned half = (ctas + 1) / 2, most = 64u * sms;
    return launch<2>(a, half < most ? half : most, kb, blocks, pdl, stream);
}

cudaError_t launch_quantize_weight_f8(const float *w, int64_t ldw, int N, int K, uint8_t *w_q, float *s_w, cudaStream_t stream)
{
    const int kb = f8_blocks(K), most = 65535 * kF8Block;
    for (int n = 0; n < N; n += most) {                  // a grid's second axis ends at 65535
        const int rows = N - n < most ? N - n : most;
        quantize_weight_f8_kernel<<<dim3(kb, f8_blocks(rows)), kThreads, 0, stream>>>(
            w + n * ldw, ldw, rows, K, w_q + static_cast<int64_t>(n) * K, s_w + static_cast<int64_t>(n / kF8Block) * kb);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || N - n <= most) return e;
    }
    return cudaSuccess;
}

}  // namespace bi
