// Residual addition, RMS norm and per-token int8 quantisation in one pass.
//
// t = h' w is exact in fp32 (two bf16 factors), and the codes rne(t / st),
// st = max|t| / 127, are those of the normalised row t r for any r > 0: the
// per-row absmax rule is invariant to a row's factor.  So the codes need no
// rounding of r, and r enters the scale alone, s_a = st r.
//
// Bound: HBM; 7 bytes an element (h, y read; h', q written).  One CTA a row,
// the row held in registers between the two reductions and the codes (8192 rows
// of 4096: 42 us, 5.6 TB/s, where the codes' instructions show beside the copies;
// without the residual, 3 bytes an element, 27.8 us, 3.6 TB/s: instructions; one row
// 2.5 us, a launch's latency, two passes over a barrier and the memory's).
#include "ptx.cuh"
#include "row_ops.cuh"
#include "step.cuh"

namespace bi {

namespace {

constexpr int kFold = 256;              // sums of squares of a row: chunk j of 8 elements goes to sum j % kFold

template <int THREADS>
__device__ __forceinline__ float2 block_sum_max(float s, float m, float2 *red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = make_float2(s, m);
    __syncthreads();
    s = 0.0f;
    m = 0.0f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        s = __fadd_rn(s, red[w].x);
        m = fmaxf(m, red[w].y);
    }
    return make_float2(s, m);
}

// t = h w of 8 elements: adds their squares of h to s, their |t| to m.
__device__ __forceinline__ void norm8(const uint4 &h, const uint4 &w, float (&t)[8], float &s, float &m)
{
    const uint32_t a[4] = {h.x, h.y, h.z, h.w};
    const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float x = bf16_lo(a[e]), y = bf16_hi(a[e]);
        s = __fmaf_rn(x, x, s);
        s = __fmaf_rn(y, y, s);
        t[2 * e] = __fmul_rn(x, bf16_lo(b[e]));
        t[2 * e + 1] = __fmul_rn(y, bf16_hi(b[e]));
        m = fmaxf(m, fmaxf(fabsf(t[2 * e]), fabsf(t[2 * e + 1])));
    }
}

// bf16_rne(h + y) elementwise (one fp32 add each).
__device__ __forceinline__ uint4 sum8(const uint4 &h, const uint4 &y)
{
    const uint32_t a[4] = {h.x, h.y, h.z, h.w};
    const uint32_t b[4] = {y.x, y.y, y.z, y.w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 v =
            __floats2bfloat162_rn(__fadd_rn(bf16_lo(a[e]), bf16_lo(b[e])), __fadd_rn(bf16_hi(a[e]), bf16_hi(b[e])));
        o[e] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ uint2 codes8_div(const float (&t)[8], float st)
{
    uint32_t o[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e >> 2] |= code_byte(__fdiv_rn(t[e], st)) << (8 * (e & 3));
    return make_uint2(o[0], o[1]);
}

// The codes of 8 elements, r = RN(1 / st), 2^-64 <= st <= 2^64.  A quotient q by
// quotient_rn is t / st but for an error far below an ulp, so rne(q) is the code
// unless q lies within two ulps (2^-16 below 128) of the middle of two codes;
// then (one element in 30,000) all 8 are divided.  |t| / st is at most 127 and a
// rounding, so no code needs a clamp.
__device__ __forceinline__ uint2 codes8(const float (&t)[8], float st, float r)
{
    uint32_t u[8];
    float far = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float q = quotient_rn(t[e], st, r), c = __fadd_rn(q, 12582912.0f);   // rne, as in code_byte
        u[e] = __float_as_uint(c);
        far = fmaxf(far, fabsf(__fsub_rn(q, __fsub_rn(c, 12582912.0f))));
    }
    if (far >= 0.5f - 0x1p-16f) return codes8_div(t, st);
    return make_uint2(__byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410));
}

__device__ __forceinline__ uint4 ldg16(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }

// C chunks of 8 elements a thread in registers; C = 0: any K, the row read twice.
// The sum of a row does not depend on THREADS: chunks to their sums in order, then the kFold sums in the order of warps
// of 32.  With fewer threads than kFold the others' sums are zeros, with more they are handed over.
template <int C, int THREADS>
__global__ void __launch_bounds__(THREADS) rmsnorm_quant_kernel(NormArgs a, int pdl)
{
    static_assert(THREADS == kFold || C == 1 || THREADS > kFold, "a thread has every chunk of its sums");
    __shared__ float2 red[THREADS / 32];
    __shared__ float handed[THREADS > kFold ? C * THREADS : 1];
    if (pdl) {
        pdl_launch_dependents();
        pdl_wait();
    }
    const int64_t row = blockIdx.x;
    const uint16_t *hr = a.h + row * a.ldh;
    const uint16_t *yr = a.y ? a.y + row * a.ldy : nullptr;
    const int K = a.K;
    float s = 0.0f, m = 0.0f;
    float t[C > 0 ? C : 1][8];
    auto load = [&](int k) {
        uint4 h = ldg16(hr + k);
        return yr ? sum8(h, ldg16(yr + k)) : h;
    };
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * THREADS + threadIdx.x) * 8;
            float sum = 0.0f;
            if (k < K) {
                const uint4 h = load(k);
                if (yr) *reinterpret_cast<uint4 *>(a.h_out + row * a.ldo + k) = h;
                norm8(h, ldg16(a.w + k), t[c], sum, m);
            }
            if constexpr (THREADS > kFold) handed[c * THREADS + threadIdx.x] = sum;
            else s = __fadd_rn(s, sum);
        }
        if constexpr (THREADS > kFold) {
            __syncthreads();
            if (threadIdx.x < kFold)
#pragma unroll
                for (int j = 0; j < C * THREADS / kFold; ++j) s = __fadd_rn(s, handed[j * kFold + threadIdx.x]);
        }
    } else {
        for (int k = threadIdx.x * 8; k < K; k += THREADS * 8) {
            float sum = 0.0f;
            norm8(load(k), ldg16(a.w + k), t[0], sum, m);
            s = __fadd_rn(s, sum);
        }
    }
    const float2 r = block_sum_max<THREADS>(s, m, red);
    const float st = r.y == 0.0f ? 1.0f : __fdiv_rn(r.y, 127.0f);
    const bool plain = st >= kQuotientMinScale && st <= 0x1p64f;
    const float inv = __fdiv_rn(1.0f, st);
    auto codes = [&](const float (&x)[8]) { return plain ? codes8(x, st, inv) : codes8_div(x, st); };
    int8_t *qr = a.q + row * K;
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * THREADS + threadIdx.x) * 8;
            if (k < K) *reinterpret_cast<uint2 *>(qr + k) = codes(t[c]);
        }
    } else {
        for (int k = threadIdx.x * 8; k < K; k += THREADS * 8) {
            const uint4 h = load(k);                  // h_out may be h: it is written after its last read
            if (yr) *reinterpret_cast<uint4 *>(a.h_out + row * a.ldo + k) = h;
            norm8(h, ldg16(a.w + k), t[0], s, m);
            *reinterpret_cast<uint2 *>(qr + k) = codes(t[0]);
        }
    }
    if (threadIdx.x == 0) {
        const float rms = __fsqrt_rn(__fadd_rn(__fdiv_rn(r.x, static_cast<float>(K)), a.eps));
        a.s_a[row] = r.y == 0.0f ? 1.0f : __fmul_rn(st, __fdiv_rn(1.0f, rms));
    }
}

template <int C, int THREADS>
cudaError_t launch(const NormArgs &a, bool pdl, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.M));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, rmsnorm_quant_kernel<C, THREADS>, a, pdl ? 1 : 0);
}

}  // namespace

cudaError_t launch_rmsnorm_quantize(const NormArgs &a, int sms, bool pdl, cudaStream_t stream)
{
    // A chunk a thread while that fills warps (8192 rows of 1024: 10.2 us, 12.7 with 256 threads).  Rows that leave an SM at
    // most two CTAs are bound by latency and take 512 threads, longer calls 256: 4 x 8192 3.7 us (256: 4.1), 150 x 4096 3.0
    // (3.6), 300 x 5136 4.3 (4.3), 600 x 5136 6.6 (5.1), 2048 x 4096 11.8 (9.4).
    if (a.K <= 1024) return launch<1, 128>(a, pdl, stream);
    if (a.M <= 2 * sms && a.K > 2048 && a.K <= 16384)
        switch ((a.K + 4095) / 4096) {
        case 1: return launch<1, 512>(a, pdl, stream);
        case 2: return launch<2, 512>(a, pdl, stream);
        case 3: return launch<3, 512>(a, pdl, stream);
        default: return launch<4, 512>(a, pdl, stream);
        }
    // Above 6144 the registers of a row in 256 threads cost more than a second reading from L2 (2048 x 8192: 25.0 us, held
    // 26.8; 2048 x 16384: 50, held 67; 2048 x 5136: 14.3, held 11.6).
    switch ((a.K + 2047) / 2048) {
    case 1: return launch<1, 256>(a, pdl, stream);
    case 2: return launch<2, 256>(a, pdl, stream);
    case 3: return launch<3, 256>(a, pdl, stream);
    default: return launch<0, 256>(a, pdl, stream);
    }
}

}  // namespace bi
