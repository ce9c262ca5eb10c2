// Quantizers of the float8 (e4m3) operators: activations with one scale for each row and block of
// 128 along K (plain, scattered to expert slots, or of a gated activation), weights with one scale
// for each 128 x 128 block.
//
// Over a block: a = max(max |x|, 1e-30), s = a / 448, q = e4m3(x * (448 / a)), every operation
// rounded to nearest even in fp32 and the code rounded once to e4m3 (at most 448 (1 + 2^-22) before
// it, which rounds to 448). The maximum is taken over the bits of |x|, under which an infinity is
// larger than every number and a NaN larger than an infinity: a block that holds one gets the scale
// inf or NaN, and its codes times its scale are NaN, so that a broken value is not hidden.
#include <cuda_fp8.h>

#include "q8_fp8.h"
#include "q8_internal.h"

namespace q8 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ void scale_of(uint32_t amax_bits, float& s, float& r) {
    float a = __uint_as_float(amax_bits);
    a = a < kFp8Tiny ? kFp8Tiny : a;   // a NaN stays
    s = __fdiv_rn(a, kFp8Max);
    r = __fdiv_rn(kFp8Max, a);
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// u * g / (1 + exp(-g)). The fast exponential and division are off by a few 2^-22 relative for
// g > -20 (a thousandth of an e4m3 step); below, the value is under 5e-8 |u|. For 1 + exp(-g) above
// 2^126 the division gives 0, its limit.
__device__ __forceinline__ float silu_mul(float g, float u) {
    return __fmul_rn(__fdividef(g, 1.0f + __expf(-g)), u);
}

// One block of 128 is held by 128 / n lanes, 16 bytes of input each; a warp works on kUnroll x
// (32 n / 128) blocks at once, all loads first, so that enough bytes are in flight to fill the
// memory pipe.
template <class T, bool kGated>
__global__ void __launch_bounds__(kThreads)
    quantize_fp8_kernel(const T* __restrict__ x, uint32_t total, uint32_t KB, uint32_t K, int64_t ldx,
                        const int32_t* __restrict__ slots, int top_k, int64_t rows_out, uint8_t* __restrict__ q,
                        float* __restrict__ s) {
    constexpr int n = Vec16<T>::n, kLanes = kFp8Block / n, kGroups = 32 / kLanes;
    constexpr int kUnroll = kGated ? 2 : 4;
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    const uint32_t mask = kLanes == 32 ? 0xffffffffu : (0xffffu << (lane & 16));
    const uint64_t warp = (uint64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const uint64_t b0 = warp * (kUnroll * kGroups) + lane / kLanes;
    Vec16<T> v[kUnroll], up[kGated ? kUnroll : 1];
    uint32_t row[kUnroll], k0[kUnroll];
    bool in[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const uint64_t b = b0 + (uint64_t)i * kGroups;
        row[i] = (uint32_t)b / KB;
        k0[i] = ((uint32_t)b - row[i] * KB) * kFp8Block + sub * n;
        in[i] = b < total && k0[i] < K;
        v[i].u = make_uint4(0, 0, 0, 0);
        if (kGated) up[i].u = make_uint4(0, 0, 0, 0);
        if (in[i]) {
            const T* p = x + (int64_t)row[i] * ldx + k0[i];
            v[i].u = __ldcs(reinterpret_cast<const uint4*>(p));
            if (kGated) up[i].u = __ldcs(reinterpret_cast<const uint4*>(p + K));
        }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        float f[n];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            f[j] = to_float(v[i].t[j]);
            if (kGated) f[j] = silu_mul(f[j], to_float(up[i].t[j]));
            m = max(m, abs_bits(f[j]));
        }
        m = __reduce_max_sync(mask, m);
        float sc, r;
        scale_of(m, sc, r);
        uint32_t c[n / 4];
#pragma unroll
        for (int j = 0; j < n / 4; ++j)
            c[j] = pack4(__fmul_rn(f[4 * j], r), __fmul_rn(f[4 * j + 1], r), __fmul_rn(f[4 * j + 2], r),
                         __fmul_rn(f[4 * j + 3], r));
        if (!in[i]) continue;
        auto put = [&](int64_t d) {
            uint32_t* o = reinterpret_cast<uint32_t*>(q + d * K + k0[i]);
            if constexpr (n == 8) *reinterpret_cast<uint2*>(o) = make_uint2(c[0], c[n / 4 - 1]);
            else *o = c[0];
            if (sub == 0) s[d * KB + k0[i] / kFp8Block] = sc;
        };
        if (kGated || !slots) {
            put(row[i]);
        } else {
            for (int j = 0; j < top_k; ++j) {
                const int64_t d = __ldg(slots + (int64_t)row[i] * top_k + j);
                if (d >= 0 && d < rows_out) put(d);
            }
        }
    }
}

// One 128 x 128 block for a CTA: two sweeps over it (the second hits L2), offline.
template <class T>
__global__ void __launch_bounds__(kThreads)
    quantize_weight_fp8_kernel(const T* __restrict__ w, int64_t N, int64_t K, uint8_t* __restrict__ q,
                               float* __restrict__ s) {
    __shared__ uint32_t part[kThreads / 32];
    const int64_t k = (int64_t)blockIdx.x * kFp8Block + (threadIdx.x & 31) * 4;
    const int64_t n0 = (int64_t)blockIdx.y * kFp8Block;
    const int64_t base = (int64_t)blockIdx.z * N;
    const int rows = (int)min((int64_t)kFp8Block, N - n0), warp = threadIdx.x / 32;
    uint32_t m = 0;
    if (k < K)
        for (int r = warp; r < rows; r += kThreads / 32)
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max(m, abs_bits(to_float(w[(base + n0 + r) * K + k + j])));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, part[i]);
    float sc, r;
    scale_of(m, sc, r);
    if (k < K)
        for (int row = warp; row < rows; row += kThreads / 32) {
            const T* p = w + (base + n0 + row) * K + k;
            *reinterpret_cast<uint32_t*>(q + (base + n0 + row) * K + k) =
                pack4(__fmul_rn(to_float(p[0]), r), __fmul_rn(to_float(p[1]), r), __fmul_rn(to_float(p[2]), r),
                      __fmul_rn(to_float(p[3]), r));
        }
    if (threadIdx.x == 0) s[((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = sc;
}

template <class T, bool kGated>
cudaError_t launch(const void* x, int64_t M, int64_t K, int64_t ldx, const int32_t* slots, int top_k,
                   int64_t rows_out, uint8_t* q, float* s, cudaStream_t stream) {
    const int64_t KB = (K + kFp8Block - 1) / kFp8Block, total = M * KB;
    if (total >= (1LL << 31)) return cudaErrorNotSupported;
    constexpr int kPerCta = (kThreads / 32) * (kGated ? 2 : 4) * (32 * Vec16<T>::n / kFp8Block);
    const int64_t ctas = (total + kPerCta - 1) / kPerCta;
    quantize_fp8_kernel<T, kGated><<<(unsigned)ctas, kThreads, 0, stream>>>(
        static_cast<const T*>(x), (uint32_t)total, (uint32_t)KB, (uint32_t)K, ldx, slots, top_k, rows_out, q, s);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_fp8(const void* x, q8_float_type t, int64_t M, int64_t K, int64_t ldx,
                                const int32_t* slots, int top_k, int64_t rows_out, uint8_t* q, float* s,
                                cudaStream_t stream) {
    switch (t) {
        case Q8_F32: return launch<float, false>(x, M, K, ldx, slots, top_k, rows_out, q, s, stream);
        case Q8_BF16: return launch<__nv_bfloat16, false>(x, M, K, ldx, slots, top_k, rows_out, q, s, stream);
        default: return launch<__half, false>(x, M, K, ldx, slots, top_k, rows_out, q, s, stream);
    }
}

cudaError_t launch_swiglu_quantize_fp8(const void* h, q8_float_type t, int64_t M, int64_t I, int64_t ldh, uint8_t* q,
                                       float* s, cudaStream_t stream) {
    switch (t) {
        case Q8_F32: return launch<float, true>(h, M, I, ldh, nullptr, 0, M, q, s, stream);
        case Q8_BF16: return launch<__nv_bfloat16, true>(h, M, I, ldh, nullptr, 0, M, q, s, stream);
        default: return launch<__half, true>(h, M, I, ldh, nullptr, 0, M, q, s, stream);
    }
}

cudaError_t launch_quantize_weight_fp8(const void* w, q8_float_type t, int64_t E, int64_t N, int64_t K, uint8_t* q,
                                       float* s, cudaStream_t stream) {
    const int64_t KB = (K + kFp8Block - 1) / kFp8Block, NB = (N + kFp8Block - 1) / kFp8Block;
    if (KB >= (1LL << 31) || NB > 65535 || E > 65535) return cudaErrorNotSupported;
    const dim3 grid((unsigned)KB, (unsigned)NB, (unsigned)E);
    switch (t) {
        case Q8_F32:
            quantize_weight_fp8_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const float*>(w), N, K, q, s);
            break;
        case Q8_BF16:
            quantize_weight_fp8_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const __nv_bfloat16*>(w), N, K, q, s);
            break;
        default:
            quantize_weight_fp8_kernel<<<grid, kThreads, 0, stream>>>(static_cast<const __half*>(w), N, K, q, s);
    }
    note_launch();
    return cudaGetLastError();
}

}  // namespace q8
