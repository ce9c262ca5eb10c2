// Internal declarations of the float8 and routed-expert operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/q8.h"

namespace q8 {

constexpr int kFp8Block = 128;          // K elements (and weight rows) that share a scale
constexpr float kFp8Max = 448.0f;       // largest e4m3 value
constexpr float kFp8Tiny = 1e-30f;      // smallest block maximum a scale is made from: s and 1/s stay normal
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;
constexpr int kMaxGroups = 32;

cudaError_t launch_quantize_fp8(const void* x, q8_float_type t, int64_t M, int64_t K, int64_t ldx,
                                const int32_t* slots, int top_k, int64_t rows_out, uint8_t* q, float* s,
                                cudaStream_t stream);
cudaError_t launch_swiglu_quantize_fp8(const void* h, q8_float_type t, int64_t M, int64_t I, int64_t ldh, uint8_t* q,
                                       float* s, cudaStream_t stream);
cudaError_t launch_quantize_weight_fp8(const void* w, q8_float_type t, int64_t E, int64_t N, int64_t K, uint8_t* q,
                                       float* s, cudaStream_t stream);

struct RouteArgs {
    const void* logits;
    int64_t T, ldl;
    int E, k;
    bool softmax;
    const float* bias;
    int n_group, topk_group;
    bool renorm;
    float scale;
    int32_t* idx;
    float* w;
};
cudaError_t launch_moe_route(const RouteArgs& a, q8_float_type t, cudaStream_t stream);
cudaError_t launch_moe_plan(const int32_t* idx, int64_t n, int E, int32_t* offsets, int32_t* slots,
                            cudaStream_t stream);
cudaError_t launch_moe_combine(const void* h, q8_float_type t, int64_t rows, int64_t N, const int32_t* slots,
                               const float* w, int64_t T, int k, void* y, cudaStream_t stream);

// y[rows, N] = sum over K blocks of (sa sw) (qa . qw); offsets == nullptr: one matrix qw[N, K] for
// all rows; else rows offsets[e] .. offsets[e + 1] use qw[e] of qw[E, N, K].
cudaError_t launch_gemm_fp8(const uint8_t* qa, const float* sa, const uint8_t* qw, const float* sw,
                            const int32_t* offsets, int64_t rows, int E, int64_t N, int64_t K, void* y,
                            q8_float_type t, cudaStream_t stream);
cudaError_t read_and_clear_gemm_fp8_error(uint32_t* code);

#ifdef __CUDACC__
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// 16 bytes of T as floats.
template <class T>
struct Vec16 {
    static constexpr int n = 16 / sizeof(T);
    union {
        uint4 u;
        T t[n];
    };
    __device__ __forceinline__ Vec16() {}
};
__device__ __forceinline__ void to_floats(const Vec16<float>& v, float (&f)[4]) {
    f[0] = v.t[0];
    f[1] = v.t[1];
    f[2] = v.t[2];
    f[3] = v.t[3];
}
__device__ __forceinline__ void to_floats(const Vec16<__nv_bfloat16>& v, float (&f)[8]) {   // a shift or a mask each
    const uint32_t w[4] = {v.u.x, v.u.y, v.u.z, v.u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void to_floats(const Vec16<__half>& v, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 t = __half22float2(__halves2half2(v.t[2 * j], v.t[2 * j + 1]));
        f[2 * j] = t.x;
        f[2 * j + 1] = t.y;
    }
}
#endif

}  // namespace q8
