// Internal declarations of the 4-bit floating-point operators.
#pragma once

#include "q8_fp8.h"

namespace q8 {

constexpr int kFp4Span = 256;             // K of one stage of the products: 128 bytes of codes a row
constexpr float kFp4RowMax = 2688.0f;     // 6 * 448: a row's largest value in units of its scale (blocks of 16)

// Bytes of scales of a row: whole spans of 256 K.
inline int64_t fp4_pitch(int64_t K, int block) { return (K + kFp4Span - 1) / kFp4Span * (kFp4Span / block); }

cudaError_t launch_quantize_fp4(const void* x, q8_float_type t, int block, int64_t M, int64_t K, int64_t ldx,
                                const int32_t* slots, int top_k, int64_t rows_out, uint8_t* q, uint8_t* sf, float* s,
                                cudaStream_t stream);
cudaError_t launch_swiglu_quantize_fp4(const void* h, q8_float_type t, int block, int64_t M, int64_t I, int64_t ldh,
                                       uint8_t* q, uint8_t* sf, float* s, cudaStream_t stream);
cudaError_t launch_quantize_weight_fp4(const void* w, q8_float_type t, int block, int64_t E, int64_t N, int64_t K,
                                       uint8_t* q, uint8_t* sf, float* s, cudaStream_t stream);
// sf: nullptr (the codes' own values), rows of scales (tile_rows = 0), or tiles for matrices of tile_rows rows each. e4m3: the
// output type is float8 (type is ignored).
cudaError_t launch_dequantize_fp4(const uint8_t* q, const uint8_t* sf, const float* s, int block, int64_t rows, int64_t K,
                                  int64_t tile_rows, void* y, q8_float_type type, bool e4m3, cudaStream_t stream);

// y[rows, N] = sa[m] sw[n] sum over blocks of (sfa sfw) (qa . qw); offsets == nullptr: one matrix qw[N, K / 2] for all
// rows; else rows offsets[e] .. offsets[e + 1] use qw[e]. sa, sw: nullptr stands for ones.
struct Fp4Product {
    const uint8_t* qa;
    const uint8_t* sfa;
    const float* sa;
    const uint8_t* qw;
    const uint8_t* sfw;
    const float* sw;
    const int32_t* offsets;
    int64_t rows, E, N, K;
    void* y;
    q8_float_type type;
};
cudaError_t launch_gemm_fp4(const Fp4Product& p, int block, cudaStream_t stream);
cudaError_t read_and_clear_gemm_fp4_error(uint32_t* code);

}  // namespace q8
