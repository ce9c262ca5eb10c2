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

#ifdef __CUDACC__
// The kernels of these operators may start while the one before them on the stream still runs (programmatic stream
// serialization): each touches global memory only after depend_wait(), which returns once that kernel has completed and its
// writes can be seen, and then lets the next one start. What overlaps is the set-up and the launch (128x8192x8192 13.4 ->
// 12.5 us, 2050 rows of 32 experts 34.3 -> 32.8, called one after another). What they read may have been written while they
// were already there, so it is read by the loads of q8_loads.cuh.
__device__ __forceinline__ void depend_wait() {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}
// cluster: CTAs of a cluster, 0 where the kernel names them itself or has none.
template <class... KArgs, class... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, int smem, int cluster, cudaStream_t stream,
                             Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

}  // namespace q8
