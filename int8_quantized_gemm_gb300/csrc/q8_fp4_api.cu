// C ABI of the 4-bit floating-point operators: host-side argument validation. As in q8_api.cu, it runs before any CUDA call, so
// a rejected call enqueues nothing.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "q8_fp4.h"
#include "q8_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool valid_type(q8_float_type t) { return t == Q8_F32 || t == Q8_BF16 || t == Q8_F16; }
bool valid_block(int block) { return block == 16 || block == 32; }
int64_t size_of(q8_float_type t) { return t == Q8_F32 ? 4 : 2; }
cudaStream_t cu(q8_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

q8_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return Q8_OK;
    if (e == cudaErrorNotSupported) return Q8_ERR_UNSUPPORTED;
    return Q8_ERR_CUDA;
}

// Sizes up to 2^31 - 1 each and products of two below 2^62: no 64-bit index overflows.
bool in_range(int64_t v) { return v <= INT32_MAX; }

// Codes, block scales and (blocks of 16) row scales: all there and aligned.
bool codes_ok(const void* q, const void* sf, const void* s, int block) {
    return q && sf && aligned(q, 16) && aligned(sf, 16) && (block == 32 || (s && aligned(s, 4)));
}

q8_status check_rows(const void* x, q8_float_type t, int block, int64_t M, int64_t cols, int64_t K, int64_t ld,
                     const uint8_t* q, const uint8_t* sf, const float* s) {
    if (M < 0 || K < 0 || !valid_type(t) || !valid_block(block)) return Q8_ERR_INVALID_ARG;
    if (K % 32 != 0 || !in_range(M) || !in_range(cols)) return Q8_ERR_UNSUPPORTED;
    if (ld < cols || ld > (1LL << 40)) return Q8_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return Q8_OK;
    if (!x || !aligned(x, 16) || !codes_ok(q, sf, s, block)) return Q8_ERR_INVALID_ARG;
    if (ld * size_of(t) % 16 != 0) return Q8_ERR_UNSUPPORTED;
    return Q8_OK;
}

q8_status gemm_fp4(const q8::Fp4Product& p, int block, q8_stream_t stream) {
    if (p.rows < 0 || p.E < 0 || p.N < 0 || p.K < 0 || !valid_type(p.type) || !valid_block(block)) return Q8_ERR_INVALID_ARG;
    if (p.K % 32 != 0 || p.E > q8::kMaxExperts) return Q8_ERR_UNSUPPORTED;
    // The kernels count rows and K in 32 bits, and so are TMA's coordinates: the end of a tile that begins inside has to
    // be a number too (rows of a tile up to 256, and as many again of the tokens; 256 K of a stage).
    if (p.rows > INT32_MAX - 1024 || p.K > INT32_MAX - 2 * q8::kFp4Span) return Q8_ERR_UNSUPPORTED;
    if (!in_range(p.N) || (p.E > 0 && p.N > (INT32_MAX - 1024) / p.E)) return Q8_ERR_UNSUPPORTED;
    // So are the weights' tiles of scales, as rows of 128 bytes, 16 for each 128 weight rows and 256 K (two weight tiles
    // at a time).
    const int64_t NB = (p.N + 127) / 128, KB = (p.K + q8::kFp4Span - 1) / q8::kFp4Span;
    if (KB > 0 && p.E * NB + 2 > INT32_MAX / (16 * KB)) return Q8_ERR_UNSUPPORTED;
    if (p.rows == 0 || p.N == 0 || p.E == 0) return Q8_OK;
    if (!p.y || !aligned(p.y, 16)) return Q8_ERR_INVALID_ARG;
    if (p.K > 0) {
        if (!codes_ok(p.qa, p.sfa, nullptr, 32) || !codes_ok(p.qw, p.sfw, nullptr, 32)) return Q8_ERR_INVALID_ARG;
        if (!aligned(p.sa, 4) || !aligned(p.sw, 4)) return Q8_ERR_INVALID_ARG;
    }
    if (p.K == 0) {   // empty dot products: rows of no expert are not written, so only the dense form is filled
        if (p.offsets) return Q8_ERR_UNSUPPORTED;
        return from_cuda(cudaMemsetAsync(p.y, 0, (size_t)p.rows * (size_t)p.N * (size_t)size_of(p.type), cu(stream)));
    }
    return from_cuda(q8::launch_gemm_fp4(p, block, cu(stream)));
}

}  // namespace

extern "C" {

q8_status q8_quantize_fp4(const void* x, q8_float_type type, int block, int64_t M, int64_t K, int64_t ldx,
                          const int32_t* slots, int64_t top_k, int64_t rows_out, uint8_t* q, uint8_t* sf, float* s,
                          q8_stream_t stream) {
    q8_status st = check_rows(x, type, block, M, K, K, ldx, q, sf, s);
    if (st != Q8_OK) return st;
    if (slots || M == 0) {   // the slots of no row may have no address
        if (top_k < (slots ? 1 : 0) || rows_out < 0 || !aligned(slots, 4)) return Q8_ERR_INVALID_ARG;
        if (top_k > q8::kMaxTopK || !in_range(rows_out)) return Q8_ERR_UNSUPPORTED;
    } else if (top_k != 0 || rows_out != M) {
        return Q8_ERR_INVALID_ARG;
    }
    if (M == 0 || K == 0) return Q8_OK;
    return from_cuda(q8::launch_quantize_fp4(x, type, block, M, K, ldx, slots, (int)top_k, rows_out, q, sf, s, cu(stream)));
}

q8_status q8_swiglu_quantize_fp4(const void* h, q8_float_type type, int block, int64_t M, int64_t I, int64_t ldh, uint8_t* q,
                                 uint8_t* sf, float* s, q8_stream_t stream) {
    if (I < 0 || I > INT32_MAX) return I < 0 ? Q8_ERR_INVALID_ARG : Q8_ERR_UNSUPPORTED;
    q8_status st = check_rows(h, type, block, M, 2 * I, I, ldh, q, sf, s);
    if (st != Q8_OK) return st;
    if (M == 0 || I == 0) return Q8_OK;
    return from_cuda(q8::launch_swiglu_quantize_fp4(h, type, block, M, I, ldh, q, sf, s, cu(stream)));
}

q8_status q8_quantize_weight_fp4(const void* w, q8_float_type type, int block, int64_t E, int64_t N, int64_t K, uint8_t* qw,
                                 uint8_t* sfw, float* sw, q8_stream_t stream) {
    if (E < 0 || N < 0 || K < 0 || !valid_type(type) || !valid_block(block)) return Q8_ERR_INVALID_ARG;
    if (K % 32 != 0 || !in_range(E) || !in_range(N) || !in_range(K)) return Q8_ERR_UNSUPPORTED;
    if (E == 0 || N == 0 || K == 0) return Q8_OK;
    if (N > (1LL << 40) / E) return Q8_ERR_UNSUPPORTED;
    if (!w || !aligned(w, 16) || !codes_ok(qw, sfw, sw, block)) return Q8_ERR_INVALID_ARG;
    return from_cuda(q8::launch_quantize_weight_fp4(w, type, block, E, N, K, qw, sfw, sw, cu(stream)));
}

q8_status q8_dequantize_fp4(const uint8_t* q, const uint8_t* sf, const float* s, int block, int64_t rows, int64_t K,
                            int64_t tile_rows, void* y, q8_float_type type, q8_stream_t stream) {
    if (rows < 0 || K < 0 || tile_rows < 0 || !valid_block(block)) return Q8_ERR_INVALID_ARG;
    if (!valid_type(type) && type != Q8_E4M3) return Q8_ERR_INVALID_ARG;
    if (type == Q8_E4M3 && (sf || s)) return Q8_ERR_INVALID_ARG;
    if (tile_rows > 0 && rows % tile_rows != 0) return Q8_ERR_INVALID_ARG;
    if (K % 32 != 0 || !in_range(K) || rows > (1LL << 40) || !in_range(tile_rows)) return Q8_ERR_UNSUPPORTED;
    if (rows == 0 || K == 0) return Q8_OK;
    if (!q || !y || !aligned(q, 16) || !aligned(y, 16) || !aligned(s, 4)) return Q8_ERR_INVALID_ARG;
    return from_cuda(q8::launch_dequantize_fp4(q, sf, s, block, rows, K, sf ? tile_rows : 0, y, type, type == Q8_E4M3, cu(stream)));
}

q8_status q8_gemm_fp4(const uint8_t* qa, const uint8_t* sfa, const float* sa, const uint8_t* qw, const uint8_t* sfw,
                      const float* sw, int block, int64_t M, int64_t N, int64_t K, void* y, q8_float_type type,
                      q8_stream_t stream) {
    return gemm_fp4(q8::Fp4Product{qa, sfa, sa, qw, sfw, sw, nullptr, M, 1, N, K, y, type}, block, stream);
}

q8_status q8_gemm_fp4_grouped(const uint8_t* qa, const uint8_t* sfa, const float* sa, const uint8_t* qw, const uint8_t* sfw,
                              const float* sw, const int32_t* offsets, int block, int64_t rows, int64_t E, int64_t N,
                              int64_t K, void* y, q8_float_type type, q8_stream_t stream) {
    if (rows > 0 && E > 0 && N > 0 && (!offsets || !aligned(offsets, 4))) return Q8_ERR_INVALID_ARG;
    return gemm_fp4(q8::Fp4Product{qa, sfa, sa, qw, sfw, sw, offsets, rows, E, N, K, y, type}, block, stream);
}

}  // extern "C"
