// C ABI of the float8 and routed-expert operators: host-side argument validation. As in q8_api.cu,
// it runs before any CUDA call, so a rejected call enqueues nothing.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "q8_fp8.h"
#include "q8_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool valid_type(q8_float_type t) { return t == Q8_F32 || t == Q8_BF16 || t == Q8_F16; }
int64_t size_of(q8_float_type t) { return t == Q8_F32 ? 4 : 2; }
cudaStream_t cu(q8_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

q8_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return Q8_OK;
    if (e == cudaErrorNotSupported) return Q8_ERR_UNSUPPORTED;
    return Q8_ERR_CUDA;
}

// Sizes up to 2^31 - 1 each and products of two below 2^62: no 64-bit index overflows.
bool in_range(int64_t v) { return v <= INT32_MAX; }

q8_status check_rows(const void* x, q8_float_type t, int64_t M, int64_t cols, int64_t K, int64_t ld,
                     const uint8_t* q, const float* s) {
    if (M < 0 || K < 0 || !valid_type(t)) return Q8_ERR_INVALID_ARG;
    if (K % 16 != 0 || !in_range(M) || !in_range(cols)) return Q8_ERR_UNSUPPORTED;
    if (ld < cols || ld > (1LL << 40)) return Q8_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return Q8_OK;
    if (!x || !q || !s || !aligned(x, 16) || !aligned(q, 16) || !aligned(s, 4)) return Q8_ERR_INVALID_ARG;
    if (ld * size_of(t) % 16 != 0) return Q8_ERR_UNSUPPORTED;
    return Q8_OK;
}

q8_status gemm_fp8(const uint8_t* qa, const float* sa, const uint8_t* qw, const float* sw, const int32_t* offsets,
                   int64_t rows, int64_t E, int64_t N, int64_t K, void* y, q8_float_type t, q8_stream_t stream) {
    if (rows < 0 || E < 0 || N < 0 || K < 0 || !valid_type(t)) return Q8_ERR_INVALID_ARG;
    if (K % 16 != 0 || E > q8::kMaxExperts) return Q8_ERR_UNSUPPORTED;
    // The kernels count rows and K in 32 bits, and so are TMA's coordinates: the end of a tile that begins inside has to
    // be a number too (rows of a tile up to 256, and as many again of the tokens; 128 K of a block).
    if (rows > INT32_MAX - 1024 || K > INT32_MAX - q8::kFp8Block) return Q8_ERR_UNSUPPORTED;
    if (!in_range(N) || (E > 0 && N > (INT32_MAX - 1024) / E)) return Q8_ERR_UNSUPPORTED;
    if (rows == 0 || N == 0 || E == 0) return Q8_OK;
    if (!y || !aligned(y, 16)) return Q8_ERR_INVALID_ARG;
    if (K > 0) {
        if (!qa || !sa || !qw || !sw) return Q8_ERR_INVALID_ARG;
        if (!aligned(qa, 16) || !aligned(qw, 16) || !aligned(sa, 4) || !aligned(sw, 4)) return Q8_ERR_INVALID_ARG;
    }
    if (K == 0) {   // empty dot products: rows of no expert are not written, so only the dense form is filled
        if (offsets) return Q8_ERR_UNSUPPORTED;
        return from_cuda(cudaMemsetAsync(y, 0, (size_t)rows * (size_t)N * (size_t)size_of(t), cu(stream)));
    }
    return from_cuda(q8::launch_gemm_fp8(qa, sa, qw, sw, offsets, rows, (int)E, N, K, y, t, cu(stream)));
}

}  // namespace

extern "C" {

q8_status q8_quantize_fp8(const void* x, q8_float_type type, int64_t M, int64_t K, int64_t ldx, const int32_t* slots,
                          int64_t top_k, int64_t rows_out, uint8_t* q, float* s, q8_stream_t stream) {
    q8_status st = check_rows(x, type, M, K, K, ldx, q, s);
    if (st != Q8_OK) return st;
    if (slots || M == 0) {   // the slots of no row may have no address
        if (top_k < (slots ? 1 : 0) || rows_out < 0 || !aligned(slots, 4)) return Q8_ERR_INVALID_ARG;
        if (top_k > q8::kMaxTopK || !in_range(rows_out)) return Q8_ERR_UNSUPPORTED;
    } else if (top_k != 0 || rows_out != M) {
        return Q8_ERR_INVALID_ARG;
    }
    if (M == 0 || K == 0) return Q8_OK;
    return from_cuda(q8::launch_quantize_fp8(x, type, M, K, ldx, slots, (int)top_k, rows_out, q, s, cu(stream)));
}

q8_status q8_swiglu_quantize_fp8(const void* h, q8_float_type type, int64_t M, int64_t I, int64_t ldh, uint8_t* q,
                                 float* s, q8_stream_t stream) {
    if (I < 0 || I > INT32_MAX) return I < 0 ? Q8_ERR_INVALID_ARG : Q8_ERR_UNSUPPORTED;
    q8_status st = check_rows(h, type, M, 2 * I, I, ldh, q, s);
    if (st != Q8_OK) return st;
    if (M == 0 || I == 0) return Q8_OK;
    return from_cuda(q8::launch_swiglu_quantize_fp8(h, type, M, I, ldh, q, s, cu(stream)));
}

q8_status q8_quantize_weight_fp8(const void* w, q8_float_type type, int64_t E, int64_t N, int64_t K, uint8_t* qw,
                                 float* sw, q8_stream_t stream) {
    if (E < 0 || N < 0 || K < 0 || !valid_type(type)) return Q8_ERR_INVALID_ARG;
    if (K % 16 != 0 || !in_range(E) || !in_range(N) || !in_range(K)) return Q8_ERR_UNSUPPORTED;
    if (E == 0 || N == 0 || K == 0) return Q8_OK;
    if (!w || !qw || !sw || !aligned(w, 16) || !aligned(qw, 16) || !aligned(sw, 4)) return Q8_ERR_INVALID_ARG;
    return from_cuda(q8::launch_quantize_weight_fp8(w, type, E, N, K, qw, sw, cu(stream)));
}

q8_status q8_gemm_fp8(const uint8_t* qa, const float* sa, const uint8_t* qw, const float* sw, int64_t M, int64_t N,
                      int64_t K, void* y, q8_float_type type, q8_stream_t stream) {
    return gemm_fp8(qa, sa, qw, sw, nullptr, M, 1, N, K, y, type, stream);
}

q8_status q8_gemm_fp8_grouped(const uint8_t* qa, const float* sa, const uint8_t* qw, const float* sw,
                              const int32_t* offsets, int64_t rows, int64_t E, int64_t N, int64_t K, void* y,
                              q8_float_type type, q8_stream_t stream) {
    if (rows > 0 && E > 0 && N > 0 && (!offsets || !aligned(offsets, 4))) return Q8_ERR_INVALID_ARG;
    return gemm_fp8(qa, sa, qw, sw, offsets, rows, E, N, K, y, type, stream);
}

q8_status q8_moe_route(const void* logits, q8_float_type type, int64_t T, int64_t E, int64_t ldl, int64_t top_k,
                       q8_score score, const float* bias, int64_t n_group, int64_t topk_group, int renorm,
                       float scale, int32_t* idx, float* weights, q8_stream_t stream) {
    if (T < 0 || E < 1 || !valid_type(type) || (score != Q8_SOFTMAX && score != Q8_SIGMOID)) return Q8_ERR_INVALID_ARG;
    if (top_k < 1 || top_k > E || n_group < 1 || topk_group < 1 || topk_group > n_group || E % n_group != 0)
        return Q8_ERR_INVALID_ARG;
    if (ldl < E || ldl > (1LL << 40) || !isfinite(scale)) return Q8_ERR_INVALID_ARG;
    if (E > q8::kMaxExperts || top_k > q8::kMaxTopK || n_group > q8::kMaxGroups || !in_range(T))
        return Q8_ERR_UNSUPPORTED;
    if (T == 0) return Q8_OK;
    if (!logits || !idx || !weights || !aligned(logits, (uintptr_t)size_of(type)) || !aligned(idx, 4) ||
        !aligned(weights, 4) || (bias && !aligned(bias, 4)))
        return Q8_ERR_INVALID_ARG;
    const q8::RouteArgs a{logits, T, ldl, (int)E, (int)top_k, score == Q8_SOFTMAX, bias, (int)n_group,
                          (int)topk_group, renorm != 0, scale, idx, weights};
    return from_cuda(q8::launch_moe_route(a, type, cu(stream)));
}

q8_status q8_moe_plan(const int32_t* idx, int64_t T, int64_t top_k, int64_t E, int32_t* offsets, int32_t* slots,
                      q8_stream_t stream) {
    if (T < 0 || top_k < 1 || E < 1 || !offsets || !aligned(offsets, 4)) return Q8_ERR_INVALID_ARG;
    if (E > q8::kMaxExperts || top_k > q8::kMaxTopK || T > INT32_MAX / top_k) return Q8_ERR_UNSUPPORTED;
    if (T > 0 && (!idx || !slots || !aligned(idx, 4) || !aligned(slots, 4))) return Q8_ERR_INVALID_ARG;
    return from_cuda(q8::launch_moe_plan(idx, T * top_k, (int)E, offsets, slots, cu(stream)));
}

q8_status q8_moe_combine(const void* h, q8_float_type type, int64_t rows, int64_t N, const int32_t* slots,
                         const float* weights, int64_t T, int64_t top_k, void* y, q8_stream_t stream) {
    if (rows < 0 || N < 0 || T < 0 || top_k < 1 || !valid_type(type)) return Q8_ERR_INVALID_ARG;
    if (!in_range(rows) || !in_range(N) || !in_range(T) || top_k > q8::kMaxTopK) return Q8_ERR_UNSUPPORTED;
    if (N * size_of(type) % 16 != 0) return Q8_ERR_UNSUPPORTED;
    if (T == 0 || N == 0) return Q8_OK;
    if ((rows > 0 && !h) || !slots || !weights || !y || !aligned(h, 16) || !aligned(y, 16) || !aligned(slots, 4) ||
        !aligned(weights, 4))
        return Q8_ERR_INVALID_ARG;
    return from_cuda(q8::launch_moe_combine(h, type, rows, N, slots, weights, T, (int)top_k, y, cu(stream)));
}

}  // extern "C"
