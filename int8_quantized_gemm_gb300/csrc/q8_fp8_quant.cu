// Quantizers of the float8 (e4m3) operators: activations with one scale for each row and block of
// 128 along K (plain, scattered to expert slots, or of a gated activation), weights with one scale
// for each 128 x 128 block.
//
// Over a block: a = max(max |x|, 1e-30), s = a / 448, q = e4m3(x * (448 / a)), every operation
// rounded to nearest even in fp32 and the code rounded once to e4m3 (at most 448 (1 + 2^-22) before
// it, which rounds to 448). The maximum is taken over the bits of |x|, under which an infinity is
// larger than every number and a NaN larger than an infinity: a block that holds one gets the scale
// inf or NaN, and its codes times its scale are NaN, so that a broken value is not hidden.
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

// Four values as e4m3 codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Two fp32 values as one operand: the pair operations take one issue slot for two.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Two of u * g / (1 + exp(-g)) for |g| <= kGateFast. exp(-g) = 2^h e^-d with h = fl(-g log2 e) and d = g + h ln 2, which is
// under 2^-16, so that e^-d is 1 - d: without d the rounding of h would cost |g| half steps. Off by less than
// 2^-20 of the value: the fast exponential 2^-22, ln 2 in 24 bits times h 2^-22, 1 - d and the sum half a step each
// (2^-24), the fast reciprocal 2^-23, two products half a step each. (32768 x 2048 bf16: 53.7 us without d, 56.0 with it,
// 67.6 with fp32's own exponential for every gate.)
constexpr float kGateFast = 87.0f;   // the exponential and its reciprocal are normal numbers
__device__ __forceinline__ void silu_mul2(float& g0, float& g1, float u0, float u1) {
    const uint64_t g = pack2(g0, g1), one = pack2(1.0f, 1.0f);
    const uint64_t h = mul2(g, pack2(-1.4426950408889634f, -1.4426950408889634f));
    const uint64_t d = fma2(h, pack2(0.6931471805599453f, 0.6931471805599453f), g);
    float e0, e1, r0, r1;
    unpack2(h, e0, e1);
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e0) : "f"(e0));
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e1) : "f"(e1));
    unpack2(fma2(pack2(e0, e1), fma2(d, pack2(-1.0f, -1.0f), one), one), e0, e1);
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r0) : "f"(e0));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r1) : "f"(e1));
    unpack2(mul2(mul2(g, pack2(r0, r1)), pack2(u0, u1)), g0, g1);
}

// The same for any gate, from t = exp(-|g|), so that nothing overflows before the value does and the tail of a closed gate
// keeps its bits: u g / (1 + t) for g >= 0, u g t / (1 + t) below (the reciprocal is of a number between 1 and 2). Where t
// is subnormal (|g| > 87.3) two of its steps, 2^-148 |g u|, come on top.
__device__ __forceinline__ float silu_mul_far(float g, float u) {
    const float t = expf(-fabsf(g));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(1.0f + t));
    return (g < 0.0f ? g * t : g) * r * u;
}

// max(m, |a|, |b|), NaN if one is (its bits are then above those of inf).
__device__ __forceinline__ float max_abs(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

enum Form : int { kDense = 0, kGated = 1, kSlots = 2 };

// One block of 128 is held by 128 / n lanes, 16 bytes of input each; a warp works on kUnroll x
// (32 n / 128) blocks at once, all loads first, so that enough bytes are in flight to fill the
// memory pipe, and one lane of each block's does its two divisions. kDense, kGated: the blocks of all
// rows in order; kSlots: `wpr` warps for each row, which copies its blocks to the row's slots. kWhole:
// K is a multiple of 128, so that block b's codes are at 128 b and its scale at b.
// Bound by memory: 8192 x 16384 fp32 92 us on the device (98 us back to back, 6.9 TB/s); the gated form,
// 32768 x 2048 bf16, 56 us back to back (issue slots); 1037 x 4096 bf16 to 8 slots 10.5 us, 4.2 TB/s of
// mostly writes, launch and tail included.
template <class T, int kForm, bool kWhole>
__global__ void __launch_bounds__(kThreads, kForm == kGated ? 6 : 1)   // gated: 40 registers instead of 48, 56.0 us for 57.6
    quantize_fp8_kernel(const T* __restrict__ x, uint32_t total, uint32_t KB, uint32_t K, int64_t ldx, uint32_t wpr,
                        const int32_t* __restrict__ slots, int top_k, int64_t rows_out, uint8_t* __restrict__ q,
                        float* __restrict__ s) {
    constexpr int n = Vec16<T>::n, kLanes = kFp8Block / n, kGroups = 32 / kLanes;
    constexpr int kUnroll = kForm == kGated ? 2 : 4;
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    const uint32_t mask = kLanes == 32 ? 0xffffffffu : (0xffffu << (lane & 16));
    const uint32_t warp = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    // first block, and its row and place in the row
    uint64_t b0;
    uint32_t row, kb;
    if constexpr (kForm == kSlots) {
        row = warp / wpr;
        kb = (warp - row * wpr) * (kUnroll * kGroups) + lane / kLanes;
        b0 = (uint64_t)row * KB + kb;
    } else {
        b0 = (uint64_t)warp * (kUnroll * kGroups) + lane / kLanes;
        const uint32_t b = b0 < total ? (uint32_t)b0 : 0;
        row = b / KB;
        kb = b - row * KB;
    }
    const uint32_t row0 = row;
    Vec16<T> v[kUnroll], up[kForm == kGated ? kUnroll : 1];
    uint32_t rows[kUnroll], k0[kUnroll];   // not kWhole: where block i goes
    bool in[kUnroll];
    const T* from = x + b0 * kFp8Block + sub * n;   // kWhole: block b of row r is at 128 b + r (ldx - K)
    const int64_t skip = ldx - K;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        in[i] = b0 + i * kGroups < total;
        if (kForm == kSlots) in[i] = in[i] && kb < KB;
        const T* p;
        if constexpr (kWhole) {
            p = from + i * (kGroups * kFp8Block) + row * skip;
        } else {
            rows[i] = row;
            k0[i] = kb * kFp8Block + sub * n;
            in[i] = in[i] && k0[i] < K;
            p = x + row * ldx + k0[i];
        }
        v[i].u = make_uint4(0, 0, 0, 0);
        if (kForm == kGated) up[i].u = make_uint4(0, 0, 0, 0);
        if (in[i]) {
            v[i].u = __ldcs(reinterpret_cast<const uint4*>(p));
            if (kForm == kGated) up[i].u = __ldcs(reinterpret_cast<const uint4*>(p + K));
        }
        kb += kGroups;
        if (kForm != kSlots)
#pragma unroll
            for (int g = 0; g < kGroups; ++g)   // kGroups blocks on are at most kGroups rows on
                if (kb >= KB) { kb -= KB; ++row; }
    }
    float f[kUnroll][n];
    uint32_t m[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        float most = 0.0f;
        to_floats(v[i], f[i]);
        if constexpr (kForm == kGated) {
            float by[n], far = 0.0f;
            to_floats(up[i], by);
#pragma unroll
            for (int j = 0; j < n; j += 2) far = max_abs(far, f[i][j], f[i][j + 1]);
            if (far <= kGateFast) {
#pragma unroll
                for (int j = 0; j < n; j += 2) silu_mul2(f[i][j], f[i][j + 1], by[j], by[j + 1]);
            } else {   // some gate of the lane's is far out, infinite or NaN: rare
#pragma unroll
                for (int j = 0; j < n; ++j) f[i][j] = silu_mul_far(f[i][j], by[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < n; j += 2) most = max_abs(most, f[i][j], f[i][j + 1]);
        m[i] = __reduce_max_sync(mask, __float_as_uint(most));
    }
    // lane i of a block's lanes divides for block i
    uint32_t own = m[0];
#pragma unroll
    for (int i = 1; i < kUnroll; ++i) own = (sub & (kUnroll - 1)) == i ? m[i] : own;
    float own_s, own_r;
    scale_of(own, own_s, own_r);
    float sc[kUnroll];
    uint32_t c[kUnroll][n / 4];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        sc[i] = __shfl_sync(0xffffffffu, own_s, i, kLanes);
        const float r = __shfl_sync(0xffffffffu, own_r, i, kLanes);
#pragma unroll
        for (int j = 0; j < n / 4; ++j) {
            float a, b, d, e;
            unpack2(mul2(pack2(f[i][4 * j], f[i][4 * j + 1]), pack2(r, r)), a, b);
            unpack2(mul2(pack2(f[i][4 * j + 2], f[i][4 * j + 3]), pack2(r, r)), d, e);
            c[i][j] = pack4(a, b, d, e);
        }
    }
    auto put = [&](uint8_t* to, float* scale, int i) {
        if (!in[i]) return;
        if constexpr (n == 8) *reinterpret_cast<uint2*>(to) = make_uint2(c[i][0], c[i][n / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(to) = c[i][0];
        if (sub == 0) *scale = sc[i];
    };
    if constexpr (kForm == kSlots) {
        int to = -1;
        if (b0 - lane / kLanes < total && lane < top_k) to = __ldg(slots + (int64_t)row0 * top_k + lane);
        if (to >= rows_out) to = -1;
        const uint32_t first = (uint32_t)(b0 - (uint64_t)row0 * KB);
        for (int j = 0; j < top_k; ++j) {
            const int64_t d = __shfl_sync(0xffffffffu, to, j);
            if (d < 0) continue;
            uint8_t* qd = q + d * K + first * kFp8Block + sub * n;
            float* sd = s + d * KB + first;
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) put(qd + i * (kGroups * kFp8Block), sd + i * kGroups, i);
        }
    } else if constexpr (kWhole) {
        uint8_t* qd = q + b0 * kFp8Block + sub * n;
        float* sd = s + b0;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) put(qd + i * (kGroups * kFp8Block), sd + i * kGroups, i);
    } else {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            put(q + (uint64_t)rows[i] * K + k0[i], s + (uint64_t)rows[i] * KB + k0[i] / kFp8Block, i);
    }
}

// One 128 x 128 block for a CTA: two sweeps over it (the second hits L2), offline, so with loads of single values: 0.65 of
// the measured copy bandwidth (64 x 4096 x 4096 bf16 733 us, floor 475; 8192 x 16384 fp32 145 us, floor 99).
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

template <class T, int kForm>
cudaError_t launch(const void* x, int64_t M, int64_t K, int64_t ldx, const int32_t* slots, int top_k,
                   int64_t rows_out, uint8_t* q, float* s, cudaStream_t stream) {
    const int64_t KB = (K + kFp8Block - 1) / kFp8Block, total = M * KB;
    if (total >= (1LL << 31)) return cudaErrorNotSupported;
    constexpr int kPerWarp = (kForm == kGated ? 2 : 4) * (32 * Vec16<T>::n / kFp8Block);
    const int64_t wpr = (KB + kPerWarp - 1) / kPerWarp;
    const int64_t warps = kForm == kSlots ? M * wpr : (total + kPerWarp - 1) / kPerWarp;
    const int64_t ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
    auto* kernel = K % kFp8Block == 0 ? quantize_fp8_kernel<T, kForm, true> : quantize_fp8_kernel<T, kForm, false>;
    kernel<<<(unsigned)ctas, kThreads, 0, stream>>>(static_cast<const T*>(x), (uint32_t)total, (uint32_t)KB, (uint32_t)K,
                                                    ldx, (uint32_t)wpr, slots, top_k, rows_out, q, s);
    note_launch();
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_plain(const void* x, int64_t M, int64_t K, int64_t ldx, const int32_t* slots, int top_k,
                         int64_t rows_out, uint8_t* q, float* s, cudaStream_t stream) {
    return slots ? launch<T, kSlots>(x, M, K, ldx, slots, top_k, rows_out, q, s, stream)
                 : launch<T, kDense>(x, M, K, ldx, nullptr, 0, M, q, s, stream);
}

}  // namespace

cudaError_t launch_quantize_fp8(const void* x, q8_float_type t, int64_t M, int64_t K, int64_t ldx,
                                const int32_t* slots, int top_k, int64_t rows_out, uint8_t* q, float* s,
                                cudaStream_t stream) {
    switch (t) {
        case Q8_F32: return launch_plain<float>(x, M, K, ldx, slots, top_k, rows_out, q, s, stream);
        case Q8_BF16: return launch_plain<__nv_bfloat16>(x, M, K, ldx, slots, top_k, rows_out, q, s, stream);
        default: return launch_plain<__half>(x, M, K, ldx, slots, top_k, rows_out, q, s, stream);
    }
}

cudaError_t launch_swiglu_quantize_fp8(const void* h, q8_float_type t, int64_t M, int64_t I, int64_t ldh, uint8_t* q,
                                       float* s, cudaStream_t stream) {
    switch (t) {
        case Q8_F32: return launch<float, kGated>(h, M, I, ldh, nullptr, 0, M, q, s, stream);
        case Q8_BF16: return launch<__nv_bfloat16, kGated>(h, M, I, ldh, nullptr, 0, M, q, s, stream);
        default: return launch<__half, kGated>(h, M, I, ldh, nullptr, 0, M, q, s, stream);
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
