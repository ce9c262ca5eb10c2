// Quantizers of the 4-bit floating-point (e2m1) operators, and the way back.
//
// Blocks of 16 K: every row has an fp32 scale s and every block an e4m3 one. With a the row's and b the block's largest
// magnitude, A = max(a, 1e-30):
//   s = A / 2688,  c = e4m3(b * (448 / A)),  q = e2m1(x * ((2688 / A) / c)), 0 where c is 0,
// so that x is about q c s. Blocks of 32 K: c = 2^e, the smallest power of two with b <= 6 c (e >= -127), q = e2m1(x / c), no
// s. Every operation is rounded to nearest even in fp32, scales and codes once to their type. A NaN or an infinity makes the
// row's s NaN (the block's c, for blocks of 32), so that a broken value is not hidden.
#include "q8_fp4.h"
#include "q8_internal.h"
#include "q8_loads.cuh"
#include "q8_silu.cuh"

namespace q8 {
namespace {

enum Form : int { kDense = 0, kGated = 1, kSlots = 2, kTiles = 3 };

constexpr int kMaxThreads = 512;

// 32 bytes of T as floats.
template <class T>
struct Vec32 {
    static constexpr int n = 32 / sizeof(T);
    uint32_t w[8];
    // `wide`: the address is a multiple of 32 bytes
    __device__ __forceinline__ void load(const T* p, bool wide) {
        if (wide) {
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                         : "l"(p)
                         : "memory");
        } else {
            const uint4 a = load128(p), b = load128(reinterpret_cast<const uint4*>(p) + 1);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0;
    }
};
__device__ __forceinline__ void to_floats(const Vec32<float>& v, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v.w[j]);
}
__device__ __forceinline__ void to_floats(const Vec32<__nv_bfloat16>& v, float (&f)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        f[2 * j] = __uint_as_float(v.w[j] << 16);
        f[2 * j + 1] = __uint_as_float(v.w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void to_floats(const Vec32<__half>& v, float (&f)[16]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&v.w[j]));
        f[2 * j] = t.x;
        f[2 * j + 1] = t.y;
    }
}

// Eight values times r as e2m1 codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t codes8(const float* f, float r) {
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) unpack2(mul2(pack2(f[j], f[j + 1]), pack2(r, r)), t[j], t[j + 1]);
    uint32_t c;
    asm("{\n.reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(c)
        : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
    return c;
}

__device__ __forceinline__ uint32_t e4m3_of(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xffu;
}
__device__ __forceinline__ float of_e4m3(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)c));
    return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// The scale byte of a block with the largest magnitude b, and what its values are multiplied by. Blocks of 32: b = m 2^k is at
// most 6 2^e = 1.5 2^(e + 2) for e = k - 2 if m <= 1.5 and for k - 1 otherwise; 2^-e is an fp32 number, and the product exact.
__device__ __forceinline__ void scale16(float b, float r448, float r2688, uint32_t& c, float& up) {
    c = e4m3_of(__fmul_rn(b, r448));
    const float f = of_e4m3(c);
    up = f > 0.0f ? __fdiv_rn(r2688, f) : 0.0f;
}
__device__ __forceinline__ void scale32(float b, uint32_t& c, float& up) {
    const uint32_t bits = __float_as_uint(b);
    const int e = (int)(bits >> 23) - ((bits & 0x7fffffu) <= 0x400000u ? 2 : 1);
    c = bits >= 0x7f800000u ? 255u : (uint32_t)max(e, 0);
    up = __uint_as_float(bits >= 0x7f800000u ? 0u : (254u - c) << 23);
}

struct Args {
    const void* x;
    uint32_t K, vecs;          // vecs: vectors of 32 bytes in a row
    int64_t ldx, M;            // rows
    uint32_t N;                // kTiles: rows of a matrix
    const int32_t* slots;
    int top_k;
    int64_t rows_out;
    uint8_t* q;
    uint8_t* sf;
    uint32_t pitch;            // bytes of scales of a row
    float* s;
};

// A row is held by blockDim.x threads, kUnroll vectors of 32 bytes each, all loads first; blockDim.y rows a CTA, some in a
// warp where they are short. Blocks of 16 need the row's maximum before the first code: rows of up to 512 threads' vectors
// (32768 elements of 16 bits, 16384 of 32) stay in registers, as they were read; longer ones are read a second time, from L2.
// The gated form holds the activation instead, of rows of up to 16384 elements for 16-bit h and 4096 for fp32; longer ones are
// read and activated twice.
// Bound by memory. On the device, of the measured copy bandwidth: 8192 x 16384 fp32 91 us (0.99), bf16 51.5 (0.98; two
// vectors a thread 66); 16384 x 4096 bf16 26.8 (0.95); the gated form, 32768 x 2048 bf16, 47.4 (0.95) with CTAs of 64 threads
// (48.0 with 128, 49.5 with 256) and two vectors a thread (one 58); its fp32 form keeps one (42.6 us for 16384 x 2048, two
// 47, four 73: registers). Blocks of 32, which need no maximum of the row: 85 us and 49 for the first two. Weights, whose scales are
// single bytes 16 apart in their tiles: 97.6 us fp32, 55.5 bf16 (0.92 and 0.91).
template <class T, int kForm>
struct Unroll { static constexpr int n = kForm == kGated ? (sizeof(T) == 4 ? 1 : 2) : 4; };

template <class T, int kForm, int kBlock>
__global__ void __launch_bounds__(kMaxThreads) quantize_fp4_kernel(const Args p, bool wide) {
    constexpr int n = Vec32<T>::n, kLanes = kBlock / n;      // lanes that share a block: 1, 2 or 4
    constexpr int kUnroll = Unroll<T, kForm>::n;
    __shared__ uint32_t part[kMaxThreads / 32];
    depend_wait();
    const uint32_t tx = threadIdx.x;
    const int width = blockDim.x < 32 ? (int)blockDim.x : 32;     // lanes of a row in a warp: a power of two
    const uint32_t lane = tx & 31;                                // within the row's lanes
    const int64_t slot_row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    // kTiles: rows in tiles of 128 of each matrix, past its end too (their scales are zero)
    int64_t row = slot_row;
    bool live = row < p.M;
    uint32_t nrow = 0;
    if constexpr (kForm == kTiles) {
        const uint32_t padded = (p.N + 127) & ~127u;
        const int64_t e = slot_row / padded;
        nrow = (uint32_t)(slot_row - e * padded);
        row = e * p.N + nrow;
        live = nrow < p.N && row < p.M;
    }
    const T* x = static_cast<const T*>(p.x) + (live ? row : 0) * p.ldx;
    const uint32_t chunk = blockDim.x * kUnroll;

    Vec32<T> v[kUnroll];                                          // as they were read,
    float g[kForm == kGated ? kUnroll : 1][n];                    // or the activation
    auto load = [&](uint32_t v0) {
        Vec32<T> u[kForm == kGated ? kUnroll : 1];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const uint32_t at = v0 + i * blockDim.x + tx;
            if (live && at < p.vecs) {
                v[i].load(x + (size_t)at * n, wide);
                if constexpr (kForm == kGated) u[i].load(x + p.K + (size_t)at * n, wide);
            } else {
                v[i].zero();
                if constexpr (kForm == kGated) u[i].zero();
            }
        }
        if constexpr (kForm == kGated) {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                float by[n], far = 0.0f;
                to_floats(v[i], g[i]);
                to_floats(u[i], by);
#pragma unroll
                for (int j = 0; j < n; j += 2) far = max_abs(far, g[i][j], g[i][j + 1]);
                if (far <= kGateFast) {
#pragma unroll
                    for (int j = 0; j < n; j += 2) silu_mul2(g[i][j], g[i][j + 1], by[j], by[j + 1]);
                } else {   // some gate of the thread's is far out, infinite or NaN: rare
#pragma unroll
                    for (int j = 0; j < n; ++j) g[i][j] = silu_mul_far(g[i][j], by[j]);
                }
            }
        }
    };
    auto values = [&](int i, float (&f)[n]) {
        if constexpr (kForm == kGated) {
#pragma unroll
            for (int j = 0; j < n; ++j) f[j] = g[i][j];
        } else {
            to_floats(v[i], f);
        }
    };
    float most[kUnroll];   // of a thread's vector, then of its block
    auto maxima = [&]() {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            float f[n];
            values(i, f);
            most[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < n; j += 2) most[i] = max_abs(most[i], f[j], f[j + 1]);
        }
    };

    float r448 = 0.0f, r2688 = 0.0f, s = 0.0f;
    if constexpr (kBlock == 16) {
        float top = 0.0f;
        for (uint32_t v0 = 0; v0 < p.vecs; v0 += chunk) {
            load(v0);
            maxima();
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) top = max_abs(top, most[i], 0.0f);
        }
        uint32_t m = __float_as_uint(top);
        if (blockDim.x < 32) {
            for (int d = 1; d < width; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        } else {
            m = __reduce_max_sync(0xffffffffu, m);
            if (blockDim.x > 32) {
                const uint32_t warps = blockDim.x / 32;
                uint32_t* own = part + threadIdx.y * warps;
                if (lane == 0) own[tx / 32] = m;
                __syncthreads();
                m = lane < warps ? own[lane] : 0;
                m = __reduce_max_sync(0xffffffffu, m);
            }
        }
        float a = __uint_as_float(m >= 0x7f800000u ? 0x7fffffffu : m);
        a = a < kFp8Tiny ? kFp8Tiny : a;   // a NaN stays
        const float d = __fdiv_rn(lane == 0 ? a : lane == 1 ? kFp8Max : kFp4RowMax, lane == 0 ? kFp4RowMax : a);
        s = __shfl_sync(0xffffffffu, d, 0, width);
        r448 = __shfl_sync(0xffffffffu, d, 1, width);
        r2688 = __shfl_sync(0xffffffffu, d, 2, width);
    }

    int to = -1;           // kSlots: lane j has the row's slot j
    if constexpr (kForm == kSlots) {
        if (live && (int)lane < p.top_k) to = load_int(p.slots + row * p.top_k + lane);
        if (to >= p.rows_out) to = -1;
    }
    const bool once = kBlock == 16 && p.vecs <= chunk;
    for (uint32_t v0 = 0; v0 < p.vecs; v0 += chunk) {
        if (!once) {
            load(v0);
            maxima();
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const uint32_t at = v0 + i * blockDim.x + tx;
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) {
                const float o = __shfl_xor_sync(0xffffffffu, most[i], d);
                most[i] = max_abs(most[i], o, 0.0f);
            }
            uint32_t c;
            float up, f[n];
            if constexpr (kBlock == 16) scale16(most[i], r448, r2688, c, up);
            else scale32(most[i], c, up);
            values(i, f);
            uint32_t code[n / 8];
#pragma unroll
            for (int j = 0; j < n / 8; ++j) code[j] = codes8(f + 8 * j, up);
            auto put = [&](int64_t dst) {
                uint8_t* qd = p.q + (size_t)dst * (p.K / 2) + (size_t)at * (n / 2);
                if constexpr (n == 16) *reinterpret_cast<uint2*>(qd) = make_uint2(code[0], code[n / 8 - 1]);
                else *reinterpret_cast<uint32_t*>(qd) = code[0];
            };
            const uint32_t g = at / kLanes;      // its block
            const bool in = live && at < p.vecs;
            if constexpr (kForm == kSlots) {
                for (int j = 0; j < p.top_k; ++j) {
                    const int64_t dst = __shfl_sync(0xffffffffu, to, j);
                    if (dst < 0 || !in) continue;
                    put(dst);
                    if (at % kLanes == 0) p.sf[(size_t)dst * p.pitch + g] = (uint8_t)c;
                }
            } else if (in) {
                put(row);
                if (at % kLanes == 0) {
                    if constexpr (kForm == kTiles)
                        p.sf[((size_t)(slot_row >> 7) * (p.pitch / 4) + g / 4) * 512 + (nrow & 31) * 16 + ((nrow >> 5) & 3) * 4 +
                             g % 4] = (uint8_t)c;
                    else
                        p.sf[(size_t)row * p.pitch + g] = (uint8_t)c;
                }
            }
        }
    }
    // the rest of the row's scales, and its own
    const uint32_t have = p.K / kBlock;
    if constexpr (kForm == kSlots) {
        for (int j = 0; j < p.top_k; ++j) {
            const int64_t dst = __shfl_sync(0xffffffffu, to, j);
            if (dst < 0) continue;
            for (uint32_t g = have + tx; g < p.pitch; g += blockDim.x) p.sf[(size_t)dst * p.pitch + g] = 0;
            if (kBlock == 16 && tx == 0) p.s[dst] = s;
        }
    } else if constexpr (kForm == kTiles) {
        if (slot_row < p.rows_out)     // the padded rows of all matrices
            for (uint32_t g = (live ? have : 0) + tx; g < p.pitch; g += blockDim.x)
                p.sf[((size_t)(slot_row >> 7) * (p.pitch / 4) + g / 4) * 512 + (nrow & 31) * 16 + ((nrow >> 5) & 3) * 4 +
                     g % 4] = 0;
        if (kBlock == 16 && live && tx == 0) p.s[row] = s;
    } else if (live) {
        for (uint32_t g = have + tx; g < p.pitch; g += blockDim.x) p.sf[(size_t)row * p.pitch + g] = 0;
        if (kBlock == 16 && tx == 0) p.s[row] = s;
    }
}

template <class T, int kForm>
cudaError_t launch(Args a, int block, cudaStream_t stream) {
    constexpr int n = Vec32<T>::n, kUnroll = Unroll<T, kForm>::n;
    a.vecs = a.K / n;
    const int64_t rows = kForm == kTiles ? a.rows_out : a.M;
    const uint32_t want = (a.vecs + kUnroll - 1) / kUnroll;
    uint32_t tx = (want + 31) / 32 * 32;
    if (kForm != kSlots && want <= 16) tx = want <= 4 ? 4 : want <= 8 ? 8 : 16;   // several rows a warp; the slots take all of it
    if (tx > kMaxThreads) tx = kMaxThreads;
    const uint32_t ty = tx >= 64 ? 1 : 64 / tx;
    const int64_t ctas = (rows + ty - 1) / ty;
    if (ctas >= (1LL << 31)) return cudaErrorNotSupported;
    const bool wide = reinterpret_cast<uintptr_t>(a.x) % 32 == 0 && a.ldx * sizeof(T) % 32 == 0;
    auto* kernel = block == 16 ? quantize_fp4_kernel<T, kForm, 16> : quantize_fp4_kernel<T, kForm, 32>;
    const cudaError_t e = launch_dependent(kernel, dim3((unsigned)ctas), dim3(tx, ty), 0, 0, stream, a, wide);
    note_launch();
    return e;
}

template <int kForm>
cudaError_t by_type(const Args& a, q8_float_type t, int block, cudaStream_t stream) {
    switch (t) {
        case Q8_F32: return launch<float, kForm>(a, block, stream);
        case Q8_BF16: return launch<__nv_bfloat16, kForm>(a, block, stream);
        default: return launch<__half, kForm>(a, block, stream);
    }
}

// Four codes, in the low 16 bits of c, as e4m3: a table of eight bytes by their low bits, and the signs.
__device__ __forceinline__ uint32_t e4m3x4(uint32_t c) {
    uint32_t v;
    asm("prmt.b32 %0, %1, %2, %3;\n" : "=r"(v) : "r"(0x3C383000u), "r"(0x4C484440u), "r"(c & 0x7777u));
    return v | (c & 0x8u) << 4 | (c & 0x80u) << 8 | (c & 0x800u) << 12 | (c & 0x8000u) << 16;
}

// Eight codes as floats.
__device__ __forceinline__ void floats8(uint32_t c, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h;
        asm("{\n.reg .b8 b;\ncvt.u8.u32 b, %1;\ncvt.rn.f16x2.e2m1x2 %0, b;\n}\n" : "=r"(h) : "r"((c >> (8 * j)) & 0xffu));
        const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * j] = t.x;
        f[2 * j + 1] = t.y;
    }
}

// 32 bytes to y: at once where its rows start on them.
__device__ __forceinline__ void put32(void* y, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(y), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(y)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(y)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// 32 codes at a time, two of them a thread with both loads first: one scale of blocks of 32, two of blocks of 16. Bound by
// memory: the codes of 8192 x 16384 to e4m3 30.5 us (0.97 of the measured copy bandwidth; 34.9 with 16 at a time), with scales to bf16
// 53 us (0.96).
constexpr int kBack = 256, kBackUnroll = 2;
template <class T>
__global__ void __launch_bounds__(kBack) dequantize_fp4_kernel(const uint8_t* q, const uint8_t* sf, const float* s, int block,
                                                               uint64_t total, uint32_t per_row, uint32_t pitch,
                                                               uint32_t tile_rows, T* y, bool wide) {
    depend_wait();
    const uint64_t first = (uint64_t)blockIdx.x * (kBack * kBackUnroll) + threadIdx.x;
    uint4 c[kBackUnroll];
#pragma unroll
    for (int r = 0; r < kBackUnroll; ++r)
        c[r] = first + r * kBack < total ? load128(reinterpret_cast<const uint4*>(q) + first + r * kBack) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < kBackUnroll; ++r) {
        const uint64_t i = first + r * kBack;
        if (i >= total) return;
        const uint32_t w[4] = {c[r].x, c[r].y, c[r].z, c[r].w};
        if constexpr (sizeof(T) == 1) {
            uint32_t out[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                out[2 * j] = e4m3x4(w[j]);
                out[2 * j + 1] = e4m3x4(w[j] >> 16);
            }
            put32(y + i * 32, out, wide);
        } else {
            float scale[2] = {1.0f, 1.0f}, by = 1.0f;
            if (sf || s) {
                const uint64_t row = i / per_row;
                const uint32_t k = (uint32_t)(i - row * per_row) * 32;
                if (sf) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t b = (k + 16 * h) / block;
                        size_t at = row * pitch + b;
                        if (tile_rows) {
                            const uint64_t e = row / tile_rows;
                            const uint32_t n = (uint32_t)(row - e * tile_rows);
                            at = ((e * ((tile_rows + 127) / 128) + n / 128) * (pitch / 4) + b / 4) * 512 + (n % 32) * 16 +
                                 n % 128 / 32 * 4 + b % 4;
                        }
                        const uint32_t v = load8(sf + at);
                        // 2^-127 is subnormal: its bit is below the exponent's
                        scale[h] = block == 16 ? of_e4m3(v) : v == 255u ? __uint_as_float(0x7fffffffu)
                                                                         : __uint_as_float(v ? v << 23 : 0x400000u);
                    }
                }
                if (s) by = load_float(s + row);
            }
            constexpr int kPer = 32 / sizeof(T);       // values of a store
            uint32_t out[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[8];
                floats8(w[j], f);
#pragma unroll
                for (int l = 0; l < 8; ++l) {
                    const float v = __fmul_rn(__fmul_rn(f[l], scale[j / 2]), by);
                    if constexpr (sizeof(T) == 4) {
                        out[l] = __float_as_uint(v);
                    } else {
                        const T t = from_float<T>(v);
                        const uint32_t bits = *reinterpret_cast<const uint16_t*>(&t);
                        uint32_t& word = out[(j % 2) * 4 + l / 2];
                        word = l % 2 ? word | bits << 16 : bits;
                    }
                }
                if (sizeof(T) == 4 || j % 2) put32(y + i * 32 + (sizeof(T) == 4 ? j : j / 2) * kPer, out, wide);
            }
        }
    }
}

template <class T>
cudaError_t dequantize(const uint8_t* q, const uint8_t* sf, const float* s, int block, uint64_t total, int64_t K, int64_t tile_rows,
                       void* y, cudaStream_t stream) {
    const uint64_t per = kBack * kBackUnroll;
    return launch_dependent(dequantize_fp4_kernel<T>, dim3((unsigned)((total + per - 1) / per)), dim3(kBack), 0, 0, stream, q, sf,
                            s, block, total, (uint32_t)(K / 32), (uint32_t)fp4_pitch(K, block), (uint32_t)tile_rows,
                            static_cast<T*>(y), reinterpret_cast<uintptr_t>(y) % 32 == 0);
}

}  // namespace

cudaError_t launch_quantize_fp4(const void* x, q8_float_type t, int block, int64_t M, int64_t K, int64_t ldx,
                                const int32_t* slots, int top_k, int64_t rows_out, uint8_t* q, uint8_t* sf, float* s,
                                cudaStream_t stream) {
    const Args a{x, (uint32_t)K, 0, ldx, M, 0, slots, top_k, rows_out, q, sf, (uint32_t)fp4_pitch(K, block), s};
    return slots ? by_type<kSlots>(a, t, block, stream) : by_type<kDense>(a, t, block, stream);
}

cudaError_t launch_swiglu_quantize_fp4(const void* h, q8_float_type t, int block, int64_t M, int64_t I, int64_t ldh,
                                       uint8_t* q, uint8_t* sf, float* s, cudaStream_t stream) {
    const Args a{h, (uint32_t)I, 0, ldh, M, 0, nullptr, 0, M, q, sf, (uint32_t)fp4_pitch(I, block), s};
    return by_type<kGated>(a, t, block, stream);
}

cudaError_t launch_quantize_weight_fp4(const void* w, q8_float_type t, int block, int64_t E, int64_t N, int64_t K,
                                       uint8_t* q, uint8_t* sf, float* s, cudaStream_t stream) {
    const Args a{w, (uint32_t)K, 0, K, E * N, (uint32_t)N, nullptr, 0, E * ((N + 127) / 128 * 128), q, sf,
                 (uint32_t)fp4_pitch(K, block), s};
    return by_type<kTiles>(a, t, block, stream);
}

cudaError_t launch_dequantize_fp4(const uint8_t* q, const uint8_t* sf, const float* s, int block, int64_t rows, int64_t K,
                                  int64_t tile_rows, void* y, q8_float_type type, bool e4m3, cudaStream_t stream) {
    const uint64_t total = (uint64_t)rows * (uint64_t)(K / 32);
    if (total > 255ull << 31) return cudaErrorNotSupported;
    const cudaError_t e = e4m3             ? dequantize<uint8_t>(q, sf, s, block, total, K, tile_rows, y, stream)
                          : type == Q8_F32  ? dequantize<float>(q, sf, s, block, total, K, tile_rows, y, stream)
                          : type == Q8_BF16 ? dequantize<__nv_bfloat16>(q, sf, s, block, total, K, tile_rows, y, stream)
                                            : dequantize<__half>(q, sf, s, block, total, K, tile_rows, y, stream);
    note_launch();
    return e;
}

}  // namespace q8
