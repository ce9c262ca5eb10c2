// Tiles of the products with routed experts and their way out of registers: shared by the float8 and the 4-bit products.
#pragma once

#include "q8_fp8.h"
#include "q8_fp8_ptx.cuh"
#include "q8_loads.cuh"

namespace q8 {
namespace tc {

// Token tiles before each group, and the rows of a group, from the offsets. Ranges are cut to
// [0, rows], so that no offset, whatever its value, leads outside of qa and y. Offsets that fall make ranges overlap, and
// up to E times the tiles that disjoint ranges have: `units` cuts the work to what those can have, which the host has
// checked to be below 2^31 (so that no unit's number wraps and no kernel runs for the sum of all overlaps).
// kEarly: the kernel may have started before the one that wrote the offsets was done.
template <bool kEarly>
struct GroupsOf {
    const int32_t* offsets;
    const int* cum;   // shared: tiles before group e
    int rows, E, tn;
    __device__ __forceinline__ void range(int e, int& lo, int& hi) const {
        if (!offsets) {
            lo = 0;
            hi = rows;
        } else {
            lo = min(max(at(e), 0), rows);
            hi = min(max(at(e + 1), lo), rows);
        }
    }
    __device__ __forceinline__ int at(int e) const {
        if constexpr (kEarly) return load_int(offsets + e);
        else return __ldg(offsets + e);
    }
    // token tile t -> its group, first row and rows
    __device__ __forceinline__ void tile(int t, int& e, int& row, int& n) const {
        int a = 0, b = E;
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (cum[mid] <= t) a = mid;
            else b = mid;
        }
        e = a;
        int lo, hi;
        range(e, lo, hi);
        row = lo + (t - cum[e]) * tn;
        n = min(tn, hi - row);
    }
    // tiles (token tiles times the NT weight tiles) to work on
    __device__ __forceinline__ uint32_t units(int NT, uint32_t most) const {
        const uint64_t all = (uint64_t)(uint32_t)cum[E] * (uint32_t)NT;
        return all < most ? (uint32_t)all : most;
    }
    // one warp: the prefix sums
    __device__ __forceinline__ void scan(int* out, int lane) const {
        int run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            int c = 0;
            if (e0 + lane < E) {
                int lo, hi;
                range(e0 + lane, lo, hi);
                c = (hi - lo + tn - 1) / tn;
            }
            int s = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, s, d);
                if (lane >= d) s += o;
            }
            if (e0 + lane < E) out[e0 + lane] = run + s - c;
            run += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) out[E] = run;
    }
};
using Groups = GroupsOf<false>;
using EarlyGroups = GroupsOf<true>;

__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
    const uint4 u = lds128(addr);
    return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
}

// Two values of a 16-bit type as one word.
template <class T>
__device__ __forceinline__ uint32_t pack16(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// acc[j]: weight row (column of y) col, token t0 + j. Tokens are stored where t < n and (t / 4) % split == rank
// (all of them for split = 1). 16-bit types: neighbouring lanes trade values, so that each stores two
// columns of one token as a word; y's rows have to start on whole words for that.
template <class T, int CW>
__device__ __forceinline__ void store_tokens(T* y, int64_t row, int t0, int n, int col, int N, const float (&acc)[CW],
                                             int split, int rank, int lane) {
    if (sizeof(T) == 2 && N % 2 == 0) {
        const int odd = lane & 1;
        if constexpr (sizeof(T) == 2) {
            T* out = y + (row + t0 + odd) * N + (col - odd);
#pragma unroll
            for (int j = 0; j < CW; j += 2, out += 2 * (int64_t)N) {
                const float give = odd ? acc[j] : acc[j + 1];
                const float got = __shfl_xor_sync(0xffffffffu, give, 1);
                const int t = t0 + j + odd;
                if (t < n && col < N && (split == 1 || ((t / 4) & (split - 1)) == rank))
                    *reinterpret_cast<uint32_t*>(out) = odd ? pack16<T>(got, acc[j + 1]) : pack16<T>(acc[j], got);
            }
        }
    } else if (col < N) {
        T* out = y + (row + t0) * N + col;
#pragma unroll
        for (int j = 0; j < CW; ++j, out += N) {
            const int t = t0 + j;
            if (t < n && (split == 1 || ((t / 4) & (split - 1)) == rank)) *out = from_float<T>(acc[j]);
        }
    }
}

constexpr int kBand = 8;                         // token tiles that share a sweep over the weights (8192x8192x16384 back
                                                 // to back: 4 3 % slower, 32 6 %; 16 the same, and 2 % slower for experts)

// Units in bands of kBand token tiles, the weight tiles swept inside a band, so that the tiles that run
// together share both operands in L2.
__device__ __forceinline__ void pair_unit(uint32_t u, int tiles, int NT, int& t, int& nt) {
    const uint32_t per = (uint32_t)kBand * NT;
    const int band = (int)(u / per), within = (int)(u - band * per);
    const int here = min(kBand, tiles - band * kBand);
    t = band * kBand + within % here;
    nt = within / here;
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// A drain warp's 32 rows x 2 NC columns (one row a lane) to y, 64 bytes of each row at a time through
// shared memory (16-byte chunk j of row r at j ^ (r / 2 % 4): no bank conflicts either way), so that
// four lanes write two sectors. Rows of y that are not whole 16-byte chunks go by words, or by 16-bit values for
// an odd number of them, the lanes of a row side by side (6532 fp32 rows of 4575 columns, K = 320: 147 us when
// a lane wrote its 16 bytes value by value).
template <class T, int NC>
__device__ __forceinline__ void store_rows(T* y, int64_t row0, int live, int col0, int N, const uint64_t (&acc)[NC],
                                           uint32_t buf, int lane) {
    constexpr int kCols = 64 / sizeof(T);         // columns of a step
    const int unit = (N * sizeof(T)) % 16 == 0 ? 16 : (N * sizeof(T)) % 4 == 0 ? 4 : 2;
#pragma unroll
    for (int c = 0; c < 2 * NC / kCols; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if constexpr (sizeof(T) == 2) {
                const float2 f = unpack2(acc[c * 16 + j]);
                w[j] = pack16<T>(f.x, f.y);
            } else {
                const float2 f = unpack2(acc[c * 8 + j / 2]);
                w[j] = __float_as_uint(j & 1 ? f.y : f.x);
            }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sts128(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4),
                   make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
        __syncwarp();
        const int at = col0 + c * kCols;
        // byte b of row r of the staged step
        auto staged = [&](int r, int b) { return buf + r * 64 + (((b >> 4) ^ ((r >> 1) & 3)) << 4) + (b & 15); };
        if (unit == 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = i * 8 + lane / 4, b = (lane & 3) * 16, col = at + b / (int)sizeof(T);
                const uint4 v = lds128(staged(r, b));
                if (r < live && col < N) *reinterpret_cast<uint4*>(y + (row0 + r) * N + col) = v;
            }
        } else {
            // lane's bytes b of rows r, r + step, ...: loops, so that their addresses do not cost registers here
            const int lanes = 64 / unit, step = unit / 2;   // lanes of a row, rows of a pass: 16 and 2, or 32 and 1
            const int b = lane % lanes * unit, col = at + b / (int)sizeof(T);
#pragma unroll 2
            for (int r = lane / lanes; r < live && col < N; r += step) {
                T* out = y + (row0 + r) * N + col;
                if (unit == 4) {
                    uint32_t v;
                    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(staged(r, b)) : "memory");
                    *reinterpret_cast<uint32_t*>(out) = v;
                } else {
                    uint16_t v;
                    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(staged(r, b)) : "memory");
                    *reinterpret_cast<uint16_t*>(out) = v;
                }
            }
        }
    }
}

}  // namespace tc
}  // namespace q8
