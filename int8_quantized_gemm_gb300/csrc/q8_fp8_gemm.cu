// Products of float8 (e4m3) matrices with a scale for each row and 128 K of the activations and each
// 128 x 128 block of the weights, for one weight matrix or one for each group of rows (experts).
//
//   y[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in block b} qa[m, k] qw[n, k]
//
// The tensor core (tcgen05 kind::f8f6f4) sums one block of 128 K at a time in fp32 in tensor memory;
// drain warps read each partial sum and add it, times its scale, to fp32 registers. The MMA of the
// next block runs meanwhile, on another of the accumulator's buffers.
#include <cuda.h>

#include "q8_fp8.h"
#include "q8_fp8_ptx.cuh"
#include "q8_internal.h"

namespace q8 {
namespace {

using namespace tc;

__device__ unsigned int g_fp8_error = 0;

// Bounded waits of a whole warp: its lanes agree on how the wait ended, so that none goes on alone to an
// instruction that takes them all.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned code) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, code, &g_fp8_error));
}
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned code) {
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort_flag, code, &g_fp8_error));
}

constexpr int BK = kFp8Block;          // K of a stage: one scale block, 128 bytes a row
constexpr int TW = 128;                // weight rows of a tile: one scale block, the MMA's M side
constexpr int kTileW = TW * BK;        // 16 KB
constexpr uint32_t kIdescW = idesc_f16(TW, 0);   // fp32 D, e4m3 A and B, both K-major, M = 128

// -------------------------------------------------------------------------- weights on the MMA's M side
// For few tokens a matrix: a tile is 128 weight rows x up to TN = 16, 32 or 64 token rows, so that a weight
// block is read once whatever the tokens. Bound by the weights' bytes.
//   warp 0     TMA: weights [128 x 128] and tokens [n x 128] of each K block, 128-byte swizzle
//   warp 1     MMA issuer (N = n rounded up to 16), TMEM
//   warps 2, 3 scales of the block's tokens, sa sw, into the buffer's scale row
//   warps 4-11 drain: two warps for each quarter of the TMEM lanes (weight rows), half of the tokens each
// With few tiles, a cluster of S CTAs splits a tile's K blocks; each CTA sends the partial sums of the
// tokens it does not own to the CTA that does (st.async), which adds them in the order of the ranks:
// the same bits every time, no workspace and no second launch.
// Measured: 128 rows of 64 experts, 4096 x 4096, 163 us (0.97 of the measured copy bandwidth on the active
// weights); 16x28672x8192 43.6 us (0.80: two CTAs share a tile so that 224 tiles fill three rounds; set-up, the first
// load, the last exchange and store are about 6 us); 1x4096x4096 8.9 us.
constexpr int kSwapThreads = 384;
constexpr int kDrainWarps = 8;
constexpr int kBufs = 8;               // accumulator buffers: the MMA runs on while a tile is written out
constexpr int kMaxStages = 8;          // more bytes in flight cost DRAM row hits: 128 rows of 64 experts 4096x4096
                                       // 175 us with 12 stages, 168 with 10, 163 with 8, 166 with 6
constexpr int kTailBytes = 8 * (2 * kMaxStages + 2 * kBufs + 2) + 32 + 4 * (kMaxExperts + 2);
constexpr int kSmemMax = 227 * 1024;

struct SwapArgs {
    const float* sa;
    const float* sw;
    const int32_t* offsets;   // nullptr: one group of all rows
    int rows, E;
    int N, K;
    int stages;               // of the ring
    int split;                // CTAs of a cluster, sharing a tile's K blocks
    void* y;
    q8_float_type type;
    uint32_t most;            // units there can be
};

// Token tiles before each group, and the rows of a group, from the offsets. Ranges are cut to
// [0, rows], so that no offset, whatever its value, leads outside of qa and y. Offsets that fall make ranges overlap, and
// up to E times the tiles that disjoint ranges have: `units` cuts the work to what those can have, which the host has
// checked to be below 2^31 (so that no unit's number wraps and no kernel runs for the sum of all overlaps).
struct Groups {
    const int32_t* offsets;
    const int* cum;   // shared: tiles before group e
    int rows, E, tn;
    __device__ __forceinline__ void range(int e, int& lo, int& hi) const {
        if (!offsets) {
            lo = 0;
            hi = rows;
        } else {
            lo = min(max(__ldg(offsets + e), 0), rows);
            hi = min(max(__ldg(offsets + e + 1), lo), rows);
        }
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

template <int CW>   // tokens of a drain warp; TN = 2 CW
struct SwapCfg {
    static constexpr int TN = 2 * CW;
    static constexpr int kBox = TN < 32 ? TN : 32;              // token rows of a TMA box
    static constexpr int kStage = kTileW + TN * BK;
    static constexpr int kScale = kBufs * TN * 4;
    static constexpr int kTmem = kBufs * TN;                    // 128, 256 or 512 columns
    // receive buffer: the groups of four tokens that a CTA owns, from each other CTA
    static int reduce_bytes(int split) { return (split - 1) * ((TN / 4 + split - 1) / split) * TW * 16; }
};

template <int CW>
__global__ void __launch_bounds__(kSwapThreads, 1)
    gemm_fp8_swap_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                         SwapArgs p, int reduce_bytes) {
    using C = SwapCfg<CW>;
    constexpr int TN = C::TN;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sraw = smem_u32(smem_raw);
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - sraw);
    const uint32_t off_scale = p.stages * C::kStage;
    const uint32_t off_reduce = off_scale + C::kScale;
    const uint32_t off_bar = off_reduce + reduce_bytes;
    const uint32_t bar_full = sbase + off_bar;
    const uint32_t bar_empty = bar_full + 8 * kMaxStages;
    const uint32_t bar_accfull = bar_empty + 8 * kMaxStages;
    const uint32_t bar_accempty = bar_accfull + 8 * kBufs;
    const uint32_t bar_got = bar_accempty + 8 * kBufs;   // split: the partial sums of this CTA's tokens
    const uint32_t bar_free = bar_got + 8;               // split: every CTA's drain warps are done with a unit
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + off_bar + 8 * (2 * kMaxStages + 2 * kBufs + 2));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* cum = reinterpret_cast<int*>(tmem_slot + 2);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;

    const int NT = (p.N + TW - 1) / TW, KB = (p.K + BK - 1) / BK;
    const uint32_t first = blockIdx.x / p.split, step = gridDim.x / p.split;
    const int kb0 = KB / p.split * rank + min(rank, KB % p.split);   // this CTA's share of the K blocks
    const int kb1 = kb0 + KB / p.split + (rank < KB % p.split ? 1 : 0);
    const Groups groups{p.offsets, cum, p.rows, p.E, TN};

    if (warp == 0) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
            for (int s = 0; s < p.stages; ++s) {
                mbar_init(bar_full + 8 * s, 1);
                mbar_init(bar_empty + 8 * s, 1);
            }
            for (int b = 0; b < kBufs; ++b) {
                mbar_init(bar_accfull + 8 * b, 3);    // the MMA's commit and the two scale warps
                mbar_init(bar_accempty + 8 * b, kDrainWarps);
            }
            mbar_init(bar_got, 1);
            mbar_init(bar_free, p.split * kDrainWarps);
            *abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        }
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::kTmem);
    if (warp == 2) groups.scan(cum, lane);
    tc_fence_before();
    if (p.split > 1) cluster_sync();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t units = groups.units(NT, p.most);

    if (warp == 0) {
        // ---------------------------------------------------------------------------- TMA
        uint32_t s = 0, phase = 1;
        bool ok = true;
        for (uint32_t u = first; u < units && ok; u += step) {
            int e, row, n;
            groups.tile((int)(u / (uint32_t)NT), e, row, n);
            const int wrow = e * p.N + (int)(u % (uint32_t)NT) * TW, boxes = (n + C::kBox - 1) / C::kBox;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_wait(bar_empty + 8 * s, phase, abort_flag, kErrProducer)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = sbase + s * C::kStage, bar = bar_full + 8 * s;
                if (elect_one()) {
                    mbar_expect_tx(bar, kTileW + boxes * C::kBox * BK);
                    tma_load_2d(dst, &tmap_w, kb * BK, wrow, bar);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(dst + kTileW + b * C::kBox * BK, &tmap_a, kb * BK, row + b * C::kBox, bar);
                }
                __syncwarp();
                if (++s == (uint32_t)p.stages) { s = 0; phase ^= 1; }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------------------- MMA
        uint32_t s = 0, phase = 0, buf = 0, bphase = 1;
        bool ok = true;
        for (uint32_t u = first; u < units && ok; u += step) {
            int e, row, n;
            groups.tile((int)(u / (uint32_t)NT), e, row, n);
            const uint32_t idesc = kIdescW + ((uint32_t)((n + 15) >> 4) << 18);   // N = n rounded up to 16
            for (int kb = kb0; kb < kb1; ++kb) {
                const bool got = mbar_wait(bar_accempty + 8 * buf, bphase, abort_flag, kErrMmaAcc, &g_fp8_error) &&
                                 mbar_wait(bar_full + 8 * s, phase, abort_flag, kErrMmaFull, &g_fp8_error);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t w = smem_desc_sw128(sbase + s * C::kStage);
                const uint64_t a = smem_desc_sw128(sbase + s * C::kStage + kTileW);
                const uint32_t d = tmem_base + buf * TN;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk) mma_fp8(d, w + 2 * kk, a + 2 * kk, idesc, kk ? 1u : 0u);
                    mma_commit(bar_empty + 8 * s);
                    mma_commit(bar_accfull + 8 * buf);
                }
                __syncwarp();
                if (++s == (uint32_t)p.stages) { s = 0; phase ^= 1; }
                if (++buf == kBufs) { buf = 0; bphase ^= 1; }
            }
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------------------- scales
        // A lane has one token. Four blocks' scales are loaded ahead of the four being handed out.
        constexpr int kAhead = 4;
        const int col = (warp - 2) * 32 + lane;
        uint32_t buf = 0, bphase = 1;
        bool ok = true;
        for (uint32_t u = first; u < units && ok; u += step) {
            int e, row, n;
            groups.tile((int)(u / (uint32_t)NT), e, row, n);
            const float* sw = p.sw + ((int64_t)e * NT + (int)(u % (uint32_t)NT)) * KB;
            const float* sa = p.sa + (int64_t)(row + min(col, n - 1)) * KB;
            float next[kAhead];
            auto load = [&](int kb) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    next[i] = kb + i < kb1 && col < n ? __ldg(sa + kb + i) * __ldg(sw + kb + i) : 0.0f;
            };
            load(kb0);
            for (int kb = kb0; kb < kb1 && ok; kb += kAhead) {
                float now[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) now[i] = next[i];
                load(kb + kAhead);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (kb + i >= kb1) break;
                    if (!warp_wait(bar_accempty + 8 * buf, bphase, abort_flag, kErrConvEmpty)) {
                        ok = false;
                        break;
                    }
                    if (col < TN) reinterpret_cast<float*>(smem + off_scale)[buf * TN + col] = now[i];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_accfull + 8 * buf);
                    if (++buf == kBufs) { buf = 0; bphase ^= 1; }
                }
            }
        }
    } else {
        // -------------------------------------------------------------------------- drain
        const int quarter = warp & 3, t0 = ((warp - 4) >> 2) * CW;   // its first token
        const uint32_t tlane = tmem_base + ((uint32_t)(quarter * 32) << 16) + t0;
        uint32_t buf = 0, bphase = 0, done = 0;
        bool ok = true;
        for (uint32_t u = first; u < units && ok; u += step, ++done) {
            int e, row, n;
            groups.tile((int)(u / (uint32_t)NT), e, row, n);
            const int col = (int)(u % (uint32_t)NT) * TW + quarter * 32 + lane;   // this thread's weight row
            float acc[CW];
#pragma unroll
            for (int j = 0; j < CW; ++j) acc[j] = 0.0f;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!warp_wait(bar_accfull + 8 * buf, bphase, abort_flag, kErrDrain)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (t0 < n) {
                    uint32_t v[CW];
                    tmem_load(tlane + buf * TN, v);
                    const uint32_t sc = sbase + off_scale + (buf * TN + t0) * 4;
#pragma unroll
                    for (int j = 0; j < CW; j += 4) {
                        const float4 f = lds_f4(sc + j * 4);
                        acc[j] = __fmaf_rn(__uint_as_float(v[j]), f.x, acc[j]);
                        acc[j + 1] = __fmaf_rn(__uint_as_float(v[j + 1]), f.y, acc[j + 1]);
                        acc[j + 2] = __fmaf_rn(__uint_as_float(v[j + 2]), f.z, acc[j + 2]);
                        acc[j + 3] = __fmaf_rn(__uint_as_float(v[j + 3]), f.w, acc[j + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_accempty + 8 * buf);
                if (++buf == kBufs) { buf = 0; bphase ^= 1; }
            }
            if (!ok) break;
            if (p.split > 1) {   // tokens in groups of four: group g is added up by CTA g % split
                const int S = p.split, log = __ffs(S) - 1, groups4 = (n + 3) / 4;
                const int per = (groups4 + S - 1) / S;          // slots of groups in the receive buffer
                const int here = (groups4 - rank + S - 1) / S;  // groups that this CTA owns (may be 0)
                const uint32_t buffer = sbase + off_reduce, lane16 = (quarter * 32 + lane) * 16;
                if (done && !warp_wait_cluster(bar_free, (done - 1) & 1, abort_flag, kErrRelay)) break;
                if (warp == 4 && lane == 0) mbar_expect_tx(bar_got, (S - 1) * max(here, 0) * TW * 16);
#pragma unroll
                for (int q = 0; q < CW / 4; ++q) {
                    const int g = t0 / 4 + q, owner = g & (S - 1);
                    if (g < groups4 && owner != rank) {
                        const int slot = (rank < owner ? rank : rank - 1) * per + (g >> log);
                        st_async16(mapa_shared(buffer + slot * (TW * 16) + lane16, owner),
                                   make_uint4(__float_as_uint(acc[4 * q]), __float_as_uint(acc[4 * q + 1]),
                                              __float_as_uint(acc[4 * q + 2]), __float_as_uint(acc[4 * q + 3])),
                                   mapa_shared(bar_got, owner));
                    }
                }
                if (!warp_wait_cluster(bar_got, done & 1, abort_flag, kErrRelay)) break;
#pragma unroll
                for (int q = 0; q < CW / 4; ++q) {
                    const int g = t0 / 4 + q;
                    if (g < groups4 && (g & (S - 1)) == rank) {
                        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int r = 0; r < S; ++r) {
                            float4 f = make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
                            if (r != rank)
                                f = lds_f4(buffer + ((r < rank ? r : r - 1) * per + (g >> log)) * (TW * 16) + lane16);
                            t.x += f.x; t.y += f.y; t.z += f.z; t.w += f.w;
                        }
                        acc[4 * q] = t.x; acc[4 * q + 1] = t.y; acc[4 * q + 2] = t.z; acc[4 * q + 3] = t.w;
                    }
                }
                // To every CTA, its own too: a warp arrives for this unit only after it has seen the last one's
                // phase (the wait above), so no phase can be passed while a warp still waits for it.
                __syncwarp();
                if (lane < S) mbar_arrive_remote(mapa_shared(bar_free, lane));
            }
            if (p.type == Q8_BF16)
                store_tokens(static_cast<__nv_bfloat16*>(p.y), row, t0, n, col, p.N, acc, p.split, rank, lane);
            else if (p.type == Q8_F16)
                store_tokens(static_cast<__half*>(p.y), row, t0, n, col, p.N, acc, p.split, rank, lane);
            else
                store_tokens(static_cast<float*>(p.y), row, t0, n, col, p.N, acc, p.split, rank, lane);
        }
    }

    __syncthreads();
    if (*abort_flag) {
        const long long t0 = clock64();
        while (clock64() - t0 < (1LL << 22)) __nanosleep(1000);
    }
    tc_fence_before();
    // no CTA of a cluster leaves while another may still send to it
    if (p.split > 1) cluster_sync();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, C::kTmem);
}

// Clusters of `split` CTAs that run at once; the kernel's shared-memory limit is raised on the first call.
// Kept per device and split (a query takes longer than a small product).
template <int CW>
cudaError_t swap_clusters(int split, int& clusters) {
    static int cached[64][4] = {};
    const int log = split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && cached[dev][log] > 0) {
        clusters = cached[dev][log];
        return cudaSuccess;
    }
    e = cudaFuncSetAttribute(gemm_fp8_swap_kernel<CW>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    clusters = device_sm_count() / split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * split), 1, 1);
    cfg.blockDim = dim3(kSwapThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemMax;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)split, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int fit = 0;
    e = cudaOccupancyMaxActiveClusters(&fit, gemm_fp8_swap_kernel<CW>, &cfg);
    if (e != cudaSuccess) return e;
    if (fit > 0 && fit < clusters) clusters = fit;
    if (dev < 64) cached[dev][log] = clusters;
    return cudaSuccess;
}

// The split that ends first: rounds of tiles over the clusters, each a part of the K blocks and a fixed cost of
// about four blocks (the exchange and the store). `cost`: in blocks of one CTA.
template <int CW>
cudaError_t swap_plan(int64_t tiles, int64_t N, int64_t K, int& split, int& clusters, double& cost) {
    const int64_t units = tiles * ((N + TW - 1) / TW), KB = (K + BK - 1) / BK;
    for (int S = 1; S <= 8 && (S == 1 || S * 2 <= KB); S *= 2) {
        int fit = 0;
        const cudaError_t e = swap_clusters<CW>(S, fit);
        if (e != cudaSuccess) return e;
        const double c = (double)((units + fit - 1) / fit) * (double)((KB + S - 1) / S + 4);
        if (S == 1 || c < cost * 0.98) {
            cost = c;
            split = S;
            clusters = fit;
        }
    }
    if (units < clusters) clusters = (int)units;
    return cudaSuccess;
}

template <int CW>
cudaError_t launch_swap(const uint8_t* qa, const uint8_t* qw, SwapArgs p, int64_t tiles, cudaStream_t stream) {
    using C = SwapCfg<CW>;
    int clusters = 0;
    double cost = 0.0;
    cudaError_t e = swap_plan<CW>(tiles, p.N, p.K, p.split, clusters, cost);
    if (e != cudaSuccess) return e;
    p.most = (uint32_t)(tiles * ((p.N + TW - 1) / TW));
    const int reduce = p.split > 1 ? C::reduce_bytes(p.split) : 0;
    const int room = kSmemMax - 1024 - kTailBytes - C::kScale - reduce;
    p.stages = room / C::kStage < kMaxStages ? room / C::kStage : kMaxStages;
    CUtensorMap ma, mw;
    if (!make_tma_map_i8(&ma, reinterpret_cast<const int8_t*>(qa), p.rows, p.K, C::kBox, BK, true) ||
        !make_tma_map_i8(&mw, reinterpret_cast<const int8_t*>(qw), (int64_t)p.E * p.N, p.K, TW, BK, true))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * p.split), 1, 1);
    cfg.blockDim = dim3(kSwapThreads, 1, 1);
    cfg.dynamicSmemBytes = 1024 + p.stages * C::kStage + C::kScale + reduce + kTailBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)p.split, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gemm_fp8_swap_kernel<CW>, ma, mw, p, reduce);
    note_launch();
    return e;
}

// ------------------------------------------------------------------ tokens on the MMA's M side, CTA pairs
// For many tokens: a cluster of two CTAs shares a tile of 256 token rows x PN = 256 or 128 weight rows
// (cta_group::2; each CTA loads half of both and holds its 128 token rows' accumulators). Per CTA:
//   warp 0     TMA: tokens [128 x 128] and weights [PN / 2 x 128] of each K block, completing on the even CTA's
//              barrier
//   warp 1     even CTA: pair MMA issuer; TMEM in both
//   warps 2, 3 scales: sa sw of the CTA's 128 token rows and the tile's one or two weight blocks, four or eight
//              K blocks at a time (neighbours in a row of sa), into shared memory
//   warps 4-11 drain: a TMEM lane is a token row, so a thread's scale is one value a block, and the sum
//              costs one multiply-add a value; two warps for each quarter of the lanes, PN / 2 columns each
// Measured at 8192x8192x16384: 804 us from a cool start (2.7 PFLOP/s), 875 to 885 us back to back, where the power
// cap holds the SM clock at 1.69 GHz (with all-zero codes 2.03 GHz and 764 us). The MMAs are 0.92 M of some 1.5 M clocks
// either way, so the cap costs a sixth of the time, and the tensor pipe stands still for 40 % of it. The loads and MMAs
// alone (sums read once a tile: wrong results) take 674 us, with every block's hand-over but no sums 756: what is left is
// the round trip MMA, commit, TMEM read, arrive, next MMA on two buffers (TMEM holds no third of 256 columns;
// four of 128 in halves of a tile cost the MMA alone 838), in which a drain warp's reads and sums take turns. A second
// issuer warp, spinning without suspension, and 16 drain warps of 64 columns each were slower.
constexpr int PT = 256, PTH = 128;
constexpr int kPairDrain = 8;                    // drain warps
constexpr int kPairThreads = 128 + 32 * kPairDrain;
constexpr int kPairLd = 64;                      // columns of one TMEM load
constexpr int kPairRegsLow = 88, kPairRegsHigh = 208;
static_assert(128 * kPairRegsLow + 32 * kPairDrain * kPairRegsHigh <= kPairThreads * (65536 / kPairThreads / 8 * 8),
              "above the launch's registers");
constexpr int kPairEpi = 2048;                   // of a drain warp: 32 rows x 64 bytes
constexpr int kScalePitch = PTH + 8;             // floats of a block's row of scales

template <int PN>
struct Pair8Cfg {
    static constexpr int kHalf = PN / 2;                      // weight rows of a CTA; columns of a drain warp
    static constexpr int kStage = (PTH + kHalf) * BK;         // 32 KB, 24 KB
    static constexpr int kStages = PN == 256 ? 6 : 8;
    static constexpr int kBufs = 512 / PN;                    // accumulator buffers: block c is in stage c % kStages
    static_assert(kStages % kBufs == 0, "a stage has its buffer");   // and buffer c % kBufs
    static constexpr int kScaleBlocks = PN == 256 ? 4 : 8;    // K blocks of one hand-over of scales, as room allows
                                                              // (256x8192x8192, narrow: 27 us with 4, 25 with 8)
    static constexpr int kScaleHalf = kScaleBlocks * kScalePitch;   // of one weight block
    static constexpr int kOffEpi = kStages * kStage;
    static constexpr int kOffScale = kOffEpi + kPairDrain * kPairEpi;
    static constexpr int kScaleBuf = PN / BK * kScaleHalf;
    static constexpr int kOffBar = kOffScale + 2 * kScaleBuf * 4;
    static constexpr int kBars = 2 * kStages + kBufs + 4;
    static constexpr int kSmem = 1024 + kOffBar + 8 * kBars + 32 + 4 * (kMaxExperts + 2);
    static_assert(kSmem <= kSmemMax, "above the shared memory of one CTA");
    static constexpr uint32_t kIdesc = idesc_f16(PT, PN);
};
constexpr int kBand = 8;                         // token tiles that share a sweep over the weights (8192x8192x16384 back
                                                 // to back: 4 3 % slower, 32 6 %; 16 the same, and 2 % slower for experts)

struct PairArgs {
    const float* sa;
    const float* sw;
    const int32_t* offsets;
    int rows, E, N, K;
    void* y;
    q8_float_type type;
    uint32_t most;   // units there can be
};

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

template <int PN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                         PairArgs p) {
    using C = Pair8Cfg<PN>;
    constexpr int kStages = C::kStages, kBufs = C::kBufs, kScaleBlocks = C::kScaleBlocks;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sraw = smem_u32(smem_raw);
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - sraw);
    const uint32_t bar_full = sbase + C::kOffBar;             // used in the even CTA: both CTAs' loads
    const uint32_t bar_done = bar_full + 8 * kStages;          // both CTAs: the pair MMA's commit; the stage may
                                                               // be filled again, its partial sums be read
    const uint32_t bar_accempty = bar_done + 8 * kStages;      // used in the even CTA: both CTAs' drain warps
    const uint32_t bar_scfull = bar_accempty + 8 * kBufs;
    const uint32_t bar_scempty = bar_scfull + 16;
    float* scales = reinterpret_cast<float*>(smem + C::kOffScale);   // [2 buffers][weight block][K block][row]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 8 * C::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* cum = reinterpret_cast<int*>(tmem_slot + 2);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_done + 8 * s, 1);
        }
        for (int b = 0; b < kBufs; ++b) mbar_init(bar_accempty + 8 * b, 2 * kPairDrain);
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_scfull + 8 * b, 2);
            mbar_init(bar_scempty + 8 * b, kPairDrain);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
    }
    const Groups groups{p.offsets, cum, p.rows, p.E, PT};
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
    if (warp == 2) groups.scan(cum, lane);
    tc_fence_before();
    cluster_sync();   // barriers of both CTAs initialised, TMEM allocated in both
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int NT = (p.N + PN - 1) / PN, KB = (p.K + BK - 1) / BK;
    const int tiles = cum[p.E];
    const uint32_t units = groups.units(NT, p.most), first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kPairRegsLow));
        if (warp == 0) {
            // ------------------------------------------------------------------------ TMA
            const uint32_t full0 = mapa_shared(bar_full, 0);
            uint32_t s = 0, phase = 1;
            bool ok = true;
            for (uint32_t u = first; u < units && ok; u += step) {
                int t, nt, e, row, n;
                pair_unit(u, tiles, NT, t, nt);
                groups.tile(t, e, row, n);
                // A half without a token (or weight) row is loaded from past the end of the tensor: zeros, which cost
                // neither reads nor, under the power cap, as much of the clock as another group's rows (32768 rows of 64
                // experts back to back: 658 -> 652 us).
                const int arow = rank * PTH < n ? row + rank * PTH : p.rows;
                const int wrow = nt * PN + rank * C::kHalf < p.N ? e * p.N + nt * PN + rank * C::kHalf : p.E * p.N;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!warp_wait(bar_done + 8 * s, phase, abort_flag, kErrProducer)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + s * C::kStage;
                    if (elect_one()) {
                        if (rank == 0) mbar_expect_tx(bar_full + 8 * s, 2 * C::kStage);
                        tma_load_2d_pair(dst, &tmap_a, kb * BK, arow, full0 + 8 * s);
                        tma_load_2d_pair(dst + PTH * BK, &tmap_w, kb * BK, wrow, full0 + 8 * s);
                    }
                    __syncwarp();
                    if (++s == kStages) { s = 0; phase ^= 1; }
                }
            }
        } else if (warp == 1 && rank == 0) {
            // ------------------------------------------------------------------------ MMA
            uint32_t s = 0, phase = 0, c = 0;
            bool ok = true;
            for (uint32_t u = first; u < units && ok; u += step) {
                for (int kb = 0; kb < KB; ++kb, ++c) {
                    const uint32_t buf = c % kBufs;
                    const bool got =
                        mbar_wait_cluster(bar_accempty + 8 * buf, ((c / kBufs) & 1) ^ 1, abort_flag, kErrMmaAcc,
                                          &g_fp8_error) &&
                        mbar_wait_cluster(bar_full + 8 * s, phase, abort_flag, kErrMmaFull, &g_fp8_error);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a = smem_desc_sw128(sbase + s * C::kStage);
                    const uint64_t w = smem_desc_sw128(sbase + s * C::kStage + PTH * BK);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk)
                            mma_fp8_pair(tmem_base + buf * PN, a + 2 * kk, w + 2 * kk, C::kIdesc, kk ? 1u : 0u);
                        mma_commit_pair(bar_done + 8 * s, 3);
                    }
                    __syncwarp();
                    if (++s == kStages) { s = 0; phase ^= 1; }
                }
            }
        } else if (warp >= 2) {
            // --------------------------------------------------------------------- scales
            // A lane loads one K block of every 16th (8th) row; the next blocks' loads are in flight while
            // it waits for the buffer.
            constexpr int kStep = 64 / kScaleBlocks, kRows = PTH / kStep;   // rows of a pass, passes
            const int NB = (p.N + BK - 1) / BK;
            const int b = lane % kScaleBlocks, r0 = (warp - 2) * (kStep / 2) + lane / kScaleBlocks;
            uint32_t c = 0;
            bool ok = true;
            for (uint32_t u = first; u < units && ok; u += step) {
                int t, nt, e, row, n;
                pair_unit(u, tiles, NT, t, nt);
                groups.tile(t, e, row, n);
                row += rank * PTH + r0;
                const float* w0 = p.sw + ((int64_t)e * NB + nt * (PN / BK)) * KB;
                const float* w1 = PN > BK && nt * (PN / BK) + 1 < NB ? w0 + KB : w0;
                const float* sa = p.sa + (int64_t)row * KB;
                const int have = (p.rows - row + kStep - 1) / kStep;   // rows of this lane that exist
                float a[kRows], f0, f1;
                auto load = [&](int kb) {
                    const int rows_in = kb < KB ? have : 0;
                    f0 = kb < KB ? __ldg(w0 + kb) : 0.0f;
                    f1 = kb < KB ? __ldg(w1 + kb) : 0.0f;
                    const float* from = sa + kb;
#pragma unroll
                    for (int i = 0; i < kRows; ++i, from += kStep * KB) a[i] = i < rows_in ? __ldg(from) : 0.0f;
                };
                load(b);
                for (int kb = 0; kb < KB; kb += kScaleBlocks, ++c) {
                    const uint32_t buf = c & 1;
                    if (!warp_wait(bar_scempty + 8 * buf, ((c >> 1) & 1) ^ 1, abort_flag, kErrConvEmpty)) {
                        ok = false;
                        break;
                    }
                    float* out = scales + buf * C::kScaleBuf + b * kScalePitch + r0;
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        out[kStep * i] = a[i] * f0;
                        if (PN > BK) out[kStep * i + C::kScaleHalf] = a[i] * f1;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_scfull + 8 * buf);
                    load(kb + kScaleBlocks + b);
                }
            }
        }
    } else {
        // ---------------------------------------------------------------------------- drain
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kPairRegsHigh));
        const int quarter = warp & 3, part = ((warp - 4) >> 2) * C::kHalf;   // its first column
        const uint32_t tlane = tmem_base + ((uint32_t)(quarter * 32) << 16) + part;
        const uint32_t free_bar = mapa_shared(bar_accempty, 0);
        const float* own = scales + (part / BK) * C::kScaleHalf + quarter * 32 + lane;
        uint32_t s = 0, phase = 0, sc = 0;     // s: the block's stage; its buffer is s % kBufs
        bool ok = true;
        for (uint32_t u = first; u < units && ok; u += step) {
            int t, nt, e, row, n;
            pair_unit(u, tiles, NT, t, nt);
            groups.tile(t, e, row, n);
            const int r0 = rank * PTH + quarter * 32;      // the warp's first row in the tile
            uint64_t acc[C::kHalf / 2];
#pragma unroll
            for (int j = 0; j < C::kHalf / 2; ++j) acc[j] = 0;
            for (int kb = 0; kb < KB; ++kb) {
                const uint32_t buf = s % kBufs, sbuf = sc & 1;
                const int i = kb % kScaleBlocks;
                // A wait for a block that runs out sets the abort flag; the warp goes on together, and leaves where it
                // votes, at the next four blocks (a vote in every block costs 2 %).
                if (i == 0) {
                    const bool go = mbar_wait(bar_scfull + 8 * sbuf, (sc >> 1) & 1, abort_flag, kErrDrain, &g_fp8_error) &&
                                    !*abort_flag;
                    if (!__all_sync(0xffffffffu, go)) {
                        ok = false;
                        break;
                    }
                }
                mbar_wait(bar_done + 8 * s, phase, abort_flag, kErrDrain, &g_fp8_error);
                tc_fence_after();
                const float f = own[sbuf * C::kScaleBuf + i * kScalePitch];
                const uint64_t f2 = pack2(f, f);
                uint32_t v[kPairLd];
#pragma unroll
                for (int h = 0; h < C::kHalf / kPairLd; ++h) {
                    tmem_load(tlane + buf * PN + h * kPairLd, v);
                    if (h == C::kHalf / kPairLd - 1) {   // everything is read: the buffer may be filled again
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(free_bar + 8 * buf);
                    }
#pragma unroll
                    for (int j = 0; j < kPairLd / 2; ++j)
                        acc[h * kPairLd / 2 + j] = fma2(pack2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), f2,
                                                        acc[h * kPairLd / 2 + j]);
                }
                if (++s == kStages) { s = 0; phase ^= 1; }
                if (i == kScaleBlocks - 1 || kb == KB - 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_scempty + 8 * sbuf);
                    ++sc;
                }
            }
            if (!ok) break;
            const int live = min(32, n - r0), col0 = nt * PN + part;
            const uint32_t buf = sbase + C::kOffEpi + (warp - 4) * kPairEpi;
            if (live > 0 && col0 < p.N) {
                if (p.type == Q8_BF16)
                    store_rows(static_cast<__nv_bfloat16*>(p.y), row + r0, live, col0, p.N, acc, buf, lane);
                else if (p.type == Q8_F16)
                    store_rows(static_cast<__half*>(p.y), row + r0, live, col0, p.N, acc, buf, lane);
                else
                    store_rows(static_cast<float*>(p.y), row + r0, live, col0, p.N, acc, buf, lane);
            }
        }
    }

    __syncthreads();
    if (*abort_flag) {
        const long long t0 = clock64();
        while (clock64() - t0 < (1LL << 22)) __nanosleep(1000);
    }
    tc_fence_before();
    cluster_sync();   // neither CTA frees TMEM or leaves while the other may still use its part
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, 512);
}

// Once per device: the shared-memory limit, and the clusters of two that run at once.
template <int PN>
cudaError_t pair_clusters(int& clusters) {
    using C = Pair8Cfg<PN>;
    static int cached[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && cached[dev] > 0) {
        clusters = cached[dev];
        return cudaSuccess;
    }
    e = cudaFuncSetAttribute(gemm_fp8_pair_kernel<PN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    clusters = device_sm_count() / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * clusters), 1, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, gemm_fp8_pair_kernel<PN>, &cfg);
    if (e != cudaSuccess) return e;
    if (n > 0 && n < clusters) clusters = n;
    if (dev < 64) cached[dev] = clusters;
    return cudaSuccess;
}

template <int PN>
cudaError_t launch_pair(const uint8_t* qa, const uint8_t* qw, PairArgs p, int64_t tiles, cudaStream_t stream) {
    using C = Pair8Cfg<PN>;
    int clusters = 0;
    const cudaError_t e = pair_clusters<PN>(clusters);
    if (e != cudaSuccess) return e;
    CUtensorMap ma, mw;
    if (!make_tma_map_i8(&ma, reinterpret_cast<const int8_t*>(qa), p.rows, p.K, PTH, BK, true) ||
        !make_tma_map_i8(&mw, reinterpret_cast<const int8_t*>(qw), (int64_t)p.E * p.N, p.K, C::kHalf, BK, true))
        return cudaErrorInvalidValue;
    const int64_t units = tiles * ((p.N + PN - 1) / PN);
    if (units < clusters) clusters = (int)units;
    p.most = (uint32_t)units;
    gemm_fp8_pair_kernel<PN><<<2 * clusters, kPairThreads, C::kSmem, stream>>>(ma, mw, p);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_fp8(const uint8_t* qa, const float* sa, const uint8_t* qw, const float* sw,
                            const int32_t* offsets, int64_t rows, int E, int64_t N, int64_t K, void* y,
                            q8_float_type t, cudaStream_t stream) {
    const int64_t per = (rows + E - 1) / E;   // rows of a group, on average
    const int64_t NT = (N + TW - 1) / TW;
    auto tiles = [&](int tn) { return offsets ? rows / tn + (E < rows ? E : rows) : (rows + tn - 1) / tn; };
    // The kernels count tiles in 32 bits, whatever the offsets are (each group at most all rows).
    if (tiles(16) * NT >= (1LL << 31) - 1024 || (rows / 16 + 1) * E >= (1LL << 31)) return cudaErrorNotSupported;
    const SwapArgs p{sa, sw, offsets, (int)rows, E, (int)N, (int)K, 0, 1, y, t, 0};
    if (per > 64) {
        // What a round of tiles costs a K block: 0.47 us for 256 x 256 tiles over 76 pairs, 0.30 us for 256 x 128, 0.37 us
        // for 64 x 128 tiles of the other kernel over 152 CTAs (or fewer, larger clusters); and about six
        // blocks a tile. Measured, wide pairs / narrow pairs / other kernel, us: 100x512x16384 62 / 41 / 15; 128x8192x8192
        // 34 / 25 / 27; 517x2056x4112 25 / 17 / 27; 512x8192x8192 38 / 44 / 91; 2048x4096x4096 38 / 51 / 77; 8192
        // rows of 64 experts, 4096x4096, 268 / 311 / 369. The estimate picks the fastest in each. Where rows of y are
        // not whole 16-byte chunks, a pair's store takes 2.4 us more a tile by words and 5 us more by 16-bit values,
        // which decides for few K blocks (1778x8597x416 fp16 43 / 45 / 32; 7367 rows of 72 experts, 5318x272 bf16,
        // 126 / 159 / 95, but 5312 columns 79 / 95 / 95).
        int pairs = 0, split = 1, clusters = 0;
        double other = 0.0;
        cudaError_t e = pair_clusters<256>(pairs);
        if (e == cudaSuccess) e = swap_plan<32>(tiles(64), N, K, split, clusters, other);
        if (e != cudaSuccess) return e;
        const int64_t row_bytes = N * (t == Q8_F32 ? 4 : 2);
        const double store = row_bytes % 16 == 0 ? 0.0 : row_bytes % 4 == 0 ? 2.4 : 5.0;   // us a wide tile
        auto estimate = [&](int pn, double block) {
            const int64_t rounds = (tiles(PT) * ((N + pn - 1) / pn) + pairs - 1) / pairs;
            return (double)rounds * (block * (double)((K + BK - 1) / BK + 6) + store * pn / 256);
        };
        const double wide = estimate(256, 0.47), narrow = estimate(128, 0.30);
        const PairArgs pa{sa, sw, offsets, (int)rows, E, (int)N, (int)K, y, t, 0};
        if (0.37 * other < wide && 0.37 * other < narrow) return launch_swap<32>(qa, qw, p, tiles(64), stream);
        if (narrow < wide) return launch_pair<128>(qa, qw, pa, tiles(PT), stream);
        return launch_pair<256>(qa, qw, pa, tiles(PT), stream);
    }
    // Groups of unequal size: a tile four times the average leaves few of them more than one.
    const int64_t most = offsets ? 4 * per : per;
    if (most <= 16) return launch_swap<8>(qa, qw, p, tiles(16), stream);
    if (most <= 32) return launch_swap<16>(qa, qw, p, tiles(32), stream);
    return launch_swap<32>(qa, qw, p, tiles(64), stream);
}

cudaError_t read_and_clear_gemm_fp8_error(uint32_t* code) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp8_error, sizeof(v));
    if (e != cudaSuccess) return e;
    *code = v;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_fp8_error, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace q8
