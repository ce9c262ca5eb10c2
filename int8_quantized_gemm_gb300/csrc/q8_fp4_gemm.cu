// Products of 4-bit (e2m1) matrices with a scale for each 16 or 32 K of a row, for one weight matrix or one for each group of
// rows (experts).
//
//   y[m, n] = sa[m] sw[n] sum_b sfa[m, b] sfw[n, b] sum_{k in block b} qa[m, k] qw[n, k]
//
// The tensor core (tcgen05 kind::mxf4nvf4 / mxf4, block_scale) takes the block scales itself, from tensor memory, so that a
// tile's sum over all K stays in its fp32 accumulator; the rows' scales are applied as it is written out. A stage is 256 K: 128
// bytes of codes a row (128-byte swizzle) and the scales in tiles of 128 rows x 4 (512 bytes, tcgen05.cp). The weights'
// scales are stored in such tiles (TMA); the tokens', which may begin at any row of an expert, as rows: a warp turns
// them into tiles on the way to shared memory. In tensor memory every stage has columns of its own for its scales: they are copied
// again only after the stage's barriers have seen the MMAs that read them.
#include <cuda.h>

#include <type_traits>

#include "q8_fp4.h"
#include "q8_fp4_ptx.cuh"
#include "q8_internal.h"
#include "q8_loads.cuh"
#include "q8_tiles.cuh"

namespace q8 {
namespace {

using namespace tc;

__device__ unsigned int g_fp4_error = 0;

// Bounded waits of a whole warp: its lanes agree on how the wait ended, so that none goes on alone to an
// instruction that takes them all.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned code) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, code, &g_fp4_error));
}
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned code) {
    return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort_flag, code, &g_fp4_error));
}

constexpr int kRowBytes = kFp4Span / 2;          // of codes in a stage
constexpr int TW = 128;                          // rows of a tile of scales, and of the MMA's M side
constexpr int kSmemMax = 227 * 1024;

template <int kBlock>
struct Scales {
    static constexpr int kAtoms = 64 / kBlock;              // tiles of 128 rows x 4 scales in a stage: 4 or 2
    static constexpr int kBytes = kAtoms * 512;             // of 128 rows in a stage
    static constexpr int kRow = kFp4Span / kBlock;          // bytes of a row in a stage
    static constexpr int kCols = kAtoms * 4;                // tensor memory columns of 128 rows in a stage
};

// A stage's scales of up to 32 J token rows (J of them a lane), from rows to tiles.
template <int kBlock, int J>
struct TokenScales {
    uint4 a[J];
    // the rows row0 .. row0 + n - 1; nothing (zeros) unless `have`
    __device__ __forceinline__ void load(const uint8_t* sf, int64_t row0, int n, uint32_t pitch, int kb, bool have, int lane) {
        const uint8_t* p = sf + (row0 + lane) * pitch + (size_t)kb * Scales<kBlock>::kRow;
#pragma unroll
        for (int j = 0; j < J; ++j, p += (size_t)32 * pitch) {
            a[j] = make_uint4(0, 0, 0, 0);
            if (have && lane + 32 * j < n) {
                if constexpr (kBlock == 16) {
                    a[j] = load128(p);
                } else {
                    const uint2 v = load64(p);
                    a[j].x = v.x;
                    a[j].y = v.y;
                }
            }
        }
    }
    __device__ __forceinline__ static uint32_t word(const uint4& v, int k) {
        return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
    }
    // `groups`: scales of a row from this stage on; those past the end are not read as numbers (zero codes meet them)
    __device__ __forceinline__ void store(uint32_t dst, int groups, int lane) const {
#pragma unroll
        for (int k = 0; k < Scales<kBlock>::kAtoms; ++k) {
            const int left = groups - 4 * k;
            const uint32_t mask = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = j < J ? word(a[j < J ? j : 0], k) & mask : 0u;
            sts128(dst + k * 512 + lane * 16, make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
};

// One of two scale warps (which = 0, 1: every other stage, so that each has two stages' time for the way from a free stage to
// a full one; pairs of stages a warp, which share a sector of the rows' scales, were 15 % slower with 128 tokens): the stages
// kb0 .. kb1 - 1 of one tile. `s`, `phase`: the ring's state at kb0, moved on; `free_bar`: base of the barriers that a stage
// is free; `put(s)`: address of stage s's tiles; `done(s)`: arrival. Two stages of its own are loaded ahead. False when a
// wait gave up.
template <int kBlock, int J, class Put, class Done>
__device__ __forceinline__ bool feed_scales(const uint8_t* sf, int64_t row0, int n, uint32_t pitch, int groups, int kb0, int kb1,
                                            uint32_t& count, int which, int stages, uint32_t& s, uint32_t& phase,
                                            uint32_t free_bar, volatile int* abort_flag, int lane, Put put, Done done) {
    TokenScales<kBlock, J> set[2];
    int kb = kb0 + (int)((count ^ (uint32_t)which) & 1);       // its first stage here
    uint32_t at = s + (uint32_t)(kb - kb0), ph = phase;
    if (at >= (uint32_t)stages) { at -= stages; ph ^= 1; }
    set[0].load(sf, row0, n, pitch, kb, kb < kb1, lane);
    set[1].load(sf, row0, n, pitch, kb + 2, kb + 2 < kb1, lane);
    bool ok = true;
    while (kb < kb1 && ok) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (kb < kb1 && ok) {
                ok = warp_wait(free_bar + 8 * at, ph, abort_flag, kErrConvEmpty);
                if (ok) {
                    set[i].store(put(at), groups - kb * Scales<kBlock>::kRow, lane);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) done(at);
                    set[i].load(sf, row0, n, pitch, kb + 4, kb + 4 < kb1, lane);
                }
                kb += 2;
                at += 2;
                if (at >= (uint32_t)stages) { at -= stages; ph ^= 1; }
            }
        }
    }
    const uint32_t len = (uint32_t)(kb1 - kb0);
    count += len;
    s += len % (uint32_t)stages;
    phase ^= (len / (uint32_t)stages) & 1;
    if (s >= (uint32_t)stages) { s -= stages; phase ^= 1; }
    return ok;
}

// ------------------------------------------------------------------------ weights on the MMA's M side
// For few tokens a matrix: a tile is 128 weight rows x up to TN = 16 or 32 token rows, so that a weight matrix is read from
// memory once (a group of more tokens than a tile reads it again from L2). Bound by the weights' bytes.
//   warp 0     TMA: weights [128 x 256 codes] with their scales and tokens [n x 256 codes] of each stage
//   warp 1     MMA issuer (N = n rounded up to 16), TMEM
//   warps 2, 3 scales of the stage's tokens, every other stage each
//   warps 4-11 drain: two warps for each quarter of the TMEM lanes (weight rows), half of the tokens each
// With few tiles, a cluster of S CTAs splits a tile's stages; each CTA sends the partial sums of the tokens it does not own
// to the CTA that does (st.async), which adds them in the order of the ranks: the same bits every time, no workspace and no
// second launch. Measured, called one after another from Python with three sets of operands in turn (in brackets in a graph
// with two): 16x28672x8192 25.3 to 25.6 us (24.5), 5.2 TB/s, 0.77 of the measured copy bandwidth (two CTAs share a tile so that
// 224 tiles fill three rounds; launch, set-up, the first load and the last exchange are about 4.5 us); 128 rows of 64 experts,
// 4096 x 4096, blocks of 32, 86.6 to 87.7 us (0.96 on the active weights); 1x4096x4096 6.1 us (5.6).
constexpr int kSwapThreads = 384;
constexpr int kDrainWarps = 8;
constexpr int kBufs = 2;               // accumulator buffers: the next tile's MMAs run while one is written out
constexpr int kMaxStages = 8;          // nine: 16x28672x8192 2 % slower, 128 rows of 64 experts too
constexpr int kTailBytes = 8 * (2 * kMaxStages + 2 * kBufs + 2) + 32 + 4 * (kMaxExperts + 2);

// A value as T to shared memory.
template <class T>
__device__ __forceinline__ void sts_value(uint32_t addr, float f) {
    const T v = from_float<T>(f);
    if constexpr (sizeof(T) == 2)
        asm volatile("st.shared.u16 [%0], %1;\n" ::"r"(addr), "h"(*reinterpret_cast<const uint16_t*>(&v)) : "memory");
    else
        asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(addr), "r"(__float_as_uint(f)) : "memory");
}

constexpr int kSwapTokens = 16;        // of a drain warp, at most
constexpr int kSwapEpi = 2048 + 4 * kSwapTokens;   // of a drain warp: 2 KB of values on their way out, its tokens' scales

// acc[j]: weight row (column of y) col0 + lane, token t0 + j, as store_tokens; y's rows are whole 16-byte chunks. 2 KB of
// tokens x 32 columns at a time are turned round in shared memory, so that a token's columns leave 16 bytes a lane (with
// tiles of 64 tokens and a word a lane instead, 2050 rows of 32 experts took 57 us for 37).
template <class T, int CW>
__device__ __forceinline__ void store_tokens_staged(T* y, int64_t row, int t0, int n, int col0, int N, const float (&acc)[CW],
                                                    uint32_t buf, int split, int rank, int lane) {
    constexpr int kRow = 32 * sizeof(T), kTokens = 2048 / kRow < CW ? 2048 / kRow : CW;   // bytes of a token, tokens of a step
    constexpr int kLanes = kRow / 16, kPass = 32 / kLanes;                               // lanes of a token, tokens of a pass
    const int col = col0 + lane % kLanes * (16 / (int)sizeof(T));
#pragma unroll
    for (int c = 0; c < CW / kTokens; ++c) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            sts_value<T>(buf + j * kRow + lane * (int)sizeof(T), acc[c * kTokens + j]);
        }
        __syncwarp();
        if (col < N) {
#pragma unroll
            for (int i = 0; i < (kTokens + kPass - 1) / kPass; ++i) {
                const int r = i * kPass + lane / kLanes, t = t0 + c * kTokens + r;
                if (r < kTokens && t < n && (split == 1 || ((t / 4) & (split - 1)) == rank))
                    *reinterpret_cast<uint4*>(y + (row + t) * N + col) = lds128(buf + r * kRow + lane % kLanes * 16);
            }
        }
    }
}

struct SwapArgs {
    const uint8_t* sfa;
    const float* sa;
    const float* sw;
    const int32_t* offsets;   // nullptr: one group of all rows
    int rows, E;
    int N, K;
    uint32_t pitch;           // of sfa
    int stages;               // of the ring
    int split;                // CTAs of a cluster, sharing a tile's stages
    void* y;
    q8_float_type type;
    uint32_t most;            // units there can be
};

template <int CW, int kBlock>   // tokens of a drain warp; TN = 2 CW
struct SwapCfg {
    using S = Scales<kBlock>;
    static_assert(CW <= kSwapTokens, "above the room for a drain warp's token scales");
    static constexpr int TN = 2 * CW;
    static constexpr int kBox = TN;                             // token rows of the TMA box
    static constexpr int kOffTokens = TW * kRowBytes;
    static constexpr int kOffSfw = kOffTokens + TN * kRowBytes;
    static constexpr int kOffSfa = kOffSfw + S::kBytes;
    static constexpr int kStage = kOffSfa + S::kBytes;
    static_assert(kStage % 1024 == 0, "swizzled tiles start on 1024 bytes");
    static constexpr uint32_t kId0 = idesc_fp4(TW, 0, kBlock, 0), kId2 = idesc_fp4(TW, 0, kBlock, 2);   // N is added
    static constexpr int kScaleCols = 2 * S::kCols;             // of a stage: weights, then tokens
    static constexpr int kTmemScales = kBufs * TN;
    static constexpr int kTmem = 512;
    static_assert(kTmemScales + kMaxStages * kScaleCols <= kTmem, "above the tensor memory");
    // receive buffer: the groups of four tokens that a CTA owns, from each other CTA
    static int reduce_bytes(int split) { return (split - 1) * ((TN / 4 + split - 1) / split) * TW * 16; }
};

template <int CW, int kBlock>
__global__ void __launch_bounds__(kSwapThreads, 1)
    gemm_fp4_swap_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                         const __grid_constant__ CUtensorMap tmap_sf, SwapArgs p, int reduce_bytes) {
    using C = SwapCfg<CW, kBlock>;
    using S = Scales<kBlock>;
    constexpr int TN = C::TN;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sraw = smem_u32(smem_raw);
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - sraw);
    const uint32_t off_reduce = p.stages * C::kStage;
    const uint32_t off_epi = off_reduce + reduce_bytes;
    const uint32_t off_bar = off_epi + kDrainWarps * kSwapEpi;
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

    const int NT = (p.N + TW - 1) / TW, KB = (p.K + kFp4Span - 1) / kFp4Span;
    const uint32_t first = blockIdx.x / p.split, step = gridDim.x / p.split;
    const int kb0 = KB / p.split * rank + min(rank, KB % p.split);   // this CTA's share of the stages
    const int kb1 = kb0 + KB / p.split + (rank < KB % p.split ? 1 : 0);
    const EarlyGroups groups{p.offsets, cum, p.rows, p.E, TN};

    if (warp == 0) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_sf)) : "memory");
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
            for (int s = 0; s < p.stages; ++s) {
                mbar_init(bar_full + 8 * s, 2);       // the loads and a scale warp
                mbar_init(bar_empty + 8 * s, 1);
            }
            for (int b = 0; b < kBufs; ++b) {
                mbar_init(bar_accfull + 8 * b, 1);
                mbar_init(bar_accempty + 8 * b, kDrainWarps);
            }
            mbar_init(bar_got, 1);
            mbar_init(bar_free, p.split * kDrainWarps);
            *abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        }
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::kTmem);
    depend_wait();
    if (warp == 2) groups.scan(cum, lane);
    tc_fence_before();
    if (p.split > 1) cluster_sync();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t units = groups.units(NT, p.most);

    if (warp == 0) {
        // ---------------------------------------------------------------------------- TMA
        if (elect_one()) {   // one lane for all of it, as of the MMAs: 16x8192x8192 8.5 us, 8.9 with the warp at each stage
            uint32_t s = 0, phase = 1;
            bool ok = true;
            for (uint32_t u = first; u < units && ok; u += step) {
                int e, row, n;
                groups.tile((int)(u / (uint32_t)NT), e, row, n);
                const int nt = (int)(u % (uint32_t)NT), wrow = e * p.N + nt * TW;
                const int sfrow = (e * NT + nt) * KB * (S::kAtoms * 4);     // tiles of scales as rows of 128 bytes
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(bar_empty + 8 * s, phase, abort_flag, kErrProducer, &g_fp4_error)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + s * C::kStage, bar = bar_full + 8 * s;
                    mbar_expect_tx(bar, C::kOffTokens + S::kBytes + C::kBox * kRowBytes);
                    tma_load_2d(dst, &tmap_w, kb * kRowBytes, wrow, bar);
                    tma_load_2d(dst + C::kOffSfw, &tmap_sf, 0, sfrow + kb * (S::kAtoms * 4), bar);
                    tma_load_2d(dst + C::kOffTokens, &tmap_a, kb * kRowBytes, row, bar);
                    if (++s == (uint32_t)p.stages) { s = 0; phase ^= 1; }
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------------------- MMA
        if (elect_one()) {
            uint32_t s = 0, phase = 0, buf = 0, bphase = 1;
            bool ok = true;
            for (uint32_t u = first; u < units && ok; u += step) {
                int e, row, n;
                groups.tile((int)(u / (uint32_t)NT), e, row, n);
                const uint32_t width = (uint32_t)((n + 15) >> 4) << 18;   // N = n rounded up to 16
                const uint32_t id0 = C::kId0 + width, id2 = C::kId2 + width;
                if (!mbar_wait(bar_accempty + 8 * buf, bphase, abort_flag, kErrMmaAcc, &g_fp4_error)) break;
                const uint32_t d = tmem_base + buf * TN;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(bar_full + 8 * s, phase, abort_flag, kErrMmaFull, &g_fp4_error)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = sbase + s * C::kStage;
                    const uint64_t w = smem_desc_sw128(at), a = smem_desc_sw128(at + C::kOffTokens);
                    const uint64_t sfw = smem_desc_scales(at + C::kOffSfw), sfa = smem_desc_scales(at + C::kOffSfa);
                    const uint32_t tw = tmem_base + C::kTmemScales + s * C::kScaleCols, ta = tw + S::kCols;
#pragma unroll
                    for (int k = 0; k < S::kAtoms; ++k) {
                        copy_scales<1>(tw + 4 * k, sfw + 32 * k);
                        copy_scales<1>(ta + 4 * k, sfa + 32 * k);
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const int k = kBlock == 16 ? kk : kk / 2;
                        mma_fp4<kBlock, 1>(d, w + 2 * kk, a + 2 * kk, kBlock == 32 && kk % 2 ? id2 : id0, tw + 4 * k, ta + 4 * k,
                                           kb > kb0 || kk ? 1u : 0u);
                    }
                    mma_commit(bar_empty + 8 * s);
                    if (kb == kb1 - 1) mma_commit(bar_accfull + 8 * buf);
                    if (++s == (uint32_t)p.stages) { s = 0; phase ^= 1; }
                }
                if (++buf == kBufs) { buf = 0; bphase ^= 1; }
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------------------------------- scales
        uint32_t s = 0, phase = 1, count = 0;
        bool ok = true;
        for (uint32_t u = first; u < units && ok; u += step) {
            int e, row, n;
            groups.tile((int)(u / (uint32_t)NT), e, row, n);
            ok = feed_scales<kBlock, 1>(
                p.sfa, row, n, p.pitch, p.K / kBlock, kb0, kb1, count, warp - 2, p.stages, s, phase, bar_empty, abort_flag, lane,
                [&](uint32_t st) { return sbase + st * C::kStage + C::kOffSfa; },
                [&](uint32_t st) { mbar_arrive(bar_full + 8 * st); });
        }
    } else {
        // -------------------------------------------------------------------------- drain
        const int quarter = warp & 3, t0 = ((warp - 4) >> 2) * CW;   // its first token
        const uint32_t tlane = tmem_base + ((uint32_t)(quarter * 32) << 16) + t0;
        const uint32_t epi = sbase + off_epi + (warp - 4) * kSwapEpi;
        float* token_scales = reinterpret_cast<float*>(smem + off_epi + (warp - 4) * kSwapEpi + 2048);
        uint32_t buf = 0, bphase = 0, done = 0;
        for (uint32_t u = first; u < units; u += step, ++done) {
            int e, row, n;
            groups.tile((int)(u / (uint32_t)NT), e, row, n);
            const int col = (int)(u % (uint32_t)NT) * TW + quarter * 32 + lane;   // this thread's weight row
            const float scale = p.sw && col < p.N ? load_float(p.sw + (int64_t)e * p.N + col) : 1.0f;
            if (p.sa) {
                if (lane < CW) token_scales[lane] = t0 + lane < n ? load_float(p.sa + row + t0 + lane) : 0.0f;
                __syncwarp();
            }
            if (!warp_wait(bar_accfull + 8 * buf, bphase, abort_flag, kErrDrain)) break;
            tc_fence_after();
            float acc[CW];
            {
                uint32_t v[CW];
                if (t0 < n) tmem_load(tlane + buf * TN, v);
#pragma unroll
                for (int j = 0; j < CW; ++j) acc[j] = t0 < n ? __uint_as_float(v[j]) : 0.0f;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_accempty + 8 * buf);
            if (++buf == kBufs) { buf = 0; bphase ^= 1; }
            if (p.split > 1) {   // tokens in groups of four: group g is added up by CTA g % split
                const int S4 = p.split, log = __ffs(S4) - 1, groups4 = (n + 3) / 4;
                const int per = (groups4 + S4 - 1) / S4;          // slots of groups in the receive buffer
                const int here = (groups4 - rank + S4 - 1) / S4;  // groups that this CTA owns (may be 0)
                const uint32_t buffer = sbase + off_reduce, lane16 = (quarter * 32 + lane) * 16;
                if (done && !warp_wait_cluster(bar_free, (done - 1) & 1, abort_flag, kErrRelay)) break;
                if (warp == 4 && lane == 0) mbar_expect_tx(bar_got, (S4 - 1) * max(here, 0) * TW * 16);
#pragma unroll
                for (int q = 0; q < CW / 4; ++q) {
                    const int g = t0 / 4 + q, owner = g & (S4 - 1);
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
                    if (g < groups4 && (g & (S4 - 1)) == rank) {
                        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int r = 0; r < S4; ++r) {
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
                if (lane < S4) mbar_arrive_remote(mapa_shared(bar_free, lane));
            }
#pragma unroll
            for (int j = 0; j < CW; j += 4) {
                if (p.sa) {
                    const float4 f = *reinterpret_cast<const float4*>(token_scales + j);
                    acc[j] = __fmul_rn(acc[j], f.x);
                    acc[j + 1] = __fmul_rn(acc[j + 1], f.y);
                    acc[j + 2] = __fmul_rn(acc[j + 2], f.z);
                    acc[j + 3] = __fmul_rn(acc[j + 3], f.w);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j + i] = __fmul_rn(acc[j + i], scale);
            }
            __syncwarp();   // the tokens' scales have been read
            if (t0 < n) {
                auto store = [&](auto* y) {
                    using T = typename std::remove_pointer<decltype(y)>::type;
                    if (p.N * sizeof(T) % 16 == 0)
                        store_tokens_staged<T>(y, row, t0, n, col - lane, p.N, acc, epi, p.split, rank, lane);
                    else
                        store_tokens(y, row, t0, n, col, p.N, acc, p.split, rank, lane);
                };
                if (p.type == Q8_BF16) store(static_cast<__nv_bfloat16*>(p.y));
                else if (p.type == Q8_F16) store(static_cast<__half*>(p.y));
                else store(static_cast<float*>(p.y));
            }
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
template <int CW, int kBlock>
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
    auto* kernel = gemm_fp4_swap_kernel<CW, kBlock>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
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
    e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (fit > 0 && fit < clusters) clusters = fit;
    if (dev < 64) cached[dev][log] = clusters;
    return cudaSuccess;
}

// The split that ends first: rounds of tiles over the clusters, each a part of the stages and a fixed cost of
// about four stages (the exchange and the store). `cost`: in stages of one CTA.
template <int CW, int kBlock>
cudaError_t swap_plan(int64_t tiles, int64_t N, int64_t K, int& split, int& clusters, double& cost) {
    const int64_t units = tiles * ((N + TW - 1) / TW), KB = (K + kFp4Span - 1) / kFp4Span;
    for (int S = 1; S <= 8 && (S == 1 || S * 2 <= KB); S *= 2) {
        int fit = 0;
        const cudaError_t e = swap_clusters<CW, kBlock>(S, fit);
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

// Tensor maps of the codes (rows of K / 2 bytes) and of the weights' tiles of scales (as rows of 128 bytes).
template <int kBlock>
bool make_maps(const Fp4Product& p, int token_box, int weight_box, CUtensorMap& ma, CUtensorMap& mw, CUtensorMap& ms) {
    const int64_t tiles = p.E * ((p.N + TW - 1) / TW) * ((p.K + kFp4Span - 1) / kFp4Span) * Scales<kBlock>::kAtoms;
    return make_tma_map_i8(&ma, reinterpret_cast<const int8_t*>(p.qa), p.rows, p.K / 2, token_box, kRowBytes, true) &&
           make_tma_map_i8(&mw, reinterpret_cast<const int8_t*>(p.qw), p.E * p.N, p.K / 2, weight_box, kRowBytes, true) &&
           make_tma_map_i8(&ms, reinterpret_cast<const int8_t*>(p.sfw), tiles * 4, 128, Scales<kBlock>::kAtoms * 4, 128);
}

template <int CW, int kBlock>
cudaError_t launch_swap(const Fp4Product& g, int64_t tiles, cudaStream_t stream) {
    using C = SwapCfg<CW, kBlock>;
    SwapArgs p{g.sfa, g.sa, g.sw, g.offsets, (int)g.rows, (int)g.E, (int)g.N, (int)g.K, (uint32_t)fp4_pitch(g.K, kBlock), 0, 1,
               g.y, g.type, 0};
    int clusters = 0;
    double cost = 0.0;
    cudaError_t e = swap_plan<CW, kBlock>(tiles, g.N, g.K, p.split, clusters, cost);
    if (e != cudaSuccess) return e;
    p.most = (uint32_t)(tiles * ((g.N + TW - 1) / TW));
    const int reduce = p.split > 1 ? C::reduce_bytes(p.split) : 0;
    const int room = kSmemMax - 1024 - kTailBytes - kDrainWarps * kSwapEpi - reduce;
    p.stages = room / C::kStage < kMaxStages ? room / C::kStage : kMaxStages;
    CUtensorMap ma, mw, ms;
    if (!make_maps<kBlock>(g, C::kBox, TW, ma, mw, ms)) return cudaErrorInvalidValue;
    e = launch_dependent(gemm_fp4_swap_kernel<CW, kBlock>, dim3((unsigned)(clusters * p.split)), dim3(kSwapThreads),
                         1024 + p.stages * C::kStage + reduce + kDrainWarps * kSwapEpi + kTailBytes, p.split, stream, ma, mw, ms, p,
                         reduce);
    note_launch();
    return e;
}

// ------------------------------------------------------------------ tokens on the MMA's M side, CTA pairs
// For many tokens: a cluster of two CTAs shares a tile of 256 token rows x 256 weight rows
// (cta_group::2; each CTA loads half of both, and the scales of its own token rows and of all weight rows of the tile, and
// holds its 128 token rows' accumulators). Per CTA:
//   warp 0     TMA: tokens [128 x 256 codes], weights [128 x 256 codes], the weights' scales of each stage, completing on the
//              even CTA's barrier
//   warp 1     even CTA: pair MMA issuer; TMEM in both
//   warps 2, 3 scales of the CTA's token rows, every other stage each
//   warps 4-11 drain: a TMEM lane is a token row; two warps for each quarter of the lanes, 128 columns each
// The accumulator takes 256 of the 512 TMEM columns and five stages' scales 240, so there is one: the next tile's MMAs wait
// until the drain warps have read it into registers, and run while they write it out. Measured: 8192x8192x16384 306 us from a
// cool start (7.2 PFLOP/s, 3.8 times the measured bf16 rate), 348 to 357 us back to back, where the power cap holds the SM clock
// near 1.5 GHz; blocks of 32 294 and 317 to 322 us. A stage takes 525 to 540 clocks there against 512 of MMA; without the loads 514,
// and as many more clocks a second (252 us with neither loads nor stores: wrong results), so it is the power of what is moved
// that costs. A tile costs some 2500 clocks besides: the hand-over of the accumulator about half, the rest waits for loads
// behind the burst of stores (8192x8192x4096 95 us, 81 without its stores: wrong results). Tried: stores paced over the tile
// (no gain), 64-byte boxes (8192x8192x1024 50 us for 47), 32 bytes of a row from each lane without staging (10 %), the first
// scales' copies ahead of the accumulator's wait (3 %), one wait for both TMEM loads and scales' copies between the MMAs
// (nothing), the weights' scales multicast to the pair (nothing).
constexpr int PT = 256, PTH = 128, PN = 256;   // tile: tokens, tokens of a CTA, weight rows
constexpr int kPairDrain = 8;                    // drain warps
constexpr int kPairThreads = 128 + 32 * kPairDrain;
constexpr int kPairRegsLow = 88, kPairRegsHigh = 208;
static_assert(128 * kPairRegsLow + 32 * kPairDrain * kPairRegsHigh <= kPairThreads * (65536 / kPairThreads / 8 * 8),
              "above the launch's registers");
constexpr int kPairEpi = 4096;                   // of a drain warp: 32 rows x 128 bytes

template <int kBlock>
struct PairCfg {
    using S = Scales<kBlock>;
    static constexpr int kHalf = PN / 2;                      // weight rows of a CTA; columns of a drain warp
    static constexpr int kOffW = PTH * kRowBytes;
    static constexpr int kOffSfw = kOffW + kHalf * kRowBytes;
    static constexpr int kOffSfa = kOffSfw + PN / TW * S::kBytes;
    static constexpr int kStage = kOffSfa + S::kBytes;
    static_assert(kStage % 1024 == 0, "swizzled tiles start on 1024 bytes");
    static constexpr int kLoad = kOffSfa;                     // bytes of a CTA's loads
    static constexpr int kStages = 5;
    static constexpr int kBufs = 1;                           // accumulator buffers, beside the scales' columns
    static constexpr uint32_t kId0 = idesc_fp4(PT, PN, kBlock, 0), kId2 = idesc_fp4(PT, PN, kBlock, 2);
    static constexpr int kScaleCols = S::kCols + PN / TW * S::kCols;    // tokens, then weights
    static constexpr int kTmemScales = kBufs * PN;
    static_assert(kTmemScales + kStages * kScaleCols <= 512, "above the tensor memory");
    static constexpr int kOffEpi = kStages * kStage;
    static constexpr int kOffCol = kOffEpi + kPairDrain * kPairEpi;     // the tile's column scales
    static constexpr int kOffBar = kOffCol + PN * 4;
    static constexpr int kBars = 2 * kStages + 2 * kBufs;
    static constexpr int kSmem = 1024 + kOffBar + 8 * kBars + 32 + 4 * (kMaxExperts + 2);
    static_assert(kSmem <= kSmemMax, "above the shared memory of one CTA");
};

struct PairArgs {
    const uint8_t* sfa;
    const float* sa;
    const float* sw;
    const int32_t* offsets;
    int rows, E, N, K;
    uint32_t pitch;
    void* y;
    q8_float_type type;
    bool tma_out;    // rows of y are whole 16-byte chunks
    uint32_t most;   // units there can be
};

// A drain warp's 32 whole rows x 2 NC columns (one row a lane) to y: 128 bytes of each row at a time are staged in shared
// memory (128-byte swizzle) and leave by TMA, which cuts off columns past N.
template <class T, int NC>
__device__ __forceinline__ void store_rows_tma(const CUtensorMap* map, int row0, int col0, int N, const uint64_t (&acc)[NC],
                                               uint32_t buf, int lane) {
    constexpr int kCols = 128 / sizeof(T);         // columns of a step
#pragma unroll
    for (int c = 0; c < 2 * NC / kCols; ++c) {
        if (lane == 0) bulk_wait_read_all();      // the step before has left the buffer
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 2) {
                    const float2 f = unpack2(acc[c * 32 + j * 4 + i]);
                    w[i] = pack16<T>(f.x, f.y);
                } else {
                    const float2 f = unpack2(acc[c * 16 + j * 2 + i / 2]);
                    w[i] = __float_as_uint(i & 1 ? f.y : f.x);
                }
            }
            sts128(buf + lane * 128 + ((j ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && col0 + c * kCols < N) {
            tma_store_2d(map, buf, col0 + c * kCols, row0);
            bulk_commit();
        }
    }
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The four drain warps of one half of the columns; all of them learn whether one has given up.
__device__ __forceinline__ void part_sync(int id) { asm volatile("bar.sync %0, 128;\n" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool part_any(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\n"
        "setp.ne.u32 p, %2, 0;\n"
        "bar.red.or.pred q, %1, 128, p;\n"
        "selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(id), "r"(v ? 1u : 0u)
        : "memory");
    return r != 0;
}

template <int kBlock>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                         const __grid_constant__ CUtensorMap tmap_sf, const __grid_constant__ CUtensorMap tmap_y, PairArgs p) {
    using C = PairCfg<kBlock>;
    using S = Scales<kBlock>;
    constexpr int kStages = C::kStages, kBufs = C::kBufs;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sraw = smem_u32(smem_raw);
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - sraw);
    const uint32_t bar_full = sbase + C::kOffBar;             // used in the even CTA: both CTAs' loads and scales
    const uint32_t bar_done = bar_full + 8 * kStages;          // both CTAs: the pair MMA's commit
    const uint32_t bar_accfull = bar_done + 8 * kStages;       // both CTAs: a tile's last commit
    const uint32_t bar_accempty = bar_accfull + 8 * kBufs;     // used in the even CTA: both CTAs' drain warps
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 8 * C::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* cum = reinterpret_cast<int*>(tmem_slot + 2);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar_full + 8 * s, 3);      // the loads and a scale warp of each CTA
            mbar_init(bar_done + 8 * s, 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            mbar_init(bar_accfull + 8 * b, 1);
            mbar_init(bar_accempty + 8 * b, 2 * kPairDrain);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_sf)) : "memory");
    }
    const EarlyGroups groups{p.offsets, cum, p.rows, p.E, PT};
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
    depend_wait();
    if (warp == 2) groups.scan(cum, lane);
    tc_fence_before();
    cluster_sync();   // barriers of both CTAs initialised, TMEM allocated in both
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int NT = (p.N + PN - 1) / PN, NB = (p.N + TW - 1) / TW, KB = (p.K + kFp4Span - 1) / kFp4Span;
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
                // A half without a token (or weight) row is loaded from past the end of the tensor: zeros
                const int arow = rank * PTH < n ? row + rank * PTH : p.rows;
                const int wrow = nt * PN + rank * C::kHalf < p.N ? e * p.N + nt * PN + rank * C::kHalf : p.E * p.N;
                const int sfrow = (e * NB + nt * (PN / TW)) * KB * (S::kAtoms * 4), sfstep = KB * (S::kAtoms * 4);
                for (int kb = 0; kb < KB; ++kb) {
                    if (!warp_wait(bar_done + 8 * s, phase, abort_flag, kErrProducer)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + s * C::kStage;
                    if (elect_one()) {
                        if (rank == 0) mbar_expect_tx(bar_full + 8 * s, 2 * C::kLoad);
                        tma_load_2d_pair(dst, &tmap_a, kb * kRowBytes, arow, full0 + 8 * s);
                        tma_load_2d_pair(dst + C::kOffW, &tmap_w, kb * kRowBytes, wrow, full0 + 8 * s);
#pragma unroll
                        for (int j = 0; j < PN / TW; ++j)
                            tma_load_2d_pair(dst + C::kOffSfw + j * S::kBytes, &tmap_sf, 0,
                                             sfrow + j * sfstep + kb * (S::kAtoms * 4), full0 + 8 * s);
                    }
                    __syncwarp();
                    if (++s == kStages) { s = 0; phase ^= 1; }
                }
            }
        } else if (warp == 1 && rank == 0) {
            // ------------------------------------------------------------------------ MMA
            constexpr uint32_t id0 = C::kId0, id2 = C::kId2;
            uint32_t s = 0, phase = 0, buf = 0, bphase = 1;
            bool ok = true;
            for (uint32_t u = first; u < units && ok; u += step) {
                if (!warp_wait_cluster(bar_accempty + 8 * buf, bphase, abort_flag, kErrMmaAcc)) break;
                const uint32_t d = tmem_base + buf * PN;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!warp_wait_cluster(bar_full + 8 * s, phase, abort_flag, kErrMmaFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = sbase + s * C::kStage;
                    const uint64_t a = smem_desc_sw128(at), w = smem_desc_sw128(at + C::kOffW);
                    const uint64_t sfa = smem_desc_scales(at + C::kOffSfa), sfw = smem_desc_scales(at + C::kOffSfw);
                    const uint32_t ta = tmem_base + C::kTmemScales + s * C::kScaleCols, tw = ta + S::kCols;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < S::kAtoms; ++k) {
                            copy_scales<2>(ta + 4 * k, sfa + 32 * k);
#pragma unroll
                            for (int j = 0; j < PN / TW; ++j)
                                copy_scales<2>(tw + (k * (PN / TW) + j) * 4, sfw + (j * S::kAtoms + k) * 32);
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const int k = kBlock == 16 ? kk : kk / 2;
                            mma_fp4<kBlock, 2>(d, a + 2 * kk, w + 2 * kk, kBlock == 32 && kk % 2 ? id2 : id0, ta + 4 * k,
                                               tw + k * (PN / TW) * 4, kb || kk ? 1u : 0u);
                        }
                        mma_commit_pair(bar_done + 8 * s, 3);
                        if (kb == KB - 1) mma_commit_pair(bar_accfull + 8 * buf, 3);
                    }
                    __syncwarp();
                    if (++s == kStages) { s = 0; phase ^= 1; }
                }
                if (++buf == kBufs) { buf = 0; bphase ^= 1; }
            }
        } else if (warp >= 2) {
            // --------------------------------------------------------------------- scales
            const uint32_t full0 = mapa_shared(bar_full, 0);
            uint32_t s = 0, phase = 1, count = 0;
            bool ok = true;
            for (uint32_t u = first; u < units && ok; u += step) {
                int t, nt, e, row, n;
                pair_unit(u, tiles, NT, t, nt);
                groups.tile(t, e, row, n);
                ok = feed_scales<kBlock, 4>(
                    p.sfa, (int64_t)row + rank * PTH, n - rank * PTH, p.pitch, p.K / kBlock, 0, KB, count, warp - 2, kStages, s,
                    phase, bar_done, abort_flag, lane, [&](uint32_t st) { return sbase + st * C::kStage + C::kOffSfa; },
                    [&](uint32_t st) { mbar_arrive_remote(full0 + 8 * st); });
            }
        }
    } else {
        // ---------------------------------------------------------------------------- drain
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kPairRegsHigh));
        const int quarter = warp & 3, part = ((warp - 4) >> 2) * C::kHalf;   // its first column
        const uint32_t tlane = tmem_base + ((uint32_t)(quarter * 32) << 16) + part;
        const uint32_t free_bar = mapa_shared(bar_accempty, 0);
        float* cols = reinterpret_cast<float*>(smem + C::kOffCol) + part;   // of the four warps of these columns
        const uint32_t epi = sbase + C::kOffEpi + (warp - 4) * kPairEpi;
        uint32_t buf = 0, bphase = 0;
        const int r0 = rank * PTH + quarter * 32;      // the warp's first row in a tile
        // A tile's place and this thread's part of its scales, the row's and one of the columns'. They are fetched while the
        // tile before is written out.
        const int own = quarter * 32 + lane;           // its column scale
        struct {
            int row, live, col0;
            float f, w;
        } next;
        auto fetch = [&](uint32_t u) {
            int t, nt, e, row, n;
            pair_unit(u, tiles, NT, t, nt);
            groups.tile(t, e, row, n);
            next.row = row + r0;
            next.live = min(32, n - r0);
            next.col0 = nt * PN + part;
            next.f = p.sa && lane < next.live ? load_float(p.sa + next.row + lane) : 1.0f;
            if (p.sw)
                next.w = own < C::kHalf && next.col0 + own < p.N ? load_float(p.sw + (int64_t)e * p.N + next.col0 + own) : 0.0f;
        };
        if (first < units) fetch(first);
        for (uint32_t u = first; u < units; u += step) {
            const int row = next.row, live = next.live, col0 = next.col0;
            const uint64_t f2 = pack2(next.f, next.f);
            if (p.sw && own < C::kHalf) cols[own] = next.w;   // read after part_any
            // A warp that gives up leaves with the three that share its column scales: they wait for one another.
            const bool ok = warp_wait(bar_accfull + 8 * buf, bphase, abort_flag, kErrDrain);
            if (p.sw ? part_any(1 + part / C::kHalf, !ok) : !ok) break;
            tc_fence_after();
            uint64_t acc[C::kHalf / 2];
            uint32_t v[C::kHalf / 64][64];
#pragma unroll
            for (int h = 0; h < C::kHalf / 64; ++h) tmem_load(tlane + buf * PN + h * 64, v[h]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(free_bar + 8 * buf);
            if (++buf == kBufs) { buf = 0; bphase ^= 1; }
            if (u + step < units) fetch(u + step);
#pragma unroll
            for (int h = 0; h < C::kHalf / 32; ++h) {
                float4 w[8];
                if (p.sw)
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = reinterpret_cast<const float4*>(cols + 32 * h)[j];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t* from = &v[h / 2][h % 2 * 32 + 2 * j];
                    uint64_t x = mul2(pack2(__uint_as_float(from[0]), __uint_as_float(from[1])), f2);
                    if (p.sw) x = mul2(x, j % 2 ? pack2(w[j / 2].z, w[j / 2].w) : pack2(w[j / 2].x, w[j / 2].y));
                    acc[16 * h + j] = x;
                }
            }
            if (p.sw) part_sync(1 + part / C::kHalf);   // the column scales have been read
            auto store = [&](auto* y) {
                using T = typename std::remove_pointer<decltype(y)>::type;
                if (live == 32 && p.tma_out) {
                    store_rows_tma<T>(&tmap_y, row, col0, p.N, acc, epi, lane);
                } else {
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
                    store_rows(y, row, live, col0, p.N, acc, epi, lane);
                }
            };
            if (live > 0 && col0 < p.N) {
                if (p.type == Q8_BF16) store(static_cast<__nv_bfloat16*>(p.y));
                else if (p.type == Q8_F16) store(static_cast<__half*>(p.y));
                else store(static_cast<float*>(p.y));
            }
        }
        if (lane == 0) bulk_wait_all();   // shared memory outlives the stores from it
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

// Once per kernel and device: the shared-memory limit, and the clusters of two that run at once.
template <class Kernel>
cudaError_t clusters_of_two(Kernel* kernel, int smem, int (&cached)[64], int& clusters) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && cached[dev] > 0) {
        clusters = cached[dev];
        return cudaSuccess;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    clusters = device_sm_count() / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * clusters), 1, 1);
    cfg.blockDim = dim3(kPairThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (n > 0 && n < clusters) clusters = n;
    if (dev < 64) cached[dev] = clusters;
    return cudaSuccess;
}

template <int kBlock>
cudaError_t pair_clusters(int& clusters) {
    static int cached[64] = {0};
    return clusters_of_two(gemm_fp4_pair_kernel<kBlock>, PairCfg<kBlock>::kSmem, cached, clusters);
}

template <int kBlock>
cudaError_t launch_pair(const Fp4Product& g, int64_t tiles, cudaStream_t stream) {
    using C = PairCfg<kBlock>;
    int clusters = 0;
    cudaError_t e = pair_clusters<kBlock>(clusters);
    if (e != cudaSuccess) return e;
    CUtensorMap ma, mw, ms;
    if (!make_maps<kBlock>(g, PTH, C::kHalf, ma, mw, ms)) return cudaErrorInvalidValue;
    const int64_t units = tiles * ((g.N + PN - 1) / PN);
    if (units < clusters) clusters = (int)units;
    const bool tma_out = g.N * (g.type == Q8_F32 ? 4 : 2) % 16 == 0;
    CUtensorMap my = ma;
    if (tma_out && !make_tma_map_out(&my, g.y, g.type == Q8_F32 ? kMapF32 : kMapBF16, g.rows, g.N)) return cudaErrorInvalidValue;
    const PairArgs p{g.sfa, g.sa, g.sw, g.offsets, (int)g.rows, (int)g.E, (int)g.N, (int)g.K, (uint32_t)fp4_pitch(g.K, kBlock),
                     g.y, g.type, tma_out, (uint32_t)units};
    e = launch_dependent(gemm_fp4_pair_kernel<kBlock>, dim3((unsigned)(2 * clusters)), dim3(kPairThreads), C::kSmem, 0, stream, ma,
                         mw, ms, my, p);
    note_launch();
    return e;
}

// ------------------------------------------------------------------ weights on the MMA's M side, CTA pairs
// For some tens of tokens a matrix: a cluster of two CTAs shares a tile of 256 weight rows x up to 128 token rows
// (cta_group::2; each CTA loads half of both, the scales of its own weight rows and of all tokens of the tile, and
// holds its 128 weight rows' accumulators). The MMA's N is the tile's tokens rounded up to 16, so that the last tile of an expert
// costs what its tokens do. Per CTA:
//   warp 0     TMA: weights [128 x 256 codes] with their scales, tokens [N / 2 x 256 codes] of each stage, completing on the even
//              CTA's barrier
//   warp 1     even CTA: pair MMA issuer; TMEM in both
//   warps 2, 3 scales of the tile's tokens, every other stage each
//   warps 4-11 drain: a TMEM lane is a weight row (a column of y); two warps for each quarter of the lanes, 64 tokens each
// Bound by the weights' bytes, or by latencies where there is one round of tiles. Measured, called one after another from Python
// with three sets of operands in turn (in a graph with two in brackets): 2050 rows of 32 experts, 4096 x 2048, 32.9 to 33.3 us
// (32.5), 5.2 TB/s, 2048 rows of 64, 4096 x 4096, 97 us (99), 6.4 TB/s, 64x8192x8192 12.9 us (11.0: L2 holds two sets), 256x8192x8192
// 15.3 to 15.5 us (14.0). With
// 256 tokens a tile it would do the work of the pairs above with less waste in experts' last tiles, but the scales of 256
// token rows in each CTA take longer than the MMAs (8192x8192x4096 130 us against 95).
constexpr int TWP = 256, TNP = 128;               // weight rows of a tile, token rows at most
constexpr int kWideEpi = 2048;                    // of a drain warp

template <int kBlock>
struct WideCfg {
    using S = Scales<kBlock>;
    static constexpr int kHalf = TNP / 2;                     // token rows of a CTA at most; tokens of a drain warp
    static constexpr int kBox = 32;                           // token rows of a TMA box
    static constexpr int kOffTokens = TW * kRowBytes;
    static constexpr int kOffSfw = kOffTokens + kHalf * kRowBytes;
    static constexpr int kOffSfa = kOffSfw + S::kBytes;
    static constexpr int kStage = kOffSfa + S::kBytes;
    static_assert(kStage % 1024 == 0 && kHalf % kBox == 0, "swizzled tiles start on 1024 bytes");
    static constexpr int kStages = 6;                         // five or seven: 2 % slower for 128x8192x8192
    static constexpr int kBufs = 2;                           // accumulator buffers, beside the scales' columns
    static constexpr uint32_t kId0 = idesc_fp4(TWP, 0, kBlock, 0), kId2 = idesc_fp4(TWP, 0, kBlock, 2);   // N is added
    static constexpr int kScaleCols = 2 * S::kCols;           // weights, then tokens
    static constexpr int kTmemScales = kBufs * TNP;
    static_assert(kTmemScales + kStages * kScaleCols <= 512, "above the tensor memory");
    static constexpr int kOffEpi = kStages * kStage;
    static constexpr int kOffTok = kOffEpi + kPairDrain * kWideEpi;     // the tokens' row scales
    static constexpr int kOffBar = kOffTok + TNP * 4;
    static constexpr int kBars = 2 * kStages + 2 * kBufs;
    static constexpr int kSmem = 1024 + kOffBar + 8 * kBars + 32 + 4 * (kMaxExperts + 2);
    static_assert(kSmem <= kSmemMax, "above the shared memory of one CTA");
};

// acc[j]: weight row (column of y) col0 + lane, token t0 + j; y's rows are whole 16-byte chunks. 2 KB of tokens x 32 columns
// at a time are turned round in shared memory and leave by TMA, the last tokens of an expert 16 bytes a lane.
template <class T, int NC>
__device__ __forceinline__ void store_columns(const CUtensorMap* map, T* y, int row, int live, int col0, int N,
                                              const float (&acc)[NC], uint32_t buf, int lane) {
    constexpr int kRow = 32 * sizeof(T), kTokens = 2048 / kRow;      // bytes of a token, tokens of a step
    constexpr int kLanes = kRow / 16, kPass = 32 / kLanes;           // lanes of a token, tokens of a pass
    if (col0 >= N) return;
#pragma unroll
    for (int c = 0; c < NC / kTokens; ++c) {
        if (c * kTokens >= live) break;
        if (lane == 0) bulk_wait_read_all();      // the step before has left the buffer
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            sts_value<T>(buf + j * kRow + lane * (int)sizeof(T), acc[c * kTokens + j]);
        }
        if (live - c * kTokens >= kTokens) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(map, buf, col0, row + c * kTokens);
                bulk_commit();
            }
        } else {
            __syncwarp();
            const int col = col0 + lane % kLanes * (16 / (int)sizeof(T));
            for (int r = lane / kLanes; r < live - c * kTokens; r += kPass)
                if (col < N)
                    *reinterpret_cast<uint4*>(y + (int64_t)(row + c * kTokens + r) * N + col) =
                        lds128(buf + r * kRow + lane % kLanes * 16);
        }
    }
}

template <int kBlock>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    gemm_fp4_wide_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_w,
                         const __grid_constant__ CUtensorMap tmap_sf, const __grid_constant__ CUtensorMap tmap_y, PairArgs p) {
    using C = WideCfg<kBlock>;
    using S = Scales<kBlock>;
    constexpr int kStages = C::kStages, kBufs = C::kBufs;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t sraw = smem_u32(smem_raw);
    const uint32_t sbase = (sraw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (sbase - sraw);
    const uint32_t bar_full = sbase + C::kOffBar;             // used in the even CTA: both CTAs' loads and scales
    const uint32_t bar_done = bar_full + 8 * kStages;          // both CTAs: the pair MMA's commit
    const uint32_t bar_accfull = bar_done + 8 * kStages;       // both CTAs: a tile's last commit
    const uint32_t bar_accempty = bar_accfull + 8 * kBufs;     // used in the even CTA: both CTAs' drain warps
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 8 * C::kBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* cum = reinterpret_cast<int*>(tmem_slot + 2);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar_full + 8 * s, 3);      // the loads and a scale warp of each CTA
            mbar_init(bar_done + 8 * s, 1);
        }
        for (int b = 0; b < kBufs; ++b) {
            mbar_init(bar_accfull + 8 * b, 1);
            mbar_init(bar_accempty + 8 * b, 2 * kPairDrain);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_w)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&tmap_sf)) : "memory");
    }
    const EarlyGroups groups{p.offsets, cum, p.rows, p.E, TNP};
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
    depend_wait();
    if (warp == 2) groups.scan(cum, lane);
    tc_fence_before();
    cluster_sync();   // barriers of both CTAs initialised, TMEM allocated in both
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int NT = (p.N + TWP - 1) / TWP, NB = (p.N + TW - 1) / TW, KB = (p.K + kFp4Span - 1) / kFp4Span;
    const int tiles = cum[p.E];
    const uint32_t units = groups.units(NT, p.most), first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kPairRegsLow));
        if (warp == 0) {
            // ------------------------------------------------------------------------ TMA
            if (elect_one()) {   // one lane for all of it, as of the MMAs: 64x8192x8192 10.9 us, 11.8 with the warp at each stage
                const uint32_t full0 = mapa_shared(bar_full, 0);
                uint32_t s = 0, phase = 1;
                bool ok = true;
                for (uint32_t u = first; u < units && ok; u += step) {
                    int t, nt, e, row, n;
                    pair_unit(u, tiles, NT, t, nt);
                    groups.tile(t, e, row, n);
                    const int half = ((n + 15) >> 4) << 3, boxes = (half + C::kBox - 1) / C::kBox;   // tokens of a CTA
                    const int arow = row + rank * half;
                    // A half without a weight row is loaded from past the end of the tensor: zeros
                    const int wrow = nt * TWP + rank * TW < p.N ? e * p.N + nt * TWP + rank * TW : p.E * p.N;
                    const int sfrow = (e * NB + nt * 2 + rank) * KB * (S::kAtoms * 4);
                    const uint32_t bytes = 2 * (C::kOffTokens + S::kBytes + boxes * C::kBox * kRowBytes);
                    for (int kb = 0; kb < KB; ++kb) {
                        if (!mbar_wait(bar_done + 8 * s, phase, abort_flag, kErrProducer, &g_fp4_error)) {
                            ok = false;
                            break;
                        }
                        const uint32_t dst = sbase + s * C::kStage;
                        if (rank == 0) mbar_expect_tx(bar_full + 8 * s, bytes);
                        tma_load_2d_pair(dst, &tmap_w, kb * kRowBytes, wrow, full0 + 8 * s);
                        tma_load_2d_pair(dst + C::kOffSfw, &tmap_sf, 0, sfrow + kb * (S::kAtoms * 4), full0 + 8 * s);
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d_pair(dst + C::kOffTokens + b * C::kBox * kRowBytes, &tmap_a, kb * kRowBytes,
                                             arow + b * C::kBox, full0 + 8 * s);
                        if (++s == kStages) { s = 0; phase ^= 1; }
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1 && rank == 0) {
            // ------------------------------------------------------------------------ MMA
            if (elect_one()) {
                uint32_t s = 0, phase = 0, buf = 0, bphase = 1;
                bool ok = true;
                for (uint32_t u = first; u < units && ok; u += step) {
                    int t, nt, e, row, n;
                    pair_unit(u, tiles, NT, t, nt);
                    groups.tile(t, e, row, n);
                    const uint32_t width = (uint32_t)((n + 15) >> 4) << 18;   // N = n rounded up to 16
                    const uint32_t id0 = C::kId0 + width, id2 = C::kId2 + width;
                    if (!mbar_wait_cluster(bar_accempty + 8 * buf, bphase, abort_flag, kErrMmaAcc, &g_fp4_error)) break;
                    const uint32_t d = tmem_base + buf * TNP;
                    for (int kb = 0; kb < KB; ++kb) {
                        if (!mbar_wait_cluster(bar_full + 8 * s, phase, abort_flag, kErrMmaFull, &g_fp4_error)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t at = sbase + s * C::kStage;
                        const uint64_t w = smem_desc_sw128(at), a = smem_desc_sw128(at + C::kOffTokens);
                        const uint64_t sfw = smem_desc_scales(at + C::kOffSfw), sfa = smem_desc_scales(at + C::kOffSfa);
                        const uint32_t tw = tmem_base + C::kTmemScales + s * C::kScaleCols, ta = tw + S::kCols;
#pragma unroll
                        for (int k = 0; k < S::kAtoms; ++k) {
                            copy_scales<2>(tw + 4 * k, sfw + 32 * k);
                            copy_scales<2>(ta + 4 * k, sfa + 32 * k);
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const int k = kBlock == 16 ? kk : kk / 2;
                            mma_fp4<kBlock, 2>(d, w + 2 * kk, a + 2 * kk, kBlock == 32 && kk % 2 ? id2 : id0, tw + 4 * k,
                                               ta + 4 * k, kb || kk ? 1u : 0u);
                        }
                        mma_commit_pair(bar_done + 8 * s, 3);
                        if (kb == KB - 1) mma_commit_pair(bar_accfull + 8 * buf, 3);
                        if (++s == kStages) { s = 0; phase ^= 1; }
                    }
                    if (++buf == kBufs) { buf = 0; bphase ^= 1; }
                }
            }
            __syncwarp();
        } else if (warp >= 2) {
            // --------------------------------------------------------------------- scales
            const uint32_t full0 = mapa_shared(bar_full, 0);
            uint32_t s = 0, phase = 1, count = 0;
            bool ok = true;
            for (uint32_t u = first; u < units && ok; u += step) {
                int t, nt, e, row, n;
                pair_unit(u, tiles, NT, t, nt);
                groups.tile(t, e, row, n);
                ok = feed_scales<kBlock, TNP / 32>(
                    p.sfa, row, n, p.pitch, p.K / kBlock, 0, KB, count, warp - 2, kStages, s, phase, bar_done, abort_flag, lane,
                    [&](uint32_t st) { return sbase + st * C::kStage + C::kOffSfa; },
                    [&](uint32_t st) { mbar_arrive_remote(full0 + 8 * st); });
            }
        }
    } else {
        // ---------------------------------------------------------------------------- drain
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kPairRegsHigh));
        const int quarter = warp & 3, t0 = ((warp - 4) >> 2) * C::kHalf, id = 1 + t0 / C::kHalf;   // its first token
        const uint32_t tlane = tmem_base + ((uint32_t)(quarter * 32) << 16) + t0;
        const uint32_t free_bar = mapa_shared(bar_accempty, 0);
        float* token_scales = reinterpret_cast<float*>(smem + C::kOffTok) + t0;   // of the four warps of these tokens
        const uint32_t epi = sbase + C::kOffEpi + (warp - 4) * kWideEpi;
        const int own = quarter * 32 + lane;           // its token's scale; its weight row in the CTA's half
        uint32_t buf = 0, bphase = 0;
        // A tile's place and this thread's part of its scales. They are fetched while the tile before is written out.
        struct {
            int row, live, col0;
            float f, w;
        } next;
        auto fetch = [&](uint32_t u) {
            int t, nt, e, row, n;
            pair_unit(u, tiles, NT, t, nt);
            groups.tile(t, e, row, n);
            next.row = row + t0;
            next.live = min(C::kHalf, n - t0);
            next.col0 = nt * TWP + rank * TW + quarter * 32;
            const int col = next.col0 + lane;
            next.w = p.sw && col < p.N ? load_float(p.sw + (int64_t)e * p.N + col) : 1.0f;
            if (p.sa) next.f = own < next.live ? load_float(p.sa + next.row + own) : 0.0f;
        };
        if (first < units) fetch(first);
        for (uint32_t u = first; u < units; u += step) {
            const int row = next.row, live = next.live, col0 = next.col0;
            const float scale = next.w;
            if (p.sa && own < C::kHalf) token_scales[own] = next.f;   // read after part_any
            // A warp that gives up leaves with the three that share its tokens' scales: they wait for one another.
            const bool ok = warp_wait(bar_accfull + 8 * buf, bphase, abort_flag, kErrDrain);
            if (p.sa ? part_any(id, !ok) : !ok) break;
            tc_fence_after();
            float acc[C::kHalf];
            if (live > 0) {
                uint32_t v[C::kHalf];
                tmem_load(tlane + buf * TNP, v);
#pragma unroll
                for (int j = 0; j < C::kHalf; ++j) acc[j] = __uint_as_float(v[j]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(free_bar + 8 * buf);
            if (++buf == kBufs) { buf = 0; bphase ^= 1; }
            if (u + step < units) fetch(u + step);
            if (live > 0) {
#pragma unroll
                for (int h = 0; h < C::kHalf / 32; ++h) {
                    float4 w[8];
                    if (p.sa)
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = reinterpret_cast<const float4*>(token_scales + 32 * h)[j];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float4& f = w[j / 4];
                        float x = acc[32 * h + j];
                        if (p.sa) x = __fmul_rn(x, j % 4 == 0 ? f.x : j % 4 == 1 ? f.y : j % 4 == 2 ? f.z : f.w);
                        acc[32 * h + j] = __fmul_rn(x, scale);
                    }
                }
            }
            if (p.sa) part_sync(id);   // the tokens' scales have been read
            auto store = [&](auto* y) {
                using T = typename std::remove_pointer<decltype(y)>::type;
                if (p.tma_out) store_columns<T>(&tmap_y, y, row, live, col0, p.N, acc, epi, lane);
                else store_tokens(y, row, 0, live, col0 + lane, p.N, acc, 1, 0, lane);
            };
            if (live > 0) {
                if (p.type == Q8_BF16) store(static_cast<__nv_bfloat16*>(p.y));
                else if (p.type == Q8_F16) store(static_cast<__half*>(p.y));
                else store(static_cast<float*>(p.y));
            }
        }
        if (lane == 0) bulk_wait_all();   // shared memory outlives the stores from it
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

template <int kBlock>
cudaError_t wide_clusters(int& clusters) {
    static int cached[64] = {0};
    return clusters_of_two(gemm_fp4_wide_kernel<kBlock>, WideCfg<kBlock>::kSmem, cached, clusters);
}

template <int kBlock>
cudaError_t launch_wide(const Fp4Product& g, int64_t tiles, cudaStream_t stream) {
    using C = WideCfg<kBlock>;
    int clusters = 0;
    cudaError_t e = wide_clusters<kBlock>(clusters);
    if (e != cudaSuccess) return e;
    CUtensorMap ma, mw, ms;
    if (!make_maps<kBlock>(g, C::kBox, TW, ma, mw, ms)) return cudaErrorInvalidValue;
    const int64_t units = tiles * ((g.N + TWP - 1) / TWP);
    if (units < clusters) clusters = (int)units;
    const int size = g.type == Q8_F32 ? 4 : 2;
    const bool tma_out = g.N * size % 16 == 0;
    CUtensorMap my = ma;
    if (tma_out && !make_tma_map_box(&my, g.y, size, g.rows, g.N, 32, 64 / size)) return cudaErrorInvalidValue;
    const PairArgs p{g.sfa, g.sa, g.sw, g.offsets, (int)g.rows, (int)g.E, (int)g.N, (int)g.K, (uint32_t)fp4_pitch(g.K, kBlock),
                     g.y, g.type, tma_out, (uint32_t)units};
    e = launch_dependent(gemm_fp4_wide_kernel<kBlock>, dim3((unsigned)(2 * clusters)), dim3(kPairThreads), C::kSmem, 0, stream, ma,
                         mw, ms, my, p);
    note_launch();
    return e;
}

template <int kBlock>
cudaError_t launch(const Fp4Product& p, cudaStream_t stream) {
    const int64_t per = (p.rows + p.E - 1) / p.E;   // rows of a group, on average
    const int64_t NT = (p.N + TW - 1) / TW, KB = (p.K + kFp4Span - 1) / kFp4Span;
    auto tiles = [&](int tn) { return p.offsets ? p.rows / tn + (p.E < p.rows ? p.E : p.rows) : (p.rows + tn - 1) / tn; };
    // The kernels count tiles in 32 bits, whatever the offsets are (each group at most all rows).
    if (tiles(16) * NT >= (1LL << 31) - 1024 || (p.rows / 16 + 1) * p.E >= (1LL << 31)) return cudaErrorNotSupported;
    // Groups of unequal size: a tile four times the average leaves few of them more than one. The host does not see the offsets, so
    // a group far above the average reads its weights again from L2 for each of its tiles. Measured, us, for tiles of 16 and 32
    // tokens and the pairs' 128: 512 rows of 128 experts, 4096x4096, evenly 179 / 180 / 181; the largest with 94 rows 176 / 173 / 173,
    // with 300 191 / 183 / 181, with all 35 / 23 / 12; 2048x2048, evenly 50.9 / 51.3 / 53.4, 300 rows 54.0 / 52.4 / 52.7.
    const int64_t most = p.offsets ? 4 * per : per;
    if (most <= 16) return launch_swap<8, kBlock>(p, tiles(16), stream);
    if (most <= 32) return launch_swap<16, kBlock>(p, tiles(32), stream);
    // What a round of tiles takes, in us, as measured (a stage, and a fixed part): 0.27 and 0.3 for 128 weight rows x 32
    // tokens over 152 CTAs, 0.24 (0.20 for up to 64 tokens) and 1.0 for 256 x 128 over 76 pairs, 0.31 and 1.6 for 256 x
    // 256; and once for each kernel 4.2, 5 and 6. A group's last tile is half full on average. Weights that are not in L2
    // take their time to be read whatever the tile, and the pairs with the smaller one wait less for them. Measured, us,
    // in the same order, in a graph with two sets of operands in turn, which L2 holds: 128x2048x2048 6.7 / 8.4 / 9.1;
    // 64x8192x8192 11.4 / 11.0 / 14.1; 128x8192x8192 19.1 / 12.8 / 14.8; 256x8192x8192 39 / 14.0 / 16.6;
    // 512x8192x8192 - / 23.3 / 18.3; 2050 rows of 32 experts, 4096x2048, 55 / 34.6 / 35.7; 8192 rows of 8, 4096x4096, - /
    // 74 / 53.
    int narrow = 0, wide = 0;
    cudaError_t e = wide_clusters<kBlock>(narrow);
    if (e == cudaSuccess) e = pair_clusters<kBlock>(wide);
    if (e != cudaSuccess) return e;
    auto rounds = [&](int tn, int weights, int places) {
        const int64_t t = p.offsets ? p.rows / tn + (p.E < p.rows ? p.E : p.rows) / 2 + 1 : (p.rows + tn - 1) / tn;
        return (double)((t * ((p.N + weights - 1) / weights) + places - 1) / places);
    };
    const double memory = (double)(p.E < p.rows ? p.E : p.rows) * (double)p.N * (double)p.K * (0.5 + 1.0 / kBlock) / 6.5e6;
    auto least = [&](double us) { return us > memory ? us : memory; };
    const double slim = least(rounds(32, TW, 2 * narrow) * (0.27 * (double)KB + 0.3) + 4.2);
    const double small = least(rounds(TNP, TWP, narrow) * ((per > 64 ? 0.24 : 0.20) * (double)KB + 1.0) + 5.0);
    const double large = least(rounds(PT, PN, wide) * (0.31 * (double)KB + 1.6) + 6.0);
    if (slim < small && slim < large) return launch_swap<16, kBlock>(p, tiles(32), stream);
    if (small <= large) return launch_wide<kBlock>(p, tiles(TNP), stream);
    return launch_pair<kBlock>(p, tiles(PT), stream);
}

}  // namespace

cudaError_t launch_gemm_fp4(const Fp4Product& p, int block, cudaStream_t stream) {
    return block == 16 ? launch<16>(p, stream) : launch<32>(p, stream);
}

cudaError_t read_and_clear_gemm_fp4_error(uint32_t* code) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp4_error, sizeof(v));
    if (e != cudaSuccess) return e;
    *code = v;
    if (v) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_fp4_error, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace q8
