// Routing to experts: choice of the experts and their weights, the rows of each expert, and the
// weighted sum of the experts' answers.
#include <cooperative_groups.h>

#include "q8_fp8.h"
#include "q8_internal.h"

namespace cg = cooperative_groups;

namespace q8 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kFloatMax = 3.402823466e38f;

// ------------------------------------------------------------------------------------- route
// One warp for a token. With n_group groups of `per` experts, lpg = 32 / n_group lanes hold a group's
// experts, lane r of them the VPL experts from r * VPL on: a lane never mixes groups, and lower
// lanes hold lower experts, so that "the lowest lane that has the maximum" is the lowest index.
//
// A lane sorts its keys, as order-preserving integers whose lowest bits are replaced by their place in the
// lane; the best of the warp is then one reduction a choice, and the lane that had it moves its list up.
// Without a bias the order is that of the logits (both scores grow with the logit); with one it is that of
// score + bias in 64 bits. Where two of the chosen (or the first not chosen) are nearer than the
// fp32 keys' error bound and the replaced bits (about one token in a thousand on Gaussian logits with
// a bias), the warp decides again in fp64: among the few experts about the border where only their
// order is in doubt, over all of them where the choice of the groups is. The scores of the weights are fp32.
// Bound by issue slots (about 1000 instructions a token at 256 experts): 8192 tokens take 9 to 11 us without a bias, 12 to
// 21 us (sigmoid) or up to 28 (softmax, whose bound is wider) with one and groups, of which the last few tokens' fp64
// (64 clocks an instruction) are 7 and more; one token 3.9 us, mostly launch.
struct Place {      // where a lane's experts are
    int base, have; // first expert, how many (<= VPL, may be 0)
    int group, first, lpg;
};

struct Doubt {
    bool group = false, order = false;   // closer than the error bound: two groups, two of the best experts
    bool kept = true;                    // this lane's group can be chosen from
    float last = -INFINITY;              // the first key that was not chosen
};

// Ascending order of the floats as unsigned values; 0 is free for "masked".
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(kFull, ordered(v))); }

// The same for doubles: fp64 comparisons run at a small fraction of the integer rate.
__device__ __forceinline__ uint64_t ordered(double f) {
    const uint64_t b = (uint64_t)__double_as_longlong(f);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered(uint64_t u) {
    return __longlong_as_double((int64_t)(u ^ ((u >> 63) ? 0x8000000000000000ull : ~0ull)));
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(v >> 32));
    return (uint64_t)hi << 32 | __reduce_max_sync(kFull, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}

// A group's score: its best key, or (sum2) the sum of its two best. Keys are floats (-inf: masked) or ordered
// doubles (0: masked). Returns whether this lane's group is among the topk_group best, its score and its two best keys.
template <int VPL, class K>
__device__ __forceinline__ bool keep_group(const K (&key)[VPL], const Place& pl, const RouteArgs& a, bool sum2,
                                           K& score, K& m1, K& m2) {
    const K none = sizeof(K) == 4 ? (K)-INFINITY : (K)0;
    m1 = none;
    m2 = none;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        m2 = max(m2, min(m1, key[i]));
        m1 = max(m1, key[i]);
    }
    const K l1 = m1, l2 = m2;
    const int lane = threadIdx.x & 31;
    for (int d = 1; d < pl.lpg; ++d) {
        int src = lane + d;
        src = src >= pl.first + pl.lpg ? src - pl.lpg : src;
        const K o1 = __shfl_sync(kFull, l1, src & 31), o2 = __shfl_sync(kFull, l2, src & 31);
        m2 = max(min(m1, o1), max(m2, o2));
        m1 = max(m1, o1);
    }
    score = m1;
    if (sum2 && m2 > none) {
        if constexpr (sizeof(K) == 4) score = m1 + m2;
        else score = ordered(unordered(m1) + unordered(m2));
    }
    int rank = 0;
    for (int g = 0; g < a.n_group; ++g) {
        const K o = __shfl_sync(kFull, score, g * pl.lpg);
        rank += (o > score || (o == score && g < pl.group)) ? 1 : 0;
    }
    return rank < a.topk_group;
}

// The chosen expert of lane j in `mine` (-1: none) for j < k, from a lane's keys (-inf: masked). check: report
// decisions closer than eps + rel |key|, the error of two keys. A group's score is off by that of its own two, which goes
// with their sizes and not with the size of their sum: the groups are in doubt where the lowest that the score of one
// that is kept can be is not above the highest that another's can be.
template <int VPL>
__device__ __forceinline__ Doubt choose_fast(float (&key)[VPL], const Place& pl, const RouteArgs& a, bool check,
                                             float eps, float rel, int lane, int& mine) {
    Doubt doubt;
    if (a.topk_group < a.n_group) {   // else every group is kept, and there is nothing to decide or to doubt
        float score, m1, m2;
        doubt.kept = keep_group<VPL, float>(key, pl, a, a.bias != nullptr, score, m1, m2);
        if (a.bias) {   // else the scores are logits, and exact
            const float size = fabsf(m1) + (m2 > -INFINITY ? fabsf(m2) : 0.0f);
            const float err = eps + rel * fminf(size, kFloatMax);
            // a sum past the largest fp32 value can be anything from there on: kept finite, it is in doubt against its like
            const float mid = fminf(fmaxf(score, -kFloatMax), kFloatMax);
            const bool counts = pl.group < a.n_group, live = m1 > -INFINITY;   // a group without an expert: as low as can be
            const float lo = !counts || !doubt.kept ? INFINITY : live ? mid - err : -INFINITY;
            const float hi = !counts || doubt.kept || !live ? -INFINITY : mid + err;
            const float most = warp_max(hi);
            doubt.group = most > -INFINITY && -warp_max(-lo) <= most;
        }
    }
    uint32_t o[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        o[i] = doubt.kept && key[i] > -INFINITY ? (ordered(key[i]) & ~(uint32_t)(VPL - 1)) | (VPL - 1 - i) : 0;
    // Batcher's odd-even merge sort, falling
#pragma unroll
    for (int p = 1; p < VPL; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < VPL; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if ((i + j) / (2 * p) == (i + j + k) / (2 * p) && i + j + k < VPL) {
                        const uint32_t hi = max(o[i + j], o[i + j + k]), lo = min(o[i + j], o[i + j + k]);
                        o[i + j] = hi;
                        o[i + j + k] = lo;
                    }
    mine = -1;
    float last = INFINITY;
    for (int j = 0; j <= a.k; ++j) {
        // equal keys: the lowest lane, and in it the lowest place
        const uint32_t head = o[0] & ~(uint32_t)(VPL - 1), m = __reduce_max_sync(kFull, head);
        if (m == 0) break;
        const float top = unordered(m);
        doubt.order |= last - top <= eps + rel * fabsf(top);
        last = top;
        if (j == a.k) {
            doubt.last = top;
            break;
        }
        const int who = __ffs(__ballot_sync(kFull, head == m)) - 1;
        const int e = __shfl_sync(kFull, pl.base + (VPL - 1) - (int)(o[0] & (VPL - 1)), who);
        if (lane == j) mine = e;
        if (lane == who) {
#pragma unroll
            for (int i = 0; i + 1 < VPL; ++i) o[i] = o[i + 1];
            o[VPL - 1] = 0;
        }
    }
    doubt.order = doubt.order && check;
    doubt.group = doubt.group && check;
    return doubt;
}

template <class T>
__device__ __forceinline__ float load_logit(const T* p) {
    const float l = to_float(*p);
    return l != l ? -INFINITY : fminf(l, kFloatMax) + 0.0f;   // + 0: -0 and 0 are one value
}

// A lane's logits (-inf: masked).
template <int VPL, class T>
__device__ __forceinline__ void load_logits(const T* row, const Place& pl, float (&l)[VPL]) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] = i < pl.have ? load_logit(row + pl.base + i) : -INFINITY;
}

__device__ __forceinline__ float fast_exp(float x) {   // 2^(x log2 e)
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(__fmul_rn(x, 1.4426950408889634f)));
    return e;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

// The fp32 keys of a router with a bias, in place of the logits. A bias of -inf or NaN masks.
template <int VPL>
__device__ __forceinline__ void fast_keys(float (&key)[VPL], const Place& pl, const RouteArgs& a, float m, float inv_z) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const float p = a.softmax ? fast_exp(key[i] - m) * inv_z : fast_rcp(1.0f + fast_exp(-key[i]));
        const float b = i < pl.have ? __ldg(a.bias + pl.base + i) : 0.0f;
        const float k = p + b + 0.0f;
        key[i] = key[i] > -INFINITY && k > -INFINITY ? k : -INFINITY;   // a NaN is no key: it would count as its neighbour
    }
}

// The choice again, in fp64. Only the order is in doubt: the experts with an fp32 key of at least `from` in the
// groups that were kept, one a lane, ranked against one another. Otherwise, or with more of them
// than lanes: all experts.
template <int VPL, class T>
__device__ __noinline__ int route_exact(const T* row, const Place pl, const RouteArgs a, int lane, float m, float inv_z,
                                        const Doubt doubt, float from, int16_t* list) {
    double z = 1.0;
    if (a.bias && a.softmax) {
        z = 0.0;
        for (int i = 0; i < pl.have; ++i) {
            const float l = load_logit(row + pl.base + i);
            if (l > -INFINITY) z += exp((double)l - (double)m);
        }
        for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(kFull, z, d);
    }
    auto exact_key = [&](int e) {
        const double l = load_logit(row + e);   // not masked
        if (!a.bias) return ordered(l);
        const double k = (a.softmax ? exp(l - (double)m) / z : 1.0 / (1.0 + exp(-l))) + (double)__ldg(a.bias + e);
        return k > -(double)INFINITY ? ordered(k) : (uint64_t)0;   // a bias of -inf or NaN masks as well
    };
    int count = 0;
    if (!__any_sync(kFull, doubt.group)) {
        float key[VPL];
        load_logits<VPL>(row, pl, key);
        if (a.bias) fast_keys<VPL>(key, pl, a, m, inv_z);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const bool in = doubt.kept && key[i] > -INFINITY && key[i] >= from;
            const unsigned vote = __ballot_sync(kFull, in);
            const int at = count + __popc(vote & ((1u << lane) - 1));
            if (in && at < 32) list[at] = (int16_t)(pl.base + i);
            count += __popc(vote);
        }
        __syncwarp();
        if (count <= 32) {
            const int e = lane < count ? list[lane] : -1;
            const uint64_t k = e >= 0 ? exact_key(e) : 0;
            int rank = 0;
            for (int t = 0; t < count; ++t) {
                const uint64_t o = __shfl_sync(kFull, k, t);
                const int oe = __shfl_sync(kFull, e, t);
                rank += o > k || (o == k && oe < e) ? 1 : 0;
            }
            __syncwarp();
            if (e >= 0) list[rank] = (int16_t)e;
            __syncwarp();
            return lane < min(count, a.k) ? list[lane] : -1;
        }
    }
    uint64_t key[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        key[i] = i < pl.have && load_logit(row + pl.base + i) > -INFINITY ? exact_key(pl.base + i) : 0;
    uint64_t score, m1, m2;
    if (a.topk_group < a.n_group && !keep_group<VPL, uint64_t>(key, pl, a, a.bias != nullptr, score, m1, m2))
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = 0;
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i] > best) { best = key[i]; at = i; }
        const uint64_t top = warp_max(best);
        if (top == 0) break;
        const int who = __ffs(__ballot_sync(kFull, best == top)) - 1;
        const int e = __shfl_sync(kFull, pl.base + at, who);
        if (lane == j) mine = e;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (lane == who && i == at) key[i] = 0;
    }
    return mine;
}

template <int VPL, class T>
__global__ void __launch_bounds__(128) moe_route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (t >= a.T) return;
    __shared__ int16_t lists[4][32];
    const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
    const int per = a.E / a.n_group;
    Place pl;
    pl.lpg = 32 / a.n_group;
    pl.group = lane / pl.lpg;
    pl.first = pl.group * pl.lpg;
    const int r = lane - pl.first;
    pl.base = pl.group * per + r * VPL;
    pl.have = pl.group < a.n_group ? max(0, min(VPL, per - r * VPL)) : 0;
    float key[VPL];
    load_logits<VPL>(row, pl, key);
    float m = -INFINITY, inv_z = 1.0f;
    if (a.softmax) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = fmaxf(m, key[i]);
        m = warp_max(m);
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) z += key[i] > -INFINITY ? expf(key[i] - m) : 0.0f;
#pragma unroll
        for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(kFull, z, d);
        inv_z = z > 0.0f ? __fdiv_rn(1.0f, z) : 0.0f;
    }
    // The fp32 keys' error. Sigmoid: the fast exponential is off by |l| 2^-24 + 2^-22 relative, which moves p by
    // p (1 - p) of that, at most 1.23 2^-24 (|l| p (1 - p) < 0.23); the sum 1 + e and the fast reciprocal
    // add 3 2^-24: under 2^-21.8, for two keys 2^-20.8. Softmax: the same exponential of a rounded l - m, and the
    // sum of up to 512 terms, under 2^-18.8 of the largest score for two. The sum with the bias: half a step
    // of |key| each. The replaced bits lower a key by less than VPL steps, so the difference of two by less than
    // that. Logits are exact, and the replaced bits of 16-bit ones are 0 anyway.
    float eps = 0.0f, rel = VPL * 0x1p-23f;
    if (a.bias) {
        fast_keys<VPL>(key, pl, a, m, inv_z);
        eps = a.softmax ? inv_z * 0x1p-18f : 0x1p-20f;
        rel += 0x1p-22f;
    }
    int mine;
    const Doubt doubt = choose_fast<VPL>(key, pl, a, a.bias || (sizeof(T) == 4 && VPL > 1), eps, rel, lane, mine);
    if (__any_sync(kFull, doubt.group || doubt.order)) {
        // whatever can be among the chosen in 64 bits: within the bound of the first not chosen
        const float from = doubt.last - 2.0f * (eps + rel * fabsf(doubt.last));
        mine = route_exact<VPL, T>(row, pl, a, lane, m, inv_z, doubt, from, lists[threadIdx.x / 32]);
    }
    float p = 0.0f;
    if (mine >= 0) {
        const float l = load_logit(row + mine);
        // sigmoid: from exp(-|l|), which is at most 1; exp(-l) is past fp32's range for l < -88.7, the score is not
        const float t = expf(a.softmax ? l - m : -fabsf(l));
        p = a.softmax ? t * inv_z : __fdiv_rn(l < 0.0f ? t : 1.0f, 1.0f + t);
    }
    if (a.renorm) {
        float sum = p;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
        p = sum > 0.0f ? __fdiv_rn(p, sum) : 0.0f;
    }
    if (lane < a.k) {
        a.idx[t * a.k + lane] = mine;
        a.w[t * a.k + lane] = p * a.scale;
    }
}

template <class T>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
    const int per = a.E / a.n_group, lpg = 32 / a.n_group, vpl = (per + lpg - 1) / lpg;
    const int64_t ctas = (a.T + 3) / 4;
    if (ctas >= (1LL << 31)) return cudaErrorNotSupported;
    const unsigned grid = (unsigned)ctas;
    if (vpl <= 1) moe_route_kernel<1, T><<<grid, 128, 0, stream>>>(a);
    else if (vpl <= 2) moe_route_kernel<2, T><<<grid, 128, 0, stream>>>(a);
    else if (vpl <= 4) moe_route_kernel<4, T><<<grid, 128, 0, stream>>>(a);
    else if (vpl <= 8) moe_route_kernel<8, T><<<grid, 128, 0, stream>>>(a);
    else if (vpl <= 16) moe_route_kernel<16, T><<<grid, 128, 0, stream>>>(a);
    else if (vpl <= 32) moe_route_kernel<32, T><<<grid, 128, 0, stream>>>(a);
    else return cudaErrorNotSupported;
    note_launch();
    return cudaGetLastError();
}

// -------------------------------------------------------------------------------------- plan
// A stable counting sort of the expert indices in one launch: a cluster of CTAs, each with a
// contiguous share of the entries, each warp with a contiguous share of its CTA's. Sweep 1 counts
// the entries of each (warp, expert); prefix sums over warps, then CTAs (distributed shared memory),
// then experts give each warp its first slot of each expert; sweep 2 hands the slots out in order.
// Bound by latencies (each lane loads eight entries at once): 65536 entries of 256 experts 9.6 us, 8 entries 3.7 us.
constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32, kPlanAhead = 8;

__global__ void __launch_bounds__(kPlanThreads)
    moe_plan_kernel(const int32_t* __restrict__ idx, int64_t n, int E, int bits, int32_t* __restrict__ offsets,
                    int32_t* __restrict__ slots) {
    extern __shared__ int32_t plan_smem[];
    int32_t* count = plan_smem;                       // [warps][E]
    int32_t* total = plan_smem + kPlanWarps * E;      // [E] of this CTA
    __shared__ int32_t scan[kPlanWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    // shares in whole warps of entries
    const int64_t share = (n + (int64_t)ctas * kPlanThreads - 1) / ((int64_t)ctas * kPlanThreads) * 32;
    const int64_t lo = min(n, ((int64_t)rank * kPlanWarps + warp) * share), hi = min(n, lo + share);
    int e[kPlanAhead];
    // eight entries of this lane from i0 on: the expert, or E for nobody's and past the end
    auto load = [&](int64_t i0) {
#pragma unroll
        for (int j = 0; j < kPlanAhead; ++j) {
            const int64_t i = i0 + 32 * j + lane;
            e[j] = i < hi ? __ldg(idx + i) : E;
        }
#pragma unroll
        for (int j = 0; j < kPlanAhead; ++j)
            if (e[j] < 0 || e[j] > E) e[j] = E;
    };
    load(lo);
    for (int i = threadIdx.x; i < kPlanWarps * E; i += kPlanThreads) count[i] = 0;
    __syncthreads();
    int32_t* mine = count + warp * E;
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kPlanAhead) {
        if (i0 != lo) load(i0);
#pragma unroll
        for (int j = 0; j < kPlanAhead; ++j)
            if (e[j] < E) atomicAdd(mine + e[j], 1);   // counts: the order does not matter
    }
    if (hi - lo > 32 * kPlanAhead) load(lo);
    __syncthreads();
    if (threadIdx.x < E) {
        int run = 0;
        for (int w0 = 0; w0 < kPlanWarps; w0 += 16) {
            int c[16];
#pragma unroll
            for (int w = 0; w < 16; ++w) c[w] = count[(w0 + w) * E + threadIdx.x];
#pragma unroll
            for (int w = 0; w < 16; ++w) {
                count[(w0 + w) * E + threadIdx.x] = run;
                run += c[w];
            }
        }
        total[threadIdx.x] = run;
    }
    if (ctas > 1) cluster.sync();
    int before = 0, all = 0;
    if (threadIdx.x < E) {
        if (ctas == 1) {
            all = total[threadIdx.x];
        } else {
            for (int c = 0; c < ctas; ++c) {
                const int v = cluster.map_shared_rank(total, c)[threadIdx.x];
                all += v;
                if (c < rank) before += v;
            }
        }
    }
    int incl = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    if (ctas > 1) cluster.sync();   // also: nobody reads this CTA's totals any more
    else __syncthreads();
    if (threadIdx.x < E) {
        int start = incl - all;
        for (int w = 0; w < warp; ++w) start += scan[w];
        total[threadIdx.x] = start + before;
        if (rank == 0) {
            if (threadIdx.x == 0) offsets[0] = 0;
            offsets[threadIdx.x + 1] = start + all;
        }
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kPlanAhead) {
        if (i0 != lo) load(i0);
#pragma unroll
        for (int j = 0; j < kPlanAhead; ++j) {
            const int64_t i = i0 + 32 * j;
            if (i >= hi) break;
            // the lanes with the same expert, from one vote on each bit of it
            unsigned same = kFull;
            for (int b = 0; b < bits; ++b) {
                const bool bit = (e[j] >> b) & 1;
                const unsigned vote = __ballot_sync(kFull, bit);
                same &= bit ? vote : ~vote;
            }
            int slot = -1;
            if (e[j] < E) slot = total[e[j]] + mine[e[j]] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (e[j] < E && lane == __ffs(same) - 1) mine[e[j]] += __popc(same);
            __syncwarp();
            if (i + lane < hi) slots[i + lane] = slot;
        }
    }
}

// ----------------------------------------------------------------------------------- combine
// 16 bytes of a token's output for each thread, its k rows' loads in flight four at a time; the sum in
// fp32 in the order of the choices. Reads k rows and writes one for each token: bound by memory, 8192 x 4096 with 8
// rows each 82 us on the device, 92 us back to back (6.6 TB/s, 0.97 of the measured copy).
// A thread has U chunks of 16 bytes, a warp 32 U neighbouring ones (of one token or of two): U = 4 for one row a token,
// 2 for two or three, 1 for more, so that at least four loads are in flight (5961 x 4560, one row a token: 22 us with
// four chunks, 32 with one; 8192 x 4096 with two rows 33 us, 0.90 of the copy).
template <class T, int U>
__global__ void __launch_bounds__(256)
    moe_combine_kernel(const T* __restrict__ h, int64_t rows, uint32_t chunks, const int32_t* __restrict__ slots,
                       const float* __restrict__ w, uint64_t total, int k, T* __restrict__ y) {
    constexpr int n = Vec16<T>::n, kAhead = 4 / U;
    const uint64_t i0 = (((uint64_t)blockIdx.x * 256 + threadIdx.x) / 32) * (32 * U) + (threadIdx.x & 31);
    float acc[U][n];
    uint64_t at[U];     // of the token's first choice
    uint32_t c[U];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint64_t i = i0 + u * 32;
        live[u] = i < total;
        const uint64_t t = !live[u] ? 0 : total >> 32 ? i / chunks : (uint32_t)i / chunks;
        c[u] = live[u] ? (uint32_t)(i - t * chunks) : 0;
        at[u] = t * k;
#pragma unroll
        for (int q = 0; q < n; ++q) acc[u][q] = 0.0f;
    }
    for (int j0 = 0; j0 < k; j0 += kAhead) {
        Vec16<T> v[U][kAhead];
        float wt[U][kAhead];
        bool in[U][kAhead];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int64_t d = live[u] && j0 + j < k ? (int64_t)__ldg(slots + at[u] + j0 + j) : -1;
                in[u][j] = d >= 0 && d < rows;
                wt[u][j] = in[u][j] ? __ldg(w + at[u] + j0 + j) : 0.0f;
                v[u][j].u = make_uint4(0, 0, 0, 0);
                if (in[u][j]) v[u][j].u = __ldcs(reinterpret_cast<const uint4*>(h) + (uint64_t)d * chunks + c[u]);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (in[u][j]) {
                    float f[n];
                    to_floats(v[u][j], f);
#pragma unroll
                    for (int q = 0; q < n; ++q) acc[u][q] = __fmaf_rn(wt[u][j], f[q], acc[u][q]);
                }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (live[u]) {
            Vec16<T> o;
#pragma unroll
            for (int q = 0; q < n; ++q) o.t[q] = from_float<T>(acc[u][q]);
            reinterpret_cast<uint4*>(y)[i0 + u * 32] = o.u;
        }
}

template <class T>
cudaError_t launch_combine(const void* h, int64_t rows, int64_t N, const int32_t* slots, const float* w, int64_t T_,
                           int k, void* y, cudaStream_t stream) {
    const uint64_t chunks = (uint64_t)N / Vec16<T>::n, total = (uint64_t)T_ * chunks;
    const int U = k == 1 ? 4 : k < 4 ? 2 : 1;
    const uint64_t ctas = (total + 256 * U - 1) / (256 * U);
    if (chunks >= (1ULL << 32) || ctas >= (1ULL << 31)) return cudaErrorNotSupported;
    auto* kernel = U == 4 ? moe_combine_kernel<T, 4> : U == 2 ? moe_combine_kernel<T, 2> : moe_combine_kernel<T, 1>;
    kernel<<<(unsigned)ctas, 256, 0, stream>>>(static_cast<const T*>(h), rows, (uint32_t)chunks, slots, w, total, k,
                                               static_cast<T*>(y));
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs& a, q8_float_type t, cudaStream_t stream) {
    switch (t) {
        case Q8_F32: return launch_route<float>(a, stream);
        case Q8_BF16: return launch_route<__nv_bfloat16>(a, stream);
        default: return launch_route<__half>(a, stream);
    }
}

cudaError_t launch_moe_plan(const int32_t* idx, int64_t n, int E, int32_t* offsets, int32_t* slots,
                            cudaStream_t stream) {
    const size_t smem = (size_t)(kPlanWarps + 1) * E * 4;
    if (smem > 48 * 1024) {   // the limit is the device's, so always the same: another thread may be about to launch
        const cudaError_t e = cudaFuncSetAttribute(moe_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (kPlanWarps + 1) * kMaxExperts * 4);
        if (e != cudaSuccess) return e;
    }
    // A CTA for each 2048 entries, up to the portable cluster of 8.
    int ctas = 1, bits = 1;
    while (ctas < 8 && (int64_t)ctas * 2048 < n) ctas *= 2;
    while ((1 << bits) <= E) ++bits;   // of 0 .. E
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(kPlanThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, moe_plan_kernel, idx, n, E, bits, offsets, slots);
    note_launch();
    return e;
}

cudaError_t launch_moe_combine(const void* h, q8_float_type t, int64_t rows, int64_t N, const int32_t* slots,
                               const float* w, int64_t T, int k, void* y, cudaStream_t stream) {
    switch (t) {
        case Q8_F32: return launch_combine<float>(h, rows, N, slots, w, T, k, y, stream);
        case Q8_BF16: return launch_combine<__nv_bfloat16>(h, rows, N, slots, w, T, k, y, stream);
        default: return launch_combine<__half>(h, rows, N, slots, w, T, k, y, stream);
    }
}

}  // namespace q8
