// qz_route.cu -- the router of a mixture-of-experts layer (sm_100a): scores,
// group limit, top-k choice and weights; its gradient; and the expert order
// (plan) of the choices.
//
// Router.  One warp owns one token: lane l holds the logits of experts
// l, l + 32, ... in registers, so a row is read once and every reduction is a
// warp reduction.  Keys are order-preserving integers.  The choice first bounds
// itself from below by the top_k-th largest of the lanes' own maxima (one
// redux.sync a round), which leaves little more than top_k candidates; these go
// one to a lane and rank themselves against each other, ties to the lower
// index.  16384 x 256 fp32 logits take 11 us; top_k rounds of a warp-wide argmax
// over all keys took 8 us more: what bounds the kernel is instruction issue, not
// the 17 MB it reads.
//
// Without a bias or groups the key is the fp32 logit itself.  With them two
// experts (or groups) may differ by less than an fp32 rounding of their scores:
// the choice is first made in fp32, and if any two neighbours that decide it are
// closer than the fp32 error bound, this token's is made again in binary64: of
// the candidates alone for a sigmoid, of all experts for a softmax or close groups
// (16384 tokens of 256 experts in 8 groups take 25 us so; every token again in
// binary64, 65).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <float.h>

#include <type_traits>

#include "../../include/qz.h"
#include "qz_act.cuh"
#include "qz_device.cuh"

namespace qz {

namespace cg = cooperative_groups;

constexpr int kRouteWarps = 4;  // tokens per CTA
constexpr unsigned kFull = 0xFFFFFFFFu;

struct RouteArgs {
    const void* logits;
    const float* bias;
    int64_t T, ld;
    int E, k, score, n_groups, top_groups, renorm;
    int step_groups, step_rest;  // 32 experts further: groups, and experts of a group
    float scale;
    int32_t* ids;
    float* weights;
    // filled in by each warp: its token's row of logits, and their type
    int64_t row;
    bool bf16;
};

// A logit as the router reads it: NaN masks like -inf, +inf counts as FLT_MAX.
__device__ __forceinline__ float clean_logit(float x) { return x != x ? -INFINITY : fminf(x, FLT_MAX); }

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    if (BF16) return clean_logit(__uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16));
    return clean_logit(__ldg(static_cast<const float*>(p) + i));
}

// Where the experts of a row live in the warp: lane l's value j is expert
// l + 32 j, or with DENSE (32 PER experts, rows that 16-byte loads can read)
// expert PER l + j.  Dense rows load and reach the groups, which then are whole
// lanes, in far fewer instructions: 25 us in place of 36 on 16384 tokens of 256
// experts in 8 groups (19 in place of 21.5 without the groups).
template <int PER, bool DENSE>
__device__ __forceinline__ int expert_at(int lane, int j) {
    return DENSE ? PER * lane + j : lane + 32 * j;
}

template <int PER, bool BF16, bool DENSE>
__device__ __forceinline__ void load_row(const void* p, int64_t row, int E, int lane, float (&x)[PER]) {
    if (!DENSE) {
#pragma unroll
        for (int j = 0; j < PER; ++j) x[j] = lane + 32 * j < E ? load_logit<BF16>(p, row + lane + 32 * j) : -INFINITY;
    } else if (BF16) {
        const uint16_t* const at = static_cast<const uint16_t*>(p) + row + PER * lane;
        uint32_t w[(PER + 1) / 2];
        if (PER == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
            w[0] = v.x;
            w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < PER / 8; ++i) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(at) + i);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) x[j] = clean_logit(j % 2 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]));
    } else {
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + row + PER * lane) + i);
            x[4 * i] = clean_logit(v.x);
            x[4 * i + 1] = clean_logit(v.y);
            x[4 * i + 2] = clean_logit(v.z);
            x[4 * i + 3] = clean_logit(v.w);
        }
    }
}

// Order-preserving integers: a < b exactly when key(a) < key(b); 0 is below
// the key of every number above -inf and stands for a masked expert.
__device__ __forceinline__ uint32_t key32(float v) {
    if (!(v > -INFINITY)) return 0u;
    v = v + 0.0f;  // -0 and +0 are one value
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The number of a key above 0.
__device__ __forceinline__ float unkey32(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ unsigned long long key64(double v) {
    if (!(v > -INFINITY)) return 0ull;
    v = v + 0.0;
    const unsigned long long b = (unsigned long long)__double_as_longlong(v);
    return (b & 0x8000000000000000ull) ? ~b : (b | 0x8000000000000000ull);
}

// Largest value of a warp and the lowest index that has it.
__device__ __forceinline__ uint32_t warp_best(uint32_t key, uint32_t& idx) {
    const uint32_t top = __reduce_max_sync(kFull, key);
    idx = __reduce_min_sync(kFull, key == top ? idx : 0xFFFFFFFFu);
    return top;
}

__device__ __forceinline__ unsigned long long warp_best(unsigned long long key, uint32_t& idx) {
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(key >> 32));
    const bool in = (uint32_t)(key >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(kFull, in ? (uint32_t)key : 0u);
    idx = __reduce_min_sync(kFull, in && (uint32_t)key == lo ? idx : 0xFFFFFFFFu);
    return ((unsigned long long)hi << 32) | lo;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// The logit below which a sigmoid is 0 in binary64.
constexpr float kNoScore = -745.0f;

// The warp's best key is taken out of `key` and its index returned (-1: no key
// is left).
template <int PER, bool DENSE, typename K>
__device__ __forceinline__ int take_best(K (&key)[PER], int lane) {
    K best = key[0];
    uint32_t idx = expert_at<PER, DENSE>(lane, 0);
#pragma unroll
    for (int j = 1; j < PER; ++j) {
        if (key[j] > best) {
            best = key[j];
            idx = expert_at<PER, DENSE>(lane, j);
        }
    }
    if (warp_best(best, idx) == 0) return -1;
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if ((int)idx == expert_at<PER, DENSE>(lane, j)) key[j] = 0;
    return (int)idx;
}

// A lane's share of the choice: expert `id` (-1: none) is choice `at`, if that is below top_k.
struct Pick {
    int id, at;
};

// top_k rounds of a warp-wide argmax.
template <int PER, bool DENSE, typename K>
__device__ __forceinline__ Pick pick_by_rounds(K (&key)[PER], int k, int lane) {
    Pick r = {-1, lane};
    for (int c = 0; c < k; ++c) {
        const int idx = take_best<PER, DENSE>(key, lane);
        if (idx < 0) break;  // no expert is left
        if (lane == c) r.id = idx;
    }
    return r;
}

// How far a value of magnitude |v| may be off is `unit` |v|, or that of the row's scores.
struct Error {
    float score, unit;
    __device__ __forceinline__ float of(float v) const { return fmaxf(score, unit * fabsf(v)); }
};

// The same by candidates (see the top of the file), `n` of them.  With GAPS
// every expert that the errors could lift to the bar is one too, and *close says
// that the lane's value is chosen and could be the next one's.  (A value below
// another by more than the errors of the other is so for its own too: |v| grows
// by the difference at most.)  false: more than 32 candidates, nothing is decided.
template <int PER, bool DENSE, bool GAPS>
__device__ __forceinline__ bool pick_by_rank(const uint32_t (&key)[PER], int k, int lane, uint2* cand, Pick& r, int& n,
                                             Error error, bool* close) {
    uint32_t left = key[0], bar = 1;
#pragma unroll
    for (int j = 1; j < PER; ++j) left = max(left, key[j]);
    const int rounds = GAPS ? k + 1 : k;  // the gaps need the value behind the last choice too
    for (int c = 0; c < rounds; ++c) {
        bar = __reduce_max_sync(kFull, left);
        if (left == bar) left = 0;
    }
    if (rounds > 32 || bar == 0) bar = 1;  // fewer lanes than choices: every key above 0
    else if (GAPS) bar = max(key32(unkey32(bar) - 2.0f * error.of(unkey32(bar))), 1u);
    n = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const bool in = key[j] >= bar;
        const unsigned mask = __ballot_sync(kFull, in);
        const int at = n + __popc(mask & ((1u << lane) - 1u));
        if (in && at < 32) cand[at] = make_uint2(key[j], (uint32_t)expert_at<PER, DENSE>(lane, j));
        n += __popc(mask);
    }
    if (n > 32) return false;
    __syncwarp();
    const uint2 mine = lane < n ? cand[lane] : make_uint2(0u, 0u);
    int before = 0;
    uint32_t behind = 0;
    for (int i = 0; i < n; ++i) {
        const uint2 other = cand[i];
        const bool ahead = other.x > mine.x || (other.x == mine.x && other.y < mine.y);
        if (ahead) ++before;
        else if (GAPS && i != lane) behind = max(behind, other.x);
    }
    r.id = lane < n ? (int)mine.y : -1;
    r.at = lane < n ? before : lane;
    if (GAPS) {
        const float value = unkey32(mine.x);
        *close = lane < n && before < k && behind != 0 && !(value - unkey32(behind) > 2.0f * error.of(value));
    }
    return true;
}

// The two largest of two pairs (a1 >= a2, b1 >= b2) into the first.
template <typename F>
__device__ __forceinline__ void merge_two(F& a1, F& a2, F b1, F b2) {
    a2 = a1 >= b1 ? (a2 > b1 ? a2 : b1) : (a1 > b2 ? a1 : b2);
    a1 = a1 > b1 ? a1 : b1;
}

__device__ __forceinline__ uint32_t key_of(float v) { return key32(v); }
__device__ __forceinline__ unsigned long long key_of(double v) { return key64(v); }
__device__ __forceinline__ float score_exp(float v) { return fast_exp(v); }
__device__ __forceinline__ double score_exp(double v) { return exp(v); }
__device__ __forceinline__ float score_rcp(float v) { return fast_rcp(v); }
__device__ __forceinline__ double score_rcp(double v) { return 1.0 / v; }

struct Choice {
    Pick pick;
    bool certain;  // the fp32 choice cannot differ from the binary64 one
};

// The picks, and for fp32 values whether the differences allow them.
template <int PER, bool DENSE>
__device__ __forceinline__ void decide(const RouteArgs& a, unsigned long long (&key)[PER], int lane, uint2*, Error, bool, Choice& r) {
    r.pick = pick_by_rounds<PER, DENSE>(key, a.k, lane);
}

template <int PER, bool DENSE>
__device__ __forceinline__ void decide(const RouteArgs& a, uint32_t (&key)[PER], int lane, uint2* cand, Error error, bool by_logit,
                                       Choice& r) {
    bool close = false;
    int n;
    if (by_logit) error = {0.0f, 0.0f};
    if (!pick_by_rank<PER, DENSE, true>(key, a.k, lane, cand, r.pick, n, error, &close)) {
        r.certain = r.certain && by_logit;
        if (r.certain) r.pick = pick_by_rounds<PER, DENSE>(key, a.k, lane);
        return;
    }
    if (by_logit || !__any_sync(kFull, close)) return;
    if (a.score != QZ_SCORE_SIGMOID) {
        r.certain = false;
        return;
    }
    // a sigmoid needs no sum over the experts: the candidates' binary64 values, one per lane
    unsigned long long* const value = reinterpret_cast<unsigned long long*>(cand + 32);
    int id = -1;
    unsigned long long mine = 0;
    if (lane < n) {
        id = (int)cand[lane].y;
        const double x = (double)(a.bf16 ? load_logit<true>(a.logits, a.row + id) : load_logit<false>(a.logits, a.row + id));
        const double e = exp(-fabs(x));
        mine = key64((x >= 0 ? 1.0 : e) / (1.0 + e) + (double)__ldg(a.bias + id));
        value[lane] = mine;
    }
    __syncwarp();
    int before = 0;
    for (int i = 0; i < n; ++i) {
        const unsigned long long other = value[i];
        if (other > mine || (other == mine && (int)cand[i].y < id)) ++before;
    }
    if (lane < n) r.pick = {id, before};
}

// The choice by values of type F (float: and whether it is certain).
// `by_logit`: the logits order the experts themselves (no bias); the values
// then only rank the groups.  `scratch` holds E + E / 32 + 1 values of F (not DENSE).
template <int PER, typename F, bool GROUPS, bool DENSE>
__device__ __forceinline__ Choice choose(const RouteArgs& a, const float (&x)[PER], float m, F* scratch, uint2* cand, int lane) {
    const bool sigmoid = a.score == QZ_SCORE_SIGMOID, by_logit = a.bias == nullptr;
    F v[PER];
    F part = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const F e = x[j] > -INFINITY ? score_exp(sigmoid ? -fabs((F)x[j]) : (F)x[j] - (F)m) : (F)0;
        v[j] = !sigmoid ? e : !(x[j] > -INFINITY) ? (F)0 : (x[j] >= 0 ? (F)1 : e) * score_rcp((F)1 + e);
        part += v[j];
    }
    F largest = 0;  // score or v, for the error bound: how far below 0 an expert is biased (masked, even) is no matter
    if (!sigmoid) {
        const F scale = score_rcp(warp_sum(part));
#pragma unroll
        for (int j = 0; j < PER; ++j) v[j] = v[j] * scale;
    }
    float bias[PER];
    if (DENSE && !by_logit) {
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
            const float4 b = __ldg(reinterpret_cast<const float4*>(a.bias + PER * lane) + i);
            bias[4 * i] = b.x;
            bias[4 * i + 1] = b.y;
            bias[4 * i + 2] = b.z;
            bias[4 * i + 3] = b.w;
        }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = lane + 32 * j;
        if (sizeof(F) == 4) largest = fmax(largest, v[j]);
        if (!by_logit && DENSE) v[j] += (F)bias[j];
        else if (!by_logit && i < a.E) v[j] += (F)__ldg(a.bias + i);
        if (!(x[j] > -INFINITY) || v[j] != v[j]) v[j] = -INFINITY;
        else if (sizeof(F) == 4 && v[j] < INFINITY) largest = fmax(largest, v[j]);
    }
    // The fp32 error of a value, in half ulps (2^-24) of the largest magnitude (`largest` is not negative: its
    // bits are ordered like it).  A softmax's exponential at d below the maximum is off by e^-d (4 + 2.22 d)
    // (2^x within 2 ulp; the difference, the product and the constant are rounded), 4 at most.  Its sum is off
    // by the terms' mean of 4 + 2.22 d, below 15 for 1024 terms, and by PER + 5 additions (a lane's in a row,
    // then a tree); reciprocal, product and the bias's addition add 4.  24 + PER covers it, as differences are
    // held against two and of groups against four of them, and two values share the sum's error.  A sigmoid has
    // no sum, but its argument is not below a maximum's: it is off by s (9 + 1.22 |x|), which is largest for the
    // largest s, and there |x| is -ln s at most.
    Error error = {0.0f, 0.0f};
    bool certain = true;
    if (sizeof(F) == 4) {
        const float top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint((float)largest)));
        const float steps = sigmoid ? 24.0f + fmaxf(-1.25f * __logf(top), 0.0f) : 24.0f + (float)PER;
        error.unit = steps / 16777216.0f;
        error.score = top * error.unit;
        // scores that are flushed to 0 (below 2^-126) are off by more than that only beside ones as small
        if (sigmoid && top < 1e-26f) {
            error = {0.0f, 0.0f};
            certain = false;
        }
    }

    decltype(key_of(F())) key[PER];
    unsigned kept = 0xFFFFFFFFu;
    const int size = a.E / a.n_groups;
    int share = 1;  // lanes that share a group, a power of two
    if (GROUPS) {
        while (2 * share * a.n_groups <= 32) share *= 2;
        F b1 = -INFINITY, b2 = -INFINITY;  // the group's two largest values
        if (DENSE) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                b2 = fmax(b2, fmin(b1, v[j]));
                b1 = fmax(b1, v[j]);
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (lane + 32 * j < a.E) scratch[lane + 33 * j] = v[j];  // a column of padding per 32: no bank conflicts
            __syncwarp();
            const int g = lane / share;
            if (g < a.n_groups) {
                for (int i = lane % share; i < size; i += share) {
                    const int e = g * size + i;
                    merge_two(b1, b2, scratch[e + e / 32], (F)-INFINITY);
                }
            }
        }
        for (int o = 1; o < share; o <<= 1) {
            const F c1 = __shfl_xor_sync(kFull, b1, o), c2 = __shfl_xor_sync(kFull, b2, o);
            merge_two(b1, b2, c1, c2);
        }
        const F mine = b2 > -INFINITY ? b1 + b2 : b1;
        const F value = __shfl_sync(kFull, mine, lane < a.n_groups ? lane * share : 0);  // lane g: group g's
        int before = 0;
        for (int h = 0; h < a.n_groups; ++h) {
            const F other = __shfl_sync(kFull, value, h);
            if (other > value || (other == value && h < lane)) ++before;
        }
        const bool mine_kept = lane < a.n_groups && before < a.top_groups;
        kept = __ballot_sync(kFull, mine_kept);
        if (sizeof(F) == 4) {
            // the least value kept against the largest that is not (0: every group with an expert is kept)
            const uint32_t low = __reduce_min_sync(kFull, mine_kept ? key32((float)value) : 0xFFFFFFFFu);
            const uint32_t high = __reduce_max_sync(kFull, lane < a.n_groups && !mine_kept ? key32((float)value) : 0u);
            certain = certain && (high == 0 || unkey32(low) - unkey32(high) > 4.0f * error.of(unkey32(low)));
        }
    }
    int group = 0, in_group = 0;  // of expert lane + 32 j, kept up without divisions
    if (GROUPS && !DENSE) {
        group = lane / size;
        in_group = lane - group * size;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        key[j] = by_logit ? (v[j] > -INFINITY ? key_of((F)x[j]) : 0) : key_of(v[j]);
        if (GROUPS && DENSE) {
            if (!((kept >> (lane / share)) & 1u)) key[j] = 0;
        } else if (GROUPS) {
            if (lane + 32 * j < a.E && !((kept >> group) & 1u)) key[j] = 0;
            group += a.step_groups;
            in_group += a.step_rest;
            if (in_group >= size) {
                in_group -= size;
                ++group;
            }
        }
    }

    Choice r = {{-1, lane}, certain};
    decide<PER, DENSE>(a, key, lane, cand, error, by_logit, r);
    return r;
}

// SIMPLE: neither a bias nor a group limit, the logits are the keys.  Ten CTAs
// per SM (48 registers; the rare binary64 path spills some) take 25.0 us, eight 25.4 and
// twelve 27.2 on 16384 tokens of 256 experts in 8 groups (rows without 16-byte loads
// 35.8, 37.8 and 35.4).
template <int PER, bool BF16, bool SIMPLE, bool GROUPS, bool DENSE>
__global__ void __launch_bounds__(kRouteWarps * 32, PER <= 8 ? 10 : 1) route_kernel(RouteArgs args) {
    extern __shared__ double s_values[];  // GROUPS, not DENSE: [warps][E + E / 32 + 1]
    __shared__ uint2 s_cand[kRouteWarps][64];  // 32 candidates, then their binary64 values
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= args.T) return;
    RouteArgs a = args;
    a.row = t * a.ld;
    a.bf16 = BF16;
    float x[PER];
    load_row<PER, BF16, DENSE>(a.logits, a.row, a.E, lane, x);
    const bool sigmoid = a.score == QZ_SCORE_SIGMOID;
    float m = 0.0f;
    if (!sigmoid && !(SIMPLE && a.renorm)) {  // what subtracts the row's maximum
        m = x[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) m = fmaxf(m, x[j]);
        m = warp_max(m);
    }

    uint2* const cand = s_cand[warp];
    Pick pick = {-1, lane};
    if (SIMPLE) {
        uint32_t key[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) key[j] = key32(x[j]);
        int n;
        if (!pick_by_rank<PER, DENSE, false>(key, a.k, lane, cand, pick, n, Error{0.0f, 0.0f}, nullptr)) pick = pick_by_rounds<PER, DENSE>(key, a.k, lane);
    } else {
        double* scratch = s_values + warp * (a.E + a.E / 32 + 1);
        Choice r = choose<PER, float, GROUPS, DENSE>(a, x, m, reinterpret_cast<float*>(scratch), cand, lane);
        if (!r.certain) r = choose<PER, double, GROUPS, DENSE>(a, x, m, scratch, cand, lane);
        pick = r.pick;
    }

    // weights: the lane's choice again from memory (the row is in L1), with the accurate exponential
    const bool live = pick.id >= 0 && pick.at < a.k;
    const float chosen = live ? load_logit<BF16>(a.logits, t * a.ld + pick.id) : -INFINITY;
    const uint32_t best = __reduce_max_sync(kFull, key32(chosen));
    const float top = best ? unkey32(best) : -INFINITY;
    float w = 0.0f;
    if (sigmoid && !(a.renorm && top < -20.0f)) {
        const float e = expf(-fabsf(chosen));
        const float s = live ? (chosen >= 0.0f ? 1.0f : e) / (1.0f + e) : 0.0f;
        w = a.renorm ? s / warp_sum(s) : s;  // the sum is at least sigmoid(-20)
    } else if (a.renorm) {
        // relative to the largest chosen logit; below -20 a sigmoid is its exponential to fp32, so that
        // a row of tiny scores keeps its ratios (below kNoScore they are 0 in binary64 too)
        const float s = live ? expf(chosen - top) : 0.0f;
        const float total = warp_sum(s);
        w = live && !(sigmoid && top < kNoScore) ? s / total : 0.0f;
    } else {
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) part += x[j] > -INFINITY ? expf(x[j] - m) : 0.0f;
        const float total = warp_sum(part);
        w = live ? expf(chosen - m) / total : 0.0f;
    }
    if (pick.at < a.k) {
        a.ids[t * a.k + pick.at] = pick.id;
        a.weights[t * a.k + pick.at] = w * a.scale;
    }
}

struct RouteGradArgs {
    const void* logits;
    const int32_t* ids;
    const float* dweights;
    void* dlogits;
    int64_t T, ld, ldd;
    int E, k, score, renorm;
    float scale;
};

// One warp per token again: lane j holds choice j and its incoming gradient,
// the dense row of gradients is accumulated in the lanes' registers in choice
// order (so a repeated id adds in a fixed order) and written once.
template <int PER, bool BF16>
__global__ void __launch_bounds__(kRouteWarps * 32) route_grad_kernel(RouteGradArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    const bool sigmoid = a.score == QZ_SCORE_SIGMOID;
    int id = -1;
    float g = 0.0f;
    if (lane < a.k) {
        id = __ldg(a.ids + t * a.k + lane);
        g = __ldg(a.dweights + t * a.k + lane) * a.scale;
        if (id < 0 || id >= a.E) id = -1;
    }
    float chosen = id >= 0 ? load_logit<BF16>(a.logits, t * a.ld + id) : -INFINITY;
    const bool live = id >= 0 && chosen > -INFINITY;
    if (!live) g = 0.0f;

    float x[PER];
    float d[PER];
    float dot = 0.0f, m = 0.0f, total = 1.0f;
    const bool dense = !sigmoid && !a.renorm;
#pragma unroll
    for (int j = 0; j < PER; ++j) d[j] = 0.0f;
    float v = 0.0f;  // what choice j adds to its expert's gradient
    if (sigmoid) {
        const float e = expf(-fabsf(chosen));
        const float s = live ? (chosen >= 0 ? 1.0f : e) / (1.0f + e) : 0.0f;
        const float rest = (chosen >= 0 ? e : 1.0f) / (1.0f + e);  // 1 - s without cancellation
        if (a.renorm) {
            // tiny scores as in the forward
            const float top = warp_max(chosen);
            const float r = top < -20.0f ? (live && top >= kNoScore ? expf(chosen - top) : 0.0f) : s;
            const float S = warp_sum(r);
            const float w = S > 0.0f ? r / S : 0.0f;
            dot = warp_sum(g * w);
            v = live ? w * (g - dot) * rest : 0.0f;
        } else {
            v = live ? g * s * rest : 0.0f;
        }
    } else if (a.renorm) {
        const float top = warp_max(chosen);
        const float s = live ? expf(chosen - top) : 0.0f;
        const float S = warp_sum(s);
        const float w = live ? s / S : 0.0f;
        dot = warp_sum(g * w);
        v = live ? w * (g - dot) : 0.0f;
    } else {
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int i = lane + 32 * j;
            x[j] = i < a.E ? load_logit<BF16>(a.logits, t * a.ld + i) : -INFINITY;
        }
        m = x[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) m = fmaxf(m, x[j]);
        m = warp_max(m);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            x[j] = x[j] > -INFINITY ? expf(x[j] - m) : 0.0f;
            part += x[j];
        }
        total = warp_sum(part);
        const float p = live ? expf(chosen - m) / total : 0.0f;
        dot = warp_sum(g * p);
        v = g * p;
    }
    for (int c = 0; c < a.k; ++c) {
        const int i = __shfl_sync(kFull, id, c);
        const float add = __shfl_sync(kFull, v, c);
        if (i < 0) continue;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (i == lane + 32 * j) d[j] += add;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = lane + 32 * j;
        if (i >= a.E) continue;
        if (dense && total > 0.0f) d[j] -= x[j] / total * dot;
        if (BF16) {
            uint16_t r;
            asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(d[j]));
            static_cast<uint16_t*>(a.dlogits)[t * a.ldd + i] = r;
        } else {
            static_cast<float*>(a.dlogits)[t * a.ldd + i] = d[j];
        }
    }
}

// ---------------------------------------------------------------------------
// the expert order
// ---------------------------------------------------------------------------
//
// A stable counting sort.  The pairs are cut into one chunk per CTA, a chunk
// into one contiguous piece per warp; a warp ranks its pairs 32 at a time with
// match_any, on top of the counts of everything before it (other chunks, then
// the warps before it in the chunk).  Three forms, by the number of pairs:
//   one CTA of 8 warps: no exchange (256 experts: 3.2 us for 8 pairs, against 5.3
//     for a cluster; 512 pairs take 6.9 against 6.0);
//   one cluster of 8 CTAs, which exchange their counts through distributed
//     shared memory (8192 pairs: 8.3 us against 25 for one CTA; 16384: 10.4);
//   two launches, one that counts each chunk and one that places, whose many CTAs
//     scatter faster (32768 pairs: 10.5 us, 131072: 12, against 15 and 42).

constexpr int kPlanWarps = 16;
constexpr int kPlanChunk = 2048;   // least pairs of a chunk of the two launches
constexpr int kPlanMost = 128;     // most chunks: each CTA of the second launch reads every chunk's counts
constexpr int kPlanOne = 256;      // pairs up to which one CTA sorts alone,
constexpr int kPlanOneWarps = 8;
constexpr int kPlanCluster = 16384;  // and one cluster
constexpr int kClusterCtas = 8;

struct PlanArgs {
    const int32_t* ids;
    int64_t n;  // pairs
    int64_t slots;
    int k, E, align;
    int chunks;
    int64_t chunk;  // pairs per chunk
    int32_t *offsets, *counts, *rows, *pair_slots;
    int* hist;  // [chunks][E] counts of each chunk
};

// The CTA's counts per warp and expert, s_cnt[warp][E].
__device__ __forceinline__ void plan_count(const PlanArgs& a, int64_t begin, int64_t end, int64_t piece, int* s_cnt) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < (int)(blockDim.x >> 5) * a.E; i += blockDim.x) s_cnt[i] = 0;
    __syncthreads();
    const int64_t lo = begin + warp * piece, hi = min(end, lo + piece);
    for (int64_t p = lo; p < hi; p += 32) {
        const int64_t i = p + lane;
        const int id = i < hi ? __ldg(a.ids + i) : -1;
        const int e = id >= 0 && id < a.E ? id : -1;
        const unsigned same = __match_any_sync(kFull, e);
        if (e >= 0 && lane == __ffs(same) - 1) s_cnt[warp * a.E + e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kPlanWarps * 32) plan_count_kernel(PlanArgs a) {
    extern __shared__ int s_cnt[];
    cudaTriggerProgrammaticLaunchCompletion();  // the second launch waits for this one's end where it must
    const int64_t begin = (int64_t)blockIdx.x * a.chunk, end = min(a.n, begin + a.chunk);
    plan_count(a, begin, end, (a.chunk + kPlanWarps - 1) / kPlanWarps, s_cnt);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int c = 0;
        for (int w = 0; w < kPlanWarps; ++w) c += s_cnt[w * a.E + e];
        a.hist[(int64_t)blockIdx.x * a.E + e] = c;
    }
    // unused slots read as -1; the placing launch fills in the others
    for (int64_t s = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; s < a.slots; s += (int64_t)gridDim.x * blockDim.x)
        a.rows[s] = -1;
}

enum PlanForm { kOneCta, kCluster, kSecondLaunch };

template <int WARPS, int FORM>
__global__ void __launch_bounds__(WARPS * 32) plan_place_kernel(PlanArgs a) {
    constexpr bool CLUSTER = FORM == kCluster;
    // [warps][E], [E] first slots, [warps] scan scratch, [E] pairs before, CLUSTER: [E] own counts
    extern __shared__ int s_cnt[];
    int* s_first = s_cnt + WARPS * a.E;
    int* s_scan = s_first + a.E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t begin = (int64_t)blockIdx.x * a.chunk, end = min(a.n, begin + a.chunk);
    const int64_t piece = (a.chunk + WARPS - 1) / WARPS;
    plan_count(a, begin, end, piece, s_cnt);
    if (FORM != kSecondLaunch) {
        for (int64_t s = blockIdx.x * blockDim.x + threadIdx.x; s < a.slots; s += gridDim.x * blockDim.x) a.rows[s] = -1;
    }
    // (the count of this chunk needs the choices only and runs beside the first launch's end)
    if (FORM == kSecondLaunch) cudaGridDependencySynchronize();
    // per expert: all pairs (its count) and the pairs of the chunks before this one, by `share` threads
    // each.  Sums of whole numbers: any order is the same.
    constexpr int threads = WARPS * 32, kPer = (QZ_MAX_ROUTE_EXPERTS + threads - 1) / threads;
    int* s_total = s_first;               // [E], then [E] before
    int* s_before = s_scan + WARPS;
    int* s_own = s_before + a.E;
    if (CLUSTER) {
        for (int e = threadIdx.x; e < a.E; e += threads) {
            int c = 0;
            for (int w = 0; w < WARPS; ++w) c += s_cnt[w * a.E + e];
            s_own[e] = c;
        }
        cg::this_cluster().sync();  // every CTA's counts, and the unused slots' rows
    }
    for (int e = threadIdx.x; e < a.E; e += threads) s_total[e] = s_before[e] = 0;
    __syncthreads();
    if (FORM == kOneCta) {
        for (int e = threadIdx.x; e < a.E; e += threads) {
            int c = 0;
            for (int w = 0; w < WARPS; ++w) c += s_cnt[w * a.E + e];
            s_total[e] = c;
        }
    } else {
        const int share = max(1, threads / a.E);
        for (int i = threadIdx.x; i < share * a.E; i += threads) {
            const int e = i % a.E;
            int all = 0, early = 0;
#pragma unroll 4
            for (int c = i / a.E; c < a.chunks; c += share) {
                const int v = CLUSTER ? cg::this_cluster().map_shared_rank(s_own, c)[e]
                                      : (int)ld_written(a.hist + (int64_t)c * a.E + e);
                all += v;
                early += c < (int)blockIdx.x ? v : 0;
            }
            if (share == 1) {
                s_total[e] = all;
                s_before[e] = early;
            } else {
                atomicAdd(s_total + e, all);
                atomicAdd(s_before + e, early);
            }
        }
    }
    if (CLUSTER) cg::this_cluster().sync();  // a CTA's counts stay until all have read them
    else __syncthreads();
    int total[kPer], before[kPer], padded = 0;  // of kPer experts
#pragma unroll
    for (int h = 0; h < kPer; ++h) {
        const int e = kPer * threadIdx.x + h;
        total[h] = before[h] = 0;
        if (e >= a.E) continue;
        total[h] = s_total[e];
        before[h] = s_before[e];
        padded += (total[h] + a.align - 1) & ~(a.align - 1);
    }
    __syncthreads();  // s_first takes s_total's place
    int incl = padded;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int first = incl - padded;
    for (int w = 0; w < warp; ++w) first += s_scan[w];
#pragma unroll
    for (int h = 0; h < kPer; ++h) {
        const int e = kPer * threadIdx.x + h;
        if (e >= a.E) continue;
        s_first[e] = first + before[h];
        if (blockIdx.x == 0) {
            a.offsets[e] = first;
            a.counts[e] = total[h];
        }
        first += (total[h] + a.align - 1) & ~(a.align - 1);
        if (blockIdx.x == 0 && e == a.E - 1) a.offsets[a.E] = first;
    }
    __syncthreads();
    // each warp's counter of an expert starts at the slot of its first pair there
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int at = s_first[e];
        for (int w = 0; w < WARPS; ++w) {
            const int c = s_cnt[w * a.E + e];
            s_cnt[w * a.E + e] = at;
            at += c;
        }
    }
    __syncthreads();
    const int64_t lo = begin + warp * piece, hi = min(end, lo + piece);
    for (int64_t p = lo; p < hi; p += 32) {
        const int64_t i = p + lane;
        const int id = i < hi ? __ldg(a.ids + i) : -1;
        const int e = id >= 0 && id < a.E ? id : -1;
        const unsigned same = __match_any_sync(kFull, e);
        int slot = -1;
        if (e >= 0) slot = s_cnt[warp * a.E + e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) s_cnt[warp * a.E + e] += __popc(same);
        __syncwarp();
        if (i < hi) {
            a.pair_slots[i] = slot;
            if (slot >= 0) a.rows[slot] = (int)(i / a.k);
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

template <int PER, bool BF16, bool DENSE>
static void route_kinds(const RouteArgs& a, cudaStream_t s) {
    const unsigned grid = (unsigned)((a.T + kRouteWarps - 1) / kRouteWarps);
    const int threads = kRouteWarps * 32;
    const size_t smem = DENSE ? 0 : (size_t)kRouteWarps * (a.E + a.E / 32 + 1) * sizeof(double);  // at most 33 KB
    const bool groups = a.top_groups < a.n_groups;
    if (groups) route_kernel<PER, BF16, false, true, DENSE><<<grid, threads, smem, s>>>(a);
    else if (a.bias) route_kernel<PER, BF16, false, false, DENSE><<<grid, threads, 0, s>>>(a);
    else route_kernel<PER, BF16, true, false, DENSE><<<grid, threads, 0, s>>>(a);
}

template <int PER, bool BF16>
static cudaError_t route_launch(const RouteArgs& a, cudaStream_t s) {
    const uintptr_t addresses = (uintptr_t)a.logits | (uintptr_t)a.bias;
    const bool dense = PER >= 4 && a.E == 32 * PER && addresses % 16 == 0 && a.ld % (BF16 ? 8 : 4) == 0;
    if (dense) route_kinds<PER, BF16, (PER >= 4)>(a, s);
    else route_kinds<PER, BF16, false>(a, s);
    return cudaGetLastError();
}

template <bool BF16>
static cudaError_t route_sized(const RouteArgs& a, cudaStream_t s) {
    const int per = (a.E + 31) / 32;
    if (per <= 1) return route_launch<1, BF16>(a, s);
    if (per <= 2) return route_launch<2, BF16>(a, s);
    if (per <= 4) return route_launch<4, BF16>(a, s);
    if (per <= 8) return route_launch<8, BF16>(a, s);
    if (per <= 16) return route_launch<16, BF16>(a, s);
    return route_launch<32, BF16>(a, s);
}

cudaError_t launch_route(const void* logits, int type, int64_t T, int E, int64_t ld, const float* bias,
                         const qz_router& r, int32_t* ids, float* weights, cudaStream_t s) {
    const int size = E / r.n_groups;
    const RouteArgs a = {logits,        bias,          T,         ld,        E,       r.top_k, r.score, r.n_groups,
                         r.top_groups, r.renormalize, 32 / size, 32 % size, r.scale, ids,     weights,    0,       false};
    return type == QZ_TYPE_BF16 ? route_sized<true>(a, s) : route_sized<false>(a, s);
}

template <bool BF16>
static cudaError_t route_grad_sized(const RouteGradArgs& a, cudaStream_t s) {
    const unsigned grid = (unsigned)((a.T + kRouteWarps - 1) / kRouteWarps);
    const int threads = kRouteWarps * 32, per = (a.E + 31) / 32;
    if (per <= 1) route_grad_kernel<1, BF16><<<grid, threads, 0, s>>>(a);
    else if (per <= 2) route_grad_kernel<2, BF16><<<grid, threads, 0, s>>>(a);
    else if (per <= 4) route_grad_kernel<4, BF16><<<grid, threads, 0, s>>>(a);
    else if (per <= 8) route_grad_kernel<8, BF16><<<grid, threads, 0, s>>>(a);
    else if (per <= 16) route_grad_kernel<16, BF16><<<grid, threads, 0, s>>>(a);
    else route_grad_kernel<32, BF16><<<grid, threads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_route_grad(const void* logits, int type, int64_t T, int E, int64_t ld, const qz_router& r,
                              const int32_t* ids, const float* dweights, void* dlogits, int64_t ldd, cudaStream_t s) {
    const RouteGradArgs a = {logits, ids, dweights, dlogits, T, ld, ldd, E, r.top_k, r.score, r.renormalize, r.scale};
    return type == QZ_TYPE_BF16 ? route_grad_sized<true>(a, s) : route_grad_sized<false>(a, s);
}

static int64_t plan_chunk(int64_t n) {
    if (n <= kPlanOne) return n > 0 ? n : 1;
    if (n <= kPlanCluster) return (n + kClusterCtas - 1) / kClusterCtas;
    const int64_t c = (n + kPlanMost - 1) / kPlanMost;
    return c > kPlanChunk ? c : kPlanChunk;
}

size_t plan_bytes(int64_t n, int E) {
    return n <= kPlanCluster ? 0 : (size_t)((n + plan_chunk(n) - 1) / plan_chunk(n)) * (size_t)E * sizeof(int);
}

template <int WARPS, int FORM>
static cudaError_t launch_place(const PlanArgs& a, int ctas, cudaStream_t s) {
    const auto kernel = plan_place_kernel<WARPS, FORM>;
    const auto bytes = [](int experts) { return (size_t)((WARPS + (FORM == kCluster ? 3 : 2)) * experts + WARPS) * sizeof(int); };
    if (bytes(a.E) > 48 * 1024) {
        // asked for at its largest every time: the attribute is one value per device and
        // a smaller value of another call must not take it back
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes(QZ_MAX_ROUTE_EXPERTS));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute form;
    if (FORM == kCluster) {
        form.id = cudaLaunchAttributeClusterDimension;
        form.val.clusterDim.x = kClusterCtas;
        form.val.clusterDim.y = form.val.clusterDim.z = 1;
    } else {
        form.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        form.val.programmaticStreamSerializationAllowed = 1;
    }
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(ctas);
    config.blockDim = dim3(WARPS * 32);
    config.dynamicSmemBytes = bytes(a.E);
    config.stream = s;
    config.attrs = &form;
    config.numAttrs = FORM == kOneCta ? 0 : 1;
    return cudaLaunchKernelEx(&config, kernel, a);
}

cudaError_t launch_plan(const int32_t* ids, int64_t T, int k, int E, int align, int64_t slots, int32_t* offsets,
                        int32_t* counts, int32_t* rows, int32_t* pair_slots, void* ws, cudaStream_t s) {
    PlanArgs a;
    a.ids = ids;
    a.n = T * k;
    a.slots = slots;
    a.k = k;
    a.E = E;
    a.align = align;
    a.chunk = plan_chunk(a.n);
    a.chunks = (int)(a.n <= kPlanOne ? 1 : a.n <= kPlanCluster ? kClusterCtas : (a.n + a.chunk - 1) / a.chunk);
    a.offsets = offsets;
    a.counts = counts;
    a.rows = rows;
    a.pair_slots = pair_slots;
    a.hist = static_cast<int*>(ws);
    if (a.n <= kPlanOne) return launch_place<kPlanOneWarps, kOneCta>(a, 1, s);
    if (a.n <= kPlanCluster) return launch_place<kPlanWarps, kCluster>(a, kClusterCtas, s);
    const size_t smem = (size_t)kPlanWarps * E * sizeof(int), most = (size_t)kPlanWarps * QZ_MAX_ROUTE_EXPERTS * sizeof(int);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(plan_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
    }
    plan_count_kernel<<<a.chunks, kPlanWarps * 32, smem, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_place<kPlanWarps, kSecondLaunch>(a, a.chunks, s);
}

}  // namespace qz
