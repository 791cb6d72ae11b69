// qz_product.cu -- the experts' block-scaled matrix products on the tensor
// cores (sm_100a): rows of x times every expert's weight, with the layer's
// epilogue, and the experts' weight gradients.
//
// Mathematics.  out[s, :] = epilogue(sum_k x[row(s), k] w_e[:, k]), both
// operands coded with one scale per 32 (MXFP8) or 16 (NVFP4) elements.
// tcgen05.mma with block scaling multiplies the codes and applies both scales
// inside the fp32 accumulation, so the dequantized operands never exist.
//
// Bound.  With few rows per expert the weights' bytes from HBM; with many, the
// tensor cores.  A CTA therefore computes 128 slots x 256 accumulator columns
// (gated: 128 of the gate and 128 of the up projection, so that the gate is
// applied in registers): per 128 bytes of contraction it reads 16 KB of x and
// 32 KB of weights, and four such stages (three for NVFP4, whose scales take
// more; almost the whole shared memory) keep enough bytes in flight for HBM when
// the tile has few live rows.  A stage's products take 512 clocks at the tensor
// cores' rate and 575 here (MXFP8; NVFP4 880: twelve copies of scales go with
// them); long runs are held back by the 1000 W limit (1.4 to 1.7 GHz).
//
// Roles of the 12 warps of the one CTA per SM (persistent over its tiles).
// Twelve, because that leaves a thread 168 registers: with the shared memory in
// use L1 is too small to hold spills, and an epilogue that spilled 500 bytes a
// thread took three times as long.
//   0, 1   x's scales: a lane owns two rows (linear) and writes them into the
//          512-byte tile form, from registers loaded three pieces ahead.  With a
//          row index the elected lane also gathers the rows of x, four at a time
//          (TMA).  (Gathering by 16-byte cp.async was measured: 16 KB a stage
//          took 1,600 clocks whatever the warps, three times the products.)
//   2      TMA: the weights (tiled, 128-byte swizzle), their scales (a swizzled
//          512-byte tile is exactly what tcgen05.cp wants: one bulk copy), and x
//          when it has no index
//   3      one thread copies scales to tensor memory and issues the products
//   4..11  epilogue: warp w % 4 owns the lanes (rows) 32 (w % 4) .. + 31
//
// Tensor memory (512 columns): two accumulators of 256 columns and the scales
// do not fit side by side, so the accumulators overlap, [0, 256) and
// [256 - V, 512 - V), with the scales in the last V columns.  The epilogue
// drains the shared V columns first; from then on the next tile's products run
// under the rest of the epilogue.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/qz.h"
#include "../../include/qz_quant.cuh"
#include "qz_act.cuh"
#include "qz_device.cuh"
#include "qz_tc.cuh"

namespace qz {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kTileM = 128;
constexpr int kProductThreads = 384;
constexpr int kRowWarps = 2;
constexpr int kEpilogueWarps = 8;
constexpr int kStagingBytes = 2048;               // of an epilogue warp: 64 bytes of its 32 rows
constexpr uint32_t kRowBytes = 128;               // contraction bytes of a stage
constexpr uint32_t kBytesA = kTileM * kRowBytes;  // 16 KB; each half of B the same
constexpr uint32_t kBytesData = 3 * kBytesA;

// Per format: elements of a stage, elements of one MMA, 512-byte scale tiles of
// 128 rows per stage, tensor-memory columns of a stage's scales (A, then B's
// two halves), buffers of them, and the accumulators' overlap V.
template <int FMT>
struct Shape;
template <>
struct Shape<QZ_FMT_MXFP8> {
    static constexpr int kElems = 128, kMma = 32, kBlock = 32, kScaleTiles = 1, kStages = 4;
    static constexpr int kScaleCols = 12, kScaleBufs = kStages, kShared = 64;
};
template <>
struct Shape<QZ_FMT_NVFP4> {
    static constexpr int kElems = 256, kMma = 64, kBlock = 16, kScaleTiles = 4, kStages = 3;
    static constexpr int kScaleCols = 48, kScaleBufs = 2, kShared = 96;
};

// Shared memory of the stages: all data first (each stage on a 1024-byte
// boundary, the swizzle's period), then all scales.
template <int FMT>
constexpr uint32_t kScaleStage = 3u * 512u * Shape<FMT>::kScaleTiles;
template <int FMT>
constexpr uint32_t kStagesBytes = Shape<FMT>::kStages * (kBytesData + kScaleStage<FMT>);

struct ProductArgs {
    int act, n_experts, gated, x_per_row, gather, n_blocks;
    int64_t n, k, x_rows, slots, w_sf_stride, ld_sf;
    int64_t ids;  // what an entry of rows (a slot number without rows) must be below to have a row of x
    const uint8_t *x_sf, *w_sf, *up_sf;
    const float *x_amax, *w_amax, *up_amax;
    const int32_t *rows, *offsets, *counts;
    const uint16_t *bias, *up_bias, *residual;
    uint16_t *out, *pre;
    int64_t ld_residual, ld_out, ld_pre;
    uint8_t *q, *sf;
    unsigned* d_err;
};

struct GradArgs {
    int n_experts, f32, accumulate, m_blocks, n_blocks;
    int64_t n, k, slots;
    const uint8_t *dz_sf, *x_sf;
    const float *dz_amax, *x_amax;
    const int32_t *offsets, *counts;
    void* out;
    unsigned* d_err;
};

// One tile of work.
struct Tile {
    int e, m, n;      // expert, row tile and column block within it
    int64_t first;    // product: first slot; gradient: first slot of the contraction
    int live;         // product: rows of this tile that exist
    int64_t depth;    // contraction elements
};

// The shared-memory words of the roles, in front of the stages.
struct Control {
    uint64_t full[4], empty[4];
    uint64_t acc_full[2], acc_free;
    uint32_t tmem;
    int abort;
    long long scratch[33];
    alignas(16) int index[kTileM];
};

// ---------------------------------------------------------------------------
// work list
// ---------------------------------------------------------------------------

struct Range {
    int64_t off, cnt;
    unsigned bad;
};

__device__ __forceinline__ Range expert_range(const int32_t* offsets, const int32_t* counts, int e, int64_t slots) {
    Range r;
    r.off = __ldg(offsets + e);
    r.cnt = __ldg(counts + e);
    r.bad = (r.off < 0 || r.cnt < 0 || r.off + r.cnt > slots) ? QZ_DERR_SHAPE : 0u;
    return r;
}

// The product's list of experts in shared memory: row tiles before each, its
// first slot, and the rows of its last tile less one (a tile must be found
// without a trip to global memory by every role, at every tile).
struct ExpertList {
    int* prefix;    // [n_experts + 1]
    int* first;     // [n_experts]
    uint8_t* last;  // [n_experts]
};

constexpr size_t list_bytes(int n) { return (size_t)(2 * n + 1) * sizeof(int) + (size_t)n; }

// An expert's tiles are ordered by column block, row tiles innermost, so that
// CTAs working side by side read the same weights.
__device__ __forceinline__ Tile product_tile(const ProductArgs& a, const ExpertList& list, int u) {
    Tile t;
    t.e = find_owner(list.prefix, a.n_experts, u / a.n_blocks);
    const int tiles = list.prefix[t.e + 1] - list.prefix[t.e];
    const int v = u - list.prefix[t.e] * a.n_blocks;
    t.n = v / tiles;
    t.m = v - t.n * tiles;
    t.first = (int64_t)list.first[t.e] + (int64_t)t.m * kTileM;
    t.live = t.m + 1 < tiles ? kTileM : list.last[t.e] + 1;
    t.depth = a.k;
    return t;
}

// The gradient's list: first slot, and in place of the prefix the live slots (-1: a bad expert).
__device__ __forceinline__ bool grad_tile(const GradArgs& a, const ExpertList& list, int u, Tile& t) {
    const int per = a.m_blocks * a.n_blocks;
    t.e = u / per;
    const int v = u - t.e * per;
    t.n = v / a.m_blocks;
    t.m = v - t.n * a.m_blocks;
    t.first = list.first[t.e];
    t.live = kTileM;
    t.depth = list.prefix[t.e];
    return t.depth >= 0;
}

// ---------------------------------------------------------------------------
// x's scales: linear rows to 512-byte tiles
// ---------------------------------------------------------------------------

// 16 bytes of a row's scales from byte `at` on, in loads of W bytes, without a
// wait: where the row ends sooner, loads stay inside it and what they bring is
// not used.  (Volatile, so that the compiler neither waits for a load to merge
// it with another value nor moves it to its use.)
template <int W>
__device__ __forceinline__ uint4 load_piece(const uint8_t* row, int64_t at, int64_t kv) {
    uint4 v;
    if (W == 16) {
        asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(row + at));
    } else if (W == 8) {
        asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(row + at));
        asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.z), "=r"(v.w) : "l"(row + min(at + 8, kv - 8)));
    } else if (W == 4) {
        asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v.x) : "l"(row + at));
        asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v.y) : "l"(row + min(at + 4, kv - 4)));
        asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v.z) : "l"(row + min(at + 8, kv - 4)));
        asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v.w) : "l"(row + min(at + 12, kv - 4)));
    } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (at + i < kv) w[i / 4] |= (uint32_t)__ldg(row + at + i) << (8 * (i % 4));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

// One of the two warps: rows 64 warp + lane and + 32 of every tile's scales, and
// the gather of rows 64 warp .. + 63.
template <int FMT, bool GATED, int W>
__device__ __forceinline__ void scale_warp(const ProductArgs& p, const ExpertList& list, Control* ctl, uint32_t base, int total,
                                           const CUtensorMap& map_low, int warp, int lane) {
    typedef Shape<FMT> S;
    constexpr int kStages = S::kStages;
    constexpr int kParts = FMT == QZ_FMT_MXFP8 ? 1 : 2;  // 16-byte parts of a piece
    constexpr int kPiece = kParts * 4 / S::kScaleTiles;  // stages of a piece: 4 (MXFP8), 2 (NVFP4)
    volatile int* const abort = &ctl->abort;
    const int64_t kv = p.k / S::kBlock;
    const int steps = (int)((p.k + S::kElems - 1) / S::kElems);
    int* const index = ctl->index + 64 * warp;
    // the pieces are loaded ahead of the stages, over a walk of the tiles of their own;
    // a row that does not exist reads some row that does (the epilogue writes zeros, or does not store it)
    int su = (int)blockIdx.x - (int)gridDim.x, ss = steps;
    const uint8_t* srow[2] = {p.x_rows > 0 ? p.x_sf : p.w_sf, p.x_rows > 0 ? p.x_sf : p.w_sf};
    auto rows_of = [&](int u, int (&r)[2]) {
        const Tile t = product_tile(p, list, u);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = 64 * warp + 32 * j + lane;
            int64_t i = t.first + at;
            if (p.gather && at < t.live) i = __ldg(p.rows + i);
            r[j] = i >= 0 && i < p.x_rows ? (int)i : 0;
        }
    };
    auto next_piece = [&](uint4 (&v)[2][kParts]) {
        ss += kPiece;
        if (ss >= steps) {
            ss = 0;
            su += gridDim.x;
            if (su < total) {
                int r[2];
                rows_of(su, r);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (p.x_rows > 0) srow[j] = p.x_sf + r[j] * p.ld_sf;
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                const int64_t at = (int64_t)ss * S::kScaleTiles * 4 + 16 * i;
                v[j][i] = load_piece<W>(srow[j], kParts == 1 ? at : min(at, (kv - 1) & ~(int64_t)15), kv);
            }
    };
    // the stages, a piece at a time; tile u at step s
    int u = blockIdx.x, s = 0, it = 0, quads = 0;
    auto open_tile = [&]() {
        if (u >= total || !p.gather) return;
        quads = max(0, min(16, (product_tile(p, list, u).live - 64 * warp + 3) / 4));
        int r[2];
        rows_of(u, r);
        __syncwarp();
        index[lane] = r[0];
        index[32 + lane] = r[1];
        __syncwarp();
    };
    // false: the last tile is done, or a wait ran out
    auto use_piece = [&](uint4 (&v)[2][kParts]) -> bool {
        const int n = min(kPiece, steps - s);
        for (int q = 0; q < n; ++q, ++it) {
            const int st = it % kStages;
            if (!__all_sync(kFull, mbar_wait(smem_addr(&ctl->empty[st]), ((it / kStages) & 1) ^ 1, abort))) return false;
            const uint32_t bar = smem_addr(&ctl->full[st]);
            // row r's four scales of a 512-byte tile: word r / 32 of its 16-byte line r % 32
            const uint32_t dst = base + kStages * kBytesData + st * kScaleStage<FMT> + 16 * lane + 8 * warp;
            if (FMT == QZ_FMT_NVFP4) {
                const uint4 a = q ? v[0][kParts - 1] : v[0][0], b = q ? v[1][kParts - 1] : v[1][0];
                st_shared_v2(dst, a.x, b.x);
                st_shared_v2(dst + 512, a.y, b.y);
                st_shared_v2(dst + 1024, a.z, b.z);
                st_shared_v2(dst + 1536, a.w, b.w);
            } else {
                const uint4 a = v[0][0], b = v[1][0];
                st_shared_v2(dst, (q & 2) ? ((q & 1) ? a.w : a.z) : ((q & 1) ? a.y : a.x),
                             (q & 2) ? ((q & 1) ? b.w : b.z) : ((q & 1) ? b.y : b.x));
            }
            fence_async();
            __syncwarp();
            if (elect_one()) {
                if (quads > 0) {
                    mbar_arrive_tx(bar, quads * 4 * kRowBytes);
                    const uint32_t to = base + st * kBytesData + 64 * warp * kRowBytes;
#pragma unroll 4
                    for (int i = 0; i < quads; ++i)
                        tma_gather4(to + i * 4 * kRowBytes, &map_low, bar, (s + q) * (int)kRowBytes,
                                    *reinterpret_cast<const int4*>(index + 4 * i));
                } else {
                    mbar_arrive(bar);
                }
            }
            __syncwarp();
        }
        s += n;
        if (s == steps) {
            s = 0;
            u += gridDim.x;
            if (u >= total) return false;
            open_tile();
        }
        next_piece(v);
        return true;
    };
    // Three pieces in registers, each refilled as soon as it is used: a load has two pieces' time.  (Passing
    // them on from one to the next instead waits for a load one piece after it was issued.)
    uint4 v0[2][kParts], v1[2][kParts], v2[2][kParts];
    next_piece(v0);
    next_piece(v1);
    next_piece(v2);
    if (u >= total) return;
    open_tile();
    while (use_piece(v0) && use_piece(v1) && use_piece(v2)) {
    }
}

// ---------------------------------------------------------------------------
// epilogue pieces
// ---------------------------------------------------------------------------

// A lane computes 32 columns of its row at a time (one MXFP8 block); the code
// that does so exists once in a kernel: unrolled over a tile's columns it was
// larger than the instruction caches and took twice the time.

// 32 fp32 columns as bf16 words.
__device__ __forceinline__ void to_words(const float (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = bf16x2_of(v[2 * i], v[2 * i + 1]);
}

// Each lane's 64 bytes w (of row `lane`) to 64-byte pieces of 32 rows in
// global memory, `pitch` bytes apart, by way of the warp's 2 KB of shared
// memory: a store instruction then covers 64 consecutive bytes of 8 rows in
// place of 32 bytes of 32 rows.  Only the first `rows` rows and `bytes` bytes
// are written; ADD adds fp32 values to what is there.
template <bool ADD>
__device__ __forceinline__ void store_rows(uint8_t* to, int64_t pitch, const uint32_t (&w)[16], int rows, int bytes,
                                           uint8_t* staging, int lane) {
    // 16-byte chunk c of row r lies at c ^ (r / 2 % 4): no bank conflicts either way
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(staging + 64 * lane + 16 * (c ^ ((lane >> 1) & 3))) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        uint4 v = *reinterpret_cast<const uint4*>(staging + 64 * r + 16 * (c ^ ((r >> 1) & 3)));
        if (r < rows && 16 * c < bytes) {
            uint8_t* const at = to + r * pitch + 16 * c;
            if (ADD) {
                const float4 b = *reinterpret_cast<const float4*>(at);
                v = make_uint4(__float_as_uint(__uint_as_float(v.x) + b.x), __float_as_uint(__uint_as_float(v.y) + b.y),
                               __float_as_uint(__uint_as_float(v.z) + b.z), __float_as_uint(__uint_as_float(v.w) + b.w));
            }
            st_v4(at, v);
        }
    }
}

// v[i] += column i at p, for the first `cols` (a multiple of 8) of N bf16 columns.
template <int N>
__device__ __forceinline__ void add_row(const uint16_t* p, int cols, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        if (8 * i >= cols) continue;
        const uint4 r = *reinterpret_cast<const uint4*>(p + 8 * i);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] += bf16_lo(w[j]);
            v[8 * i + 2 * j + 1] += bf16_hi(w[j]);
        }
    }
}

// SiLU and GELU are both z sigmoid(z (a + b z^2)), with (1, 0) and (2 sqrt(2/pi), 2 sqrt(2/pi) 0.044715).
template <int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
    if (act == QZ_ACT_NONE) return;
    if (act == QZ_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = relu(v[i]);
        return;
    }
    const float a = act == QZ_ACT_GELU ? kGelu2 : 1.0f, b = act == QZ_ACT_GELU ? kGelu2 * kGeluC : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float w = fminf(fabsf(v[i]), kActFlat);
        v[i] *= sigmoid32(v[i] * fmaf(b * w, w, a));
    }
}

__device__ __forceinline__ float amax_scale(const float* amax, int64_t i) {
    return amax != nullptr ? __fdiv_rn(__ldg(amax + i), 2688.0f) : 1.0f;
}

// Accumulator columns times g (NVFP4's second-level scales), zeros for a row that does not exist.
template <int FMT, int N>
__device__ __forceinline__ void scale_row(float g, bool exists, float (&v)[N]) {
    if (FMT == QZ_FMT_NVFP4) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= g;
    }
    if (!exists) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
    }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------

// The product without and with an epilogue beyond its output (bias, activation,
// residual, pre-activations), its gated form (args.p), and the weight gradient
// (args.g).  The bare form is a kernel of its own because the others' pointers
// cost it registers and their code instruction cache.
enum Kind { kBare, kPlain, kGated, kWeightGrad };

union Args {
    ProductArgs p;
    GradArgs g;
};

template <int FMT, int KIND>
__global__ void __launch_bounds__(kProductThreads, 1)
    experts_kernel(const __grid_constant__ Args args, const __grid_constant__ CUtensorMap map_a,
                   const __grid_constant__ CUtensorMap map_low, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_up) {
    typedef Shape<FMT> S;
    constexpr int kStages = S::kStages;
    constexpr bool GRAD = KIND == kWeightGrad, GATED = KIND == kGated;
    constexpr uint32_t kSfBase = kStages * kBytesData, kSfStage = kScaleStage<FMT>;
    constexpr uint32_t kScaleBytes = 512u * S::kScaleTiles;  // of 128 rows
    constexpr int kAcc1 = 256 - S::kShared;
    constexpr int kScaleCol = 512 - S::kShared;
    extern __shared__ __align__(1024) uint8_t smem[];
    // the stages start at the next 1024-byte boundary (the swizzle's period)
    const uint32_t base = (smem_addr(smem) + 1023u) & ~1023u;
    uint8_t* const stages = smem + (base - smem_addr(smem));
    uint8_t* const staging = stages + kStagesBytes<FMT>;  // of the epilogue warps
    Control* const ctl = reinterpret_cast<Control*>(staging + kEpilogueWarps * kStagingBytes);
    ExpertList list;
    list.prefix = reinterpret_cast<int*>(ctl + 1);
    const int n_experts = GRAD ? args.g.n_experts : args.p.n_experts;
    list.first = list.prefix + n_experts + 1;
    list.last = reinterpret_cast<uint8_t*>(list.first + n_experts);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const ProductArgs& p = args.p;
    const GradArgs& g = args.g;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_addr(&ctl->full[i]), GRAD ? 1 : 1 + kRowWarps);  // TMA; the warps of x's scales
            mbar_init(smem_addr(&ctl->empty[i]), 1);
        }
        mbar_init(smem_addr(&ctl->acc_full[0]), 1);
        mbar_init(smem_addr(&ctl->acc_full[1]), 1);
        mbar_init(smem_addr(&ctl->acc_free), kEpilogueWarps);
        ctl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
    }
    if (warp == 3) tmem_alloc(smem_addr(&ctl->tmem), 512);
    int total;
    if (GRAD) {
        total = g.n_experts * g.m_blocks * g.n_blocks;
        for (int e = threadIdx.x; e < n_experts; e += blockDim.x) {
            const Range r = expert_range(g.offsets, g.counts, e, g.slots);
            const unsigned bad = r.bad | ((r.off & 127) ? QZ_DERR_ALIGN : 0u);
            list.first[e] = (int)r.off;
            list.prefix[e] = bad ? -1 : (int)r.cnt;
            if (bad && blockIdx.x == 0 && g.d_err) atomicOr(g.d_err, bad);
        }
        __syncthreads();
    } else {
        unsigned bad = 0;
        const int row_tiles = block_prefix(p.n_experts, list.prefix, ctl->scratch,
                                           [&](int e) -> long long {
                                               const Range r = expert_range(p.offsets, p.counts, e, p.slots);
                                               bad |= r.bad;
                                               list.first[e] = (int)r.off;
                                               list.last[e] = (uint8_t)((r.cnt + kTileM - 1) % kTileM);
                                               return r.bad ? 0 : (r.cnt + kTileM - 1) / kTileM;
                                           },
                                           p.d_err);  // ends with a barrier
        const int64_t tiles = (int64_t)row_tiles * p.n_blocks;
        // ranges that overlap could make more tiles than an int counts (the roles step past the last)
        total = tiles <= 0x7FFF0000 ? (int)tiles : 0;
        if (tiles > 0x7FFF0000) bad |= QZ_DERR_TOO_LARGE;
        if (bad && blockIdx.x == 0 && p.d_err) atomicOr(p.d_err, bad);
    }
    tc_fence_after();
    const uint32_t tmem = *const_cast<volatile uint32_t*>(&ctl->tmem);
    volatile int* const abort = &ctl->abort;
    const int64_t kv = (GRAD ? g.slots : p.k) / S::kBlock;  // scale columns of the operands
    const int64_t scale_tiles = (kv + 3) / 4;               // 512-byte tiles of a 128-row block of scales

    // what each role needs to know of tile u; false: nothing is to be done
    auto tile_of = [&](int u, Tile& t) -> bool {
        if (GRAD) return grad_tile(g, list, u, t);
        t = product_tile(p, list, u);
        return true;
    };
    // 128-column halves of B that tile t multiplies with
    auto halves_of = [&](const Tile& t) -> int {
        if (GRAD) return (int64_t)t.n * 256 + 128 < g.k ? 2 : 1;
        return GATED || (int64_t)t.n * 256 + 128 < p.n ? 2 : 1;
    };
    auto stages_of = [&](const Tile& t) -> int { return (int)((t.depth + S::kElems - 1) / S::kElems); };

    if (warp == 2) {
        // ------------------------------------------------------------ TMA
        if (elect_one()) {
            int it = 0;
            for (int u = blockIdx.x; u < total; u += gridDim.x) {
                Tile t;
                if (!tile_of(u, t)) continue;
                const int halves = halves_of(t), steps = stages_of(t);
                const int row0 = GATED ? t.n * 128 : t.n * 256, row1 = GATED ? row0 : row0 + 128;
                // x without an index: one box of 128 rows, or boxes of 32 when there are fewer
                const bool tall = t.live > 96;
                const int boxes = GRAD || p.gather ? 0 : tall ? 1 : (t.live + 31) / 32;
                const uint32_t bytes = (uint32_t)halves * kBytesA +
                                       (GRAD || boxes && tall ? kBytesA : (uint32_t)boxes * 32 * kRowBytes);
                // the tiles of a 128-row block of scales lie side by side along the contraction
                int left = (int)scale_tiles;
                const uint8_t *sf0, *sf1, *sfa = nullptr;
                if (GRAD) {
                    const int64_t tile0 = t.first / (4 * S::kBlock);
                    left -= (int)tile0;
                    sf0 = g.x_sf + ((int64_t)(2 * t.n) * scale_tiles + tile0) * 512;
                    sf1 = sf0 + scale_tiles * 512;
                    sfa = g.dz_sf + ((int64_t)t.m * scale_tiles + tile0) * 512;
                } else {
                    const int64_t block = GATED ? t.n : 2 * t.n, at = t.e * p.w_sf_stride + block * scale_tiles * 512;
                    sf0 = p.w_sf + at;
                    sf1 = GATED ? p.up_sf + at : sf0 + scale_tiles * 512;
                }
                int x = GRAD ? (int)(t.first * kRowBytes / S::kElems) : 0;
                for (int s = 0; s < steps; ++s, ++it, x += kRowBytes, left -= S::kScaleTiles) {
                    const int st = it % kStages;
                    if (!mbar_wait(smem_addr(&ctl->empty[st]), ((it / kStages) & 1) ^ 1, abort)) goto done;
                    const uint32_t bar = smem_addr(&ctl->full[st]), dst = base + st * kBytesData;
                    const uint32_t sf = base + kSfBase + st * kSfStage;
                    const uint32_t sf_bytes = 512u * (uint32_t)min(S::kScaleTiles, left);
                    const int64_t at = (int64_t)s * kScaleBytes;
                    mbar_arrive_tx(bar, bytes + (halves + (GRAD ? 1 : 0)) * sf_bytes);
                    bulk_load(sf + kScaleBytes, sf0 + at, sf_bytes, bar);
                    if (halves == 2) bulk_load(sf + 2 * kScaleBytes, sf1 + at, sf_bytes, bar);
                    if (GRAD) bulk_load(sf, sfa + at, sf_bytes, bar);
                    if (GRAD) {
                        tma_load_2d(dst + kBytesA, &map_b, bar, x, row0);
                        if (halves == 2) tma_load_2d(dst + 2 * kBytesA, &map_b, bar, x, row1);
                        tma_load_2d(dst, &map_a, bar, x, t.m * kTileM);
                    } else {
                        tma_load_3d(dst + kBytesA, &map_b, bar, x, row0, t.e);
                        if (halves == 2) tma_load_3d(dst + 2 * kBytesA, GATED ? &map_up : &map_b, bar, x, row1, t.e);
                        if (tall && boxes) tma_load_2d(dst, &map_a, bar, x, (int)t.first);
                        else
                            for (int b = 0; b < boxes; ++b)
                                tma_load_2d(dst + b * 32 * kRowBytes, &map_low, bar, x, (int)t.first + 32 * b);
                    }
                }
            }
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ MMA
        if (elect_one()) {
        int it = 0, done_tiles = 0;
        for (int u = blockIdx.x; u < total; u += gridDim.x) {
            Tile t;
            if (!tile_of(u, t)) continue;
            const int halves = halves_of(t), steps = stages_of(t);
            if (steps == 0) continue;
            // the epilogue of the tile before has drained the columns both accumulators share
            if (done_tiles > 0 && !mbar_wait(smem_addr(&ctl->acc_free), (done_tiles - 1) & 1, abort)) goto done;
            tc_fence_after();
            const uint32_t acc = tmem + ((done_tiles & 1) ? kAcc1 : 0);
            const int last = (int)((t.depth - (int64_t)(steps - 1) * S::kElems + S::kMma - 1) / S::kMma);
            for (int s = 0; s < steps; ++s, ++it) {
                const int st = it % kStages;
                // scale buffers are fewer than stages: the products that read this one two steps ago are done
                if (S::kScaleBufs < kStages && it >= S::kScaleBufs) {
                    const int b = it - S::kScaleBufs;
                    if (!mbar_wait(smem_addr(&ctl->empty[b % kStages]), (b / kStages) & 1, abort)) goto done;
                }
                if (!mbar_wait(smem_addr(&ctl->full[st]), (it / kStages) & 1, abort)) goto done;
                tc_fence_after();
                const int products = s + 1 < steps ? S::kElems / S::kMma : last;
                {
                    const uint32_t data = base + st * kBytesData, sfs = base + kSfBase + st * kSfStage;
                    const uint32_t col = tmem + kScaleCol + (it % S::kScaleBufs) * S::kScaleCols;
                    const uint64_t da = operand_desc(data), db = operand_desc(data + kBytesA), ds = scale_desc(sfs);
                    const uint32_t idesc = mma_idesc<FMT>(128 * halves, 0);
                    // A's tiles, then each half's: 4 columns per tile; for NVFP4 tile j of both
                    // halves lie side by side, as one product of 256 columns reads them.
                    // (Descriptors hold addresses in units of 16 bytes.)
#pragma unroll
                    for (int k = 0; k < S::kElems / S::kMma; ++k) {
                        if (k >= products) break;
                        const int j = S::kScaleTiles == 1 ? 0 : k;
                        if (j == k) {
                            tc_copy_scales(col + 4 * j, ds + 32 * j);
                            tc_copy_scales(col + 4 * S::kScaleTiles + 8 * j, ds + ((kScaleBytes + 512 * j) >> 4));
                            if (halves == 2)
                                tc_copy_scales(col + 4 * S::kScaleTiles + 8 * j + 4, ds + ((2 * kScaleBytes + 512 * j) >> 4));
                        }
                        tc_mma<FMT>(acc, da + 2 * k, db + 2 * k,
                                    idesc | (FMT == QZ_FMT_MXFP8 ? ((uint32_t)k << 4) | ((uint32_t)k << 29) : 0u), col + 4 * j,
                                    col + 4 * S::kScaleTiles + 8 * j, (s | k) != 0);
                    }
                    tc_commit(smem_addr(&ctl->empty[st]));
                    if (s + 1 == steps) tc_commit(smem_addr(&ctl->acc_full[done_tiles & 1]));
                }
            }
            ++done_tiles;
        }
        }
    } else if (warp < kRowWarps) {
        // ------------------------------------------------------------ scales of x, gathered rows
        if (!GRAD) {
            // the widest load that a row's start and length allow; x's scales need only word alignment
            const int align = aligned(p.x_sf, 16) ? 16 : aligned(p.x_sf, 8) ? 8 : 4;
            const int width = (int)min((int64_t)align, min(kv & -kv, p.ld_sf & -p.ld_sf));
            if (width == 16) scale_warp<FMT, GATED, 16>(p, list, ctl, base, total, map_low, warp, lane);
            else if (width == 8) scale_warp<FMT, GATED, 8>(p, list, ctl, base, total, map_low, warp, lane);
            else if (width == 4) scale_warp<FMT, GATED, 4>(p, list, ctl, base, total, map_low, warp, lane);
            else scale_warp<FMT, GATED, 1>(p, list, ctl, base, total, map_low, warp, lane);
        }
    } else if (warp < 4 + kEpilogueWarps) {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3, group = (warp - 4) >> 2;
        const int r = 32 * quarter + lane;  // row of the tile
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        int done_tiles = 0;
        for (int u = blockIdx.x; u < total; u += gridDim.x) {
            Tile t;
            if (!tile_of(u, t)) continue;
            const int halves = halves_of(t);
            const bool any = stages_of(t) > 0;
            if (GRAD && !any && g.accumulate) continue;
            // per-row and per-expert facts, while the products still run
            bool exists = true;
            float scale0 = 1.0f, scale1 = 1.0f;
            const int64_t slot = t.first + r;
            if (GRAD) {
                if (FMT == QZ_FMT_NVFP4) scale0 = scale1 = amax_scale(g.dz_amax, 0) * amax_scale(g.x_amax, 0);
            } else if (r < t.live) {
                // (rows in slot order still have their index: a slot without a row is zeros whatever the weights hold)
                const int64_t id = p.rows ? (int64_t)__ldg(p.rows + slot) : slot;
                exists = id >= 0 && id < p.ids;
                if (FMT == QZ_FMT_NVFP4 && exists) {
                    const float ga = amax_scale(p.x_amax, !p.x_per_row ? 0 : p.gather ? id : slot);
                    scale0 = ga * amax_scale(p.w_amax, t.e);
                    scale1 = GATED ? ga * amax_scale(p.up_amax, t.e) : scale0;
                }
            }
            const int buf = done_tiles & 1;
            const uint32_t acc = tmem + (buf ? kAcc1 : 0) + lanes;
            if (any) {
                if (!__all_sync(kFull, mbar_wait(smem_addr(&ctl->acc_full[buf]), (done_tiles >> 1) & 1, abort))) goto done;
                tc_fence_after();
                ++done_tiles;
            }
            // A warp has 64 columns of each half, in units of 32 (gated: of both halves at once).  The columns
            // shared with the other accumulator lie in one half, the second of buffer 0, the first of buffer 1:
            // its two units are loaded first, and with that the next tile's products may begin.
            const int own = buf ? 0 : 1, c0 = 64 * group;
            const int half = GATED || halves == 2 ? own : 0;
            const int units = GATED ? 2 : 2 * halves;
            float x[32], next[32];
            if (any) {
                tc_load64(acc + 128 * half + c0, x, next);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ctl->acc_free));
            }
            uint8_t* const stage = staging + (warp - 4) * kStagingBytes;
            const int64_t width = GRAD ? g.k : p.n;
            const int rows = GRAD ? (int)min((int64_t)32, g.n - (int64_t)t.m * kTileM - 32 * quarter) : t.live - 32 * quarter;
            const bool row_in = lane < rows;
#pragma unroll 1
            for (int i = 0; i < units; ++i) {
                const int h = GATED ? 0 : i < 2 ? half : 1 - half;
                const int64_t at = (GATED ? (int64_t)t.n * 128 : (int64_t)t.n * 256 + 128 * h) + c0 + 32 * (i & 1);
                const int cols = (int)min((int64_t)32, width - at);
                uint32_t w[16];
                if (cols <= 0 || rows <= 0) {
                    // nothing of this unit is in the matrix
                } else if (GRAD) {
                    scale_row<FMT>(scale0, any, x);
                    const int64_t to = (t.e * g.n + (int64_t)t.m * kTileM + 32 * quarter) * g.k + at;
                    if (g.f32) {
                        uint8_t* o = reinterpret_cast<uint8_t*>(static_cast<float*>(g.out) + to);
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(x[16 * b + j]);
                            if (g.accumulate) store_rows<true>(o + 64 * b, 4 * g.k, w, rows, 4 * (cols - 16 * b), stage, lane);
                            else store_rows<false>(o + 64 * b, 4 * g.k, w, rows, 4 * (cols - 16 * b), stage, lane);
                        }
                    } else {
                        uint16_t* o = static_cast<uint16_t*>(g.out) + to;
                        if (g.accumulate && row_in) add_row(o + lane * g.k, cols, x);
                        to_words(x, w);
                        store_rows<false>(reinterpret_cast<uint8_t*>(o), 2 * g.k, w, rows, 2 * cols, stage, lane);
                    }
                } else {
                    const int64_t slot0 = t.first + 32 * quarter;  // of lane 0
                    if (GATED) {
                        const uint32_t other = acc + 128 * (1 - own) + c0 + 32 * i;  // the half that is not held
                        if (p.pre) {
                            // the held half, then the other: z goes to columns at, u to n + at
                            float z[32];
#pragma unroll
                            for (int j = 0; j < 32; ++j) z[j] = x[j];
#pragma unroll 1
                            for (int k = 0; k < 2; ++k) {
                                const bool is_u = (own != 0) != (k == 1);
                                if (k == 1) tc_load32(other, z);
                                scale_row<FMT>(is_u ? scale1 : scale0, exists, z);
                                const uint16_t* bias = is_u ? p.up_bias : p.bias;
                                if (bias) add_row(bias + t.e * p.n + at, cols, z);
                                to_words(z, w);
                                store_rows<false>(reinterpret_cast<uint8_t*>(p.pre + slot0 * p.ld_pre + at + (is_u ? p.n : 0)),
                                                  2 * p.ld_pre, w, rows, 2 * cols, stage, lane);
                            }
                        }
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            float z[16], u[16];
                            tc_load16(other + 16 * b, u);
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float held = x[16 * b + j], o = u[j];
                                z[j] = own ? o : held;
                                u[j] = own ? held : o;
                            }
                            scale_row<FMT>(scale0, exists, z);
                            scale_row<FMT>(scale1, exists, u);
                            if (p.bias) add_row(p.bias + t.e * p.n + at + 16 * b, cols - 16 * b, z);
                            if (p.up_bias) add_row(p.up_bias + t.e * p.n + at + 16 * b, cols - 16 * b, u);
                            activate(p.act, z);
#pragma unroll
                            for (int j = 0; j < 16; ++j) z[j] *= u[j];
                            if (p.residual && row_in) add_row(p.residual + slot * p.ld_residual + at + 16 * b, cols - 16 * b, z);
#pragma unroll
                            for (int j = 0; j < 8; ++j) w[8 * b + j] = bf16x2_of(z[2 * j], z[2 * j + 1]);
                        }
                    } else if (KIND == kBare) {
                        scale_row<FMT>(scale0, exists, x);
                        to_words(x, w);
                    } else {
                        scale_row<FMT>(scale0, exists, x);
                        if (p.bias) add_row(p.bias + t.e * p.n + at, cols, x);
                        if (p.pre) {
                            to_words(x, w);
                            store_rows<false>(reinterpret_cast<uint8_t*>(p.pre + slot0 * p.ld_pre + at), 2 * p.ld_pre, w, rows,
                                              2 * cols, stage, lane);
                        }
                        activate(p.act, x);
                        if (p.residual && row_in) add_row(p.residual + slot * p.ld_residual + at, cols, x);
                        to_words(x, w);
                    }
                    store_rows<false>(reinterpret_cast<uint8_t*>(p.out + slot0 * p.ld_out + at), 2 * p.ld_out, w, rows,
                                      2 * cols, stage, lane);
                    if (p.q && row_in) {  // n is a multiple of 32: a whole block in this lane
                        uint32_t c[8];
                        const uint32_t scale = qzq::mxfp8_block(w, c);
                        uint8_t* to = p.q + slot * p.n + at;
                        if (((uintptr_t)to & 31) == 0) {
                            st_v8(to, make_uint4(c[0], c[1], c[2], c[3]), make_uint4(c[4], c[5], c[6], c[7]));
                        } else {
                            st_v4(to, make_uint4(c[0], c[1], c[2], c[3]));
                            st_v4(to + 16, make_uint4(c[4], c[5], c[6], c[7]));
                        }
                        p.sf[slot * (p.n / 32) + at / 32] = (uint8_t)scale;
                    }
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = next[j];
                if (any && i + 2 < units) tc_load32(acc + 128 * (1 - half) + c0 + 32 * i, next);
            }
        }
    }
done:
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (ctl->abort) {
        // a wait ran out: report it, and give copies in flight time to land before the memory goes
        unsigned* d_err = GRAD ? g.d_err : p.d_err;
        if (threadIdx.x == 0 && d_err) atomicOr(d_err, QZ_DERR_TIMEOUT);
        const uint64_t start = global_ns();
        while (global_ns() - start < 20000000ull) __nanosleep(1000);
    }
    tc_fence_after();
    if (warp == 3) tmem_free(tmem, 512);
}

// ---------------------------------------------------------------------------
// rows in slot order
// ---------------------------------------------------------------------------
//
// Gathering inside the product takes about 1,150 clocks a stage (32 gathers of
// four rows), twice the products, and repeats for every column block.  A large
// call with a workspace therefore copies the rows (payload, scales, amax) into
// slot order first, at the HBM's rate, and runs without an index.  A warp copies
// a slot's row.  A slot without one (a plan's unused slots above all) is left as
// it is: the epilogue does not store it, or writes zeros.
//
// The rule, with both sides measured (us in a graph, copy against gather; K 2048;
// "2 x 768" is gated):
//   slots from which the copy pays     2 x 768, 128 experts, MXFP8: 1024 slots 78 : 76, 2048 80 : 79,
//                                      4096 83 : 94, 16384 99 : 144; 4096 columns, 16 experts, NVFP4:
//                                      2048 26 : 34, 16384 93 : 153
//   one column block gathers only      256 columns, 16 experts, MXFP8: 4096 slots 16 : 20, 8192 17 : 20,
//   once: the copy pays up to 8192     16384 22 : 21, 65536 81 : 67; NVFP4: 8192 15.1 : 15.1,
//                                      16384 17.8 : 15.4
//   padded plans of few tokens are     2 x 768, 128 experts, aligned to 128, MXFP8: 16 tokens in 16384
//   mostly unused slots: up to 64      slots (1024 a token) 54 : 50, 128 in 17280 (135) 81 : 77, 256 in
//   slots a row, twice QZ_MAX_TOP_K    18304 (71) 82 : 83, 512 in 20352 (39) 83 : 88

constexpr int kCopyWarps = 8;

__global__ void __launch_bounds__(kCopyWarps * 32)
    gather_rows_kernel(const uint8_t* __restrict__ x_q, const uint8_t* __restrict__ x_sf, const float* __restrict__ x_amax,
                       const int32_t* __restrict__ rows, int64_t slots, int64_t x_rows, int64_t row_bytes, int64_t kv,
                       int64_t ld_sf, uint8_t* __restrict__ q, uint8_t* __restrict__ sf, float* __restrict__ amax) {
    const int lane = threadIdx.x & 31;
    const int64_t s = (int64_t)blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
    if (s >= slots) return;
    const int64_t r = __ldg(rows + s);
    if (r < 0 || r >= x_rows) return;
    const uint8_t* from = x_q + r * row_bytes;
    uint8_t* to = q + s * row_bytes;
    for (int64_t c = 16 * lane; c < row_bytes; c += 4 * 512) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c + 512 * i < row_bytes) v[i] = *reinterpret_cast<const uint4*>(from + c + 512 * i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + 512 * i < row_bytes) st_v4(to + c + 512 * i, v[i]);
    }
    const uint8_t* sfrom = x_sf + r * kv;
    uint8_t* sto = sf + s * ld_sf;
    if ((kv & 3) == 0) {
        for (int64_t c = 4 * lane; c < kv; c += 128)
            st_u32(sto + c, __ldg(reinterpret_cast<const uint32_t*>(sfrom + c)));
    } else {
        for (int64_t c = lane; c < kv; c += 32) sto[c] = __ldg(sfrom + c);
    }
    if (amax != nullptr && lane == 0) amax[s] = __ldg(x_amax + r);
}

constexpr int64_t kCopySlots = 2048, kCopySlotsOneBlock = 8192, kCopySlotsPerRow = 2 * QZ_MAX_TOP_K;

struct CopyLayout {
    int64_t ld_sf, q, sf, amax, total;  // scale stride, offsets and size in bytes
};

static CopyLayout copy_layout(const qz_product& p) {
    const bool fp4 = p.fmt == QZ_FMT_NVFP4;
    CopyLayout l;
    l.ld_sf = (p.k / (fp4 ? 16 : 32) + 15) / 16 * 16;  // 16 bytes of a row's scales at a time
    l.q = 0;
    l.sf = p.slots * (fp4 ? p.k / 2 : p.k);
    l.amax = l.sf + p.slots * l.ld_sf;
    l.total = l.amax + (fp4 && p.x_amax_per_row ? p.slots * 4 : 0);
    return l;
}

static int64_t column_blocks(const qz_product& p) { return p.up_q ? (p.n + 127) / 128 : (p.n + 255) / 256; }

size_t product_bytes(const qz_product& p) {
    const bool copies = p.d_rows && p.slots >= kCopySlots && (column_blocks(p) > 1 || p.slots <= kCopySlotsOneBlock) &&
                        p.slots <= kCopySlotsPerRow * p.x_rows;
    return copies ? (size_t)copy_layout(p).total : 0;
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, reached through the runtime (no link to the driver).
static EncodeTiled encoder() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// Map of `experts` matrices [rows, row_bytes] of bytes, `stride` bytes apart, read in boxes of 128 bytes x box_rows.
static bool make_map(CUtensorMap* m, const void* p, int64_t row_bytes, int64_t rows, int64_t experts, int64_t stride,
                     int box_rows) {
    const EncodeTiled fn = encoder();
    if (!fn) return false;
    const cuuint32_t rank = experts > 0 ? 3 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)row_bytes, (cuuint64_t)rows, (cuuint64_t)experts};
    const cuuint64_t strides[2] = {(cuuint64_t)row_bytes, (cuuint64_t)stride};
    const cuuint32_t box[3] = {kRowBytes, (cuuint32_t)box_rows, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(p), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int KIND>
static cudaError_t launch_experts(const Args& a, const CUtensorMap& ma, const CUtensorMap& ml, const CUtensorMap& mb,
                                  const CUtensorMap& mu, int n_experts, int grid, cudaStream_t s) {
    constexpr size_t fixed = 1024 + kStagesBytes<FMT> + kEpilogueWarps * kStagingBytes + sizeof(Control);
    // asked for at its largest: the attribute is one value per device
    constexpr size_t most = fixed + list_bytes(QZ_MAX_ROUTE_EXPERTS);
    static_assert(most <= 232448, "shared memory of a CTA");
    static std::atomic<uint64_t> set{0};  // devices that have it
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (!(set.load(std::memory_order_acquire) & bit) || bit == 0) {
        e = cudaFuncSetAttribute(experts_kernel<FMT, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_release);
    }
    experts_kernel<FMT, KIND><<<grid, kProductThreads, fixed + list_bytes(n_experts), s>>>(a, ma, ml, mb, mu);
    return cudaGetLastError();
}

cudaError_t launch_product(const qz_product& call, int ctas, cudaStream_t s, unsigned* d_err, void* ws) {
    qz_product p = call;
    bool gather = p.d_rows != nullptr;
    int64_t ld_sf = p.k / (p.fmt == QZ_FMT_NVFP4 ? 16 : 32);
    if (ws != nullptr && product_bytes(p) > 0) {
        const CopyLayout l = copy_layout(p);
        uint8_t* const w = static_cast<uint8_t*>(ws);
        float* const amax = l.total > l.amax ? reinterpret_cast<float*>(w + l.amax) : nullptr;
        gather_rows_kernel<<<(unsigned)((p.slots + kCopyWarps - 1) / kCopyWarps), kCopyWarps * 32, 0, s>>>(
            static_cast<const uint8_t*>(p.x_q), p.x_sf, p.x_amax, p.d_rows, p.slots, p.x_rows,
            p.fmt == QZ_FMT_NVFP4 ? p.k / 2 : p.k, ld_sf, l.ld_sf, w, w + l.sf, amax);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        p.x_q = w;
        p.x_sf = w + l.sf;
        if (amax) p.x_amax = amax;
        p.x_rows = p.slots;
        gather = false;
        ld_sf = l.ld_sf;
    }
    Args a = {};
    ProductArgs& q = a.p;
    q.act = p.activation;
    q.n_experts = p.n_experts;
    q.gated = p.up_q != nullptr;
    q.x_per_row = p.x_amax_per_row;
    q.gather = gather;
    q.n_blocks = (int)column_blocks(p);
    q.n = p.n;
    q.k = p.k;
    q.x_rows = p.x_rows;
    q.ids = call.x_rows;
    q.slots = p.slots;
    q.w_sf_stride = p.w_sf_stride;
    q.ld_sf = ld_sf;
    // an x without rows: every slot reads a row of zeros, so any mapped memory does
    const void* x = p.x_rows > 0 ? p.x_q : p.w_q;
    q.x_sf = p.x_sf;
    q.w_sf = p.w_sf;
    q.up_sf = p.up_sf;
    const bool fp4 = p.fmt == QZ_FMT_NVFP4;
    q.x_amax = fp4 ? p.x_amax : nullptr;
    q.w_amax = fp4 ? p.w_amax : nullptr;
    q.up_amax = fp4 ? p.up_amax : nullptr;
    q.rows = p.d_rows;
    q.offsets = p.d_offsets;
    q.counts = p.d_counts;
    q.bias = static_cast<const uint16_t*>(p.bias);
    q.up_bias = static_cast<const uint16_t*>(p.up_bias);
    q.residual = static_cast<const uint16_t*>(p.residual);
    q.out = static_cast<uint16_t*>(p.out);
    q.pre = static_cast<uint16_t*>(p.pre);
    q.ld_residual = p.ld_residual;
    q.ld_out = p.ld_out;
    q.ld_pre = p.ld_pre;
    q.q = static_cast<uint8_t*>(p.q);
    q.sf = p.sf;
    q.d_err = d_err;
    const int64_t row_bytes = fp4 ? p.k / 2 : p.k;
    const int64_t x_rows = p.x_rows > 0 ? p.x_rows : 1;
    CUtensorMap ma, ml, mb, mu;
    if (!make_map(&ml, x, row_bytes, x_rows, 0, 0, q.gather ? 1 : 32)) return cudaErrorInvalidValue;
    ma = ml;  // of tall tiles without an index only
    if (!q.gather && p.slots > 96 && !make_map(&ma, x, row_bytes, x_rows, 0, 0, 128)) return cudaErrorInvalidValue;
    if (!make_map(&mb, p.w_q, row_bytes, p.n, p.n_experts, p.w_stride, 128)) return cudaErrorInvalidValue;
    mu = mb;
    if (q.gated && !make_map(&mu, p.up_q, row_bytes, p.n, p.n_experts, p.w_stride, 128)) return cudaErrorInvalidValue;
    // no more CTAs than the slots can make tiles
    const int64_t most = ((p.slots + kTileM - 1) / kTileM + p.n_experts) * q.n_blocks;
    const int64_t rows = p.slots < p.n_experts ? p.slots * q.n_blocks : most;
    const int grid = (int)(rows < ctas ? rows : ctas);
    if (q.gated)
        return fp4 ? launch_experts<QZ_FMT_NVFP4, kGated>(a, ma, ml, mb, mu, p.n_experts, grid, s)
                   : launch_experts<QZ_FMT_MXFP8, kGated>(a, ma, ml, mb, mu, p.n_experts, grid, s);
    if (!p.bias && !p.residual && !p.pre && p.activation == QZ_ACT_NONE)
        return fp4 ? launch_experts<QZ_FMT_NVFP4, kBare>(a, ma, ml, mb, mu, p.n_experts, grid, s)
                   : launch_experts<QZ_FMT_MXFP8, kBare>(a, ma, ml, mb, mu, p.n_experts, grid, s);
    return fp4 ? launch_experts<QZ_FMT_NVFP4, kPlain>(a, ma, ml, mb, mu, p.n_experts, grid, s)
               : launch_experts<QZ_FMT_MXFP8, kPlain>(a, ma, ml, mb, mu, p.n_experts, grid, s);
}

cudaError_t launch_weight_grad(const qz_weight_grad& p, int ctas, cudaStream_t s, unsigned* d_err) {
    Args a = {};
    GradArgs& q = a.g;
    const bool fp4 = p.fmt == QZ_FMT_NVFP4;
    q.n_experts = p.n_experts;
    q.f32 = p.out_type == QZ_TYPE_F32;
    q.accumulate = p.accumulate;
    q.m_blocks = (int)((p.n + kTileM - 1) / kTileM);
    q.n_blocks = (int)((p.k + 255) / 256);
    q.n = p.n;
    q.k = p.k;
    q.slots = p.slots;
    q.dz_sf = p.dz_sf;
    q.x_sf = p.x_sf;
    q.dz_amax = p.dz_amax;
    q.x_amax = p.x_amax;
    q.offsets = p.d_offsets;
    q.counts = p.d_counts;
    q.out = p.out;
    q.d_err = d_err;
    const int64_t row_bytes = fp4 ? p.slots / 2 : p.slots;
    CUtensorMap ma, mb;
    // without slots no tile reads an operand: any mapped memory does for the maps
    const bool none = p.slots == 0;
    if (!make_map(&ma, none ? p.out : p.dz_q, none ? 16 : row_bytes, none ? 1 : p.n, 0, 0, 128)) return cudaErrorInvalidValue;
    if (!make_map(&mb, none ? p.out : p.x_q, none ? 16 : row_bytes, none ? 1 : p.k, 0, 0, 128)) return cudaErrorInvalidValue;
    const int64_t tiles = (int64_t)p.n_experts * q.m_blocks * q.n_blocks;
    if (tiles > 0x7FFF0000LL) return cudaErrorInvalidValue;  // the roles step past the last
    const int grid = (int)(tiles < ctas ? tiles : ctas);
    return fp4 ? launch_experts<QZ_FMT_NVFP4, kWeightGrad>(a, ma, ma, mb, mb, p.n_experts, grid, s)
               : launch_experts<QZ_FMT_MXFP8, kWeightGrad>(a, ma, ma, mb, mb, p.n_experts, grid, s);
}

}  // namespace qz
