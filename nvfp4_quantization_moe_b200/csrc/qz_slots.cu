// qz_slots.cu -- moves between token order and expert order (sm_100a): the
// weighted gather that ends a mixture-of-experts layer, its adjoint (the
// scatter with the routing weights' gradients), and the gradient of the
// experts' activation with the bias gradients.
//
// All three stream bf16 rows once and are bound by HBM; the arithmetic is fp32
// with one rounding to bf16 per output.  Sums that cross threads are formed in
// a fixed order (no atomics), so results repeat bit for bit.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/qz.h"
#include "qz_act.cuh"
#include "qz_device.cuh"

namespace qz {

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    f[0] = bf16_lo(v.x);
    f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y);
    f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z);
    f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w);
    f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(bf16x2_of(f[0], f[1]), bf16x2_of(f[2], f[3]), bf16x2_of(f[4], f[5]), bf16x2_of(f[6], f[7]));
}

// ---------------------------------------------------------------------------
// combine: expert order -> token order
// ---------------------------------------------------------------------------
//
// CTA (t, c): token t, 8 columns per thread.  The token's top_k rows are read
// four at a time, so that their loads are in flight together.

constexpr int kRowThreads = 128;               // 1024 columns per CTA
constexpr int kRowCols = 8 * kRowThreads;
constexpr int kU = 4;  // rows of a token whose loads are in flight together

__global__ void __launch_bounds__(kRowThreads) combine_kernel(const uint16_t* __restrict__ y, int64_t ld_y,
                                                              const int32_t* __restrict__ slots, int k,
                                                              int64_t n_slots, int64_t H,
                                                              const float* __restrict__ weights,
                                                              const uint16_t* residual, int64_t ld_r, uint16_t* out,
                                                              int64_t ld_o) {
    const int64_t t = blockIdx.x;
    const int64_t c = (int64_t)blockIdx.y * kRowCols + 8 * threadIdx.x;
    if (c >= H) return;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (residual != nullptr) unpack8(*reinterpret_cast<const uint4*>(residual + t * ld_r + c), acc);
    for (int j = 0; j < k; j += kU) {
        uint4 v[kU];
        float w[kU];
        bool live[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t s = j + u < k ? (int64_t)__ldg(slots + t * k + j + u) : -1;
            live[u] = s >= 0 && s < n_slots;
            if (live[u]) {
                v[u] = ld_stream(y + s * ld_y + c);
                w[u] = weights ? __ldg(weights + t * k + j + u) : 1.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (!live[u]) continue;
            float f[8];
            unpack8(v[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[u], f[i], acc[i]);
        }
    }
    st_v4(out + t * ld_o + c, pack8(acc));
}

// ---------------------------------------------------------------------------
// dispatch: token order -> expert order
// ---------------------------------------------------------------------------
//
// CTA t holds token t's row in registers, writes it (times each weight) to its
// slots and forms the dot products with the slots' rows of `other`, four choices
// at a time (4096 tokens of 2048 columns in 8 slots each, 418 MB with the zeros:
// 70 us one by one, 65 so); it also zeroes the unused slots of its share of the
// slots.

constexpr int kDispatchThreads = 256;
constexpr int64_t kZeroSlots = 8, kZeroCtas = 1184;  // slots a CTA looks at, CTAs that is worth (8 per SM)

template <bool DOTS>
__global__ void __launch_bounds__(kDispatchThreads)
    dispatch_kernel(const uint16_t* __restrict__ x, int64_t ld_x, const int32_t* __restrict__ slots,
                    const int32_t* __restrict__ rows, int64_t T, int k, int64_t n_slots, int64_t H,
                    const float* __restrict__ weights, uint16_t* __restrict__ y, int64_t ld_y,
                    const uint16_t* __restrict__ other, int64_t ld_o, float* __restrict__ dots) {
    __shared__ float s_dot[kDispatchThreads / 32][QZ_MAX_TOP_K];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    if (t < T) {
        if (DOTS && lane < QZ_MAX_TOP_K) s_dot[warp][lane] = 0.0f;
        __syncwarp();
        for (int64_t c = 8 * threadIdx.x; c - 8 * lane < H; c += 8 * kDispatchThreads) {
            const bool in = c < H;
            float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (in) {
                raw = ld_stream(x + t * ld_x + c);
                unpack8(raw, f);
            }
            for (int j = 0; j < k; j += kU) {
                int64_t at[kU];  // -1: no slot; the same for the whole CTA
                uint4 o[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    at[u] = j + u < k ? (int64_t)__ldg(slots + t * k + j + u) : -1;
                    if (at[u] >= n_slots) at[u] = -1;
                    o[u] = make_uint4(0, 0, 0, 0);
                    if (DOTS && in && at[u] >= 0) o[u] = ld_stream(other + at[u] * ld_o + c);
                }
                float d[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    d[u] = 0.0f;
                    if (in && at[u] >= 0) {
                        uint4 v = raw;
                        if (weights) {
                            const float w = __ldg(weights + t * k + j + u);
                            float g[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) g[i] = w * f[i];
                            v = pack8(g);
                        }
                        st_v4(y + at[u] * ld_y + c, v);
                    }
                    if (DOTS && at[u] >= 0) {  // a pair without a slot has 0, whatever the token's row holds
                        float g[8];
                        unpack8(o[u], g);
#pragma unroll
                        for (int i = 0; i < 8; ++i) d[u] = fmaf(f[i], g[i], d[u]);
                    }
                }
                if (DOTS) {
                    // four sums over the warp at once: lanes 8 u .. 8 u + 7 end up with choice u's
                    const bool hi = lane & 16, odd = lane & 8;
                    const float a = (hi ? d[2] : d[0]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? d[0] : d[2], 16);
                    const float b = (hi ? d[3] : d[1]) + __shfl_xor_sync(0xFFFFFFFFu, hi ? d[1] : d[3], 16);
                    float e = (odd ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 8);
#pragma unroll
                    for (int m = 4; m > 0; m >>= 1) e += __shfl_xor_sync(0xFFFFFFFFu, e, m);
                    if ((lane & 7) == 0 && j + lane / 8 < k) s_dot[warp][j + lane / 8] += e;
                }
            }
        }
        if (DOTS) {
            __syncthreads();
            if ((int)threadIdx.x < k) {
                float d = 0.0f;
                for (int w = 0; w < kDispatchThreads / 32; ++w) d += s_dot[w][threadIdx.x];
                dots[t * k + threadIdx.x] = d;
            }
        }
    }
    const int64_t share = (n_slots + gridDim.x - 1) / gridDim.x;
    const int64_t end = min(n_slots, (t + 1) * share);  // for CTAs past the last token too
    for (int64_t s = t * share; s < end; ++s) {
        if (__ldg(rows + s) >= 0) continue;
        for (int64_t c = 8 * threadIdx.x; c < H; c += 8 * kDispatchThreads)
            st_v4(y + s * ld_y + c, make_uint4(0, 0, 0, 0));
    }
}

// ---------------------------------------------------------------------------
// activation gradient
// ---------------------------------------------------------------------------
//
// A piece of work is `piece` rows of one expert's range (up to the next
// expert's start, so that the unused slots are zeroed on the way) x 256 columns,
// and one warp's: 8 columns per lane, four rows' loads in flight, no barriers.  A
// persistent grid takes the pieces in turn, which evens out experts of any
// length.  On 4096 x 8 rows of 2 x 768 over 128 experts that takes 71 us.  (A cluster
// per expert and column block, joined through distributed shared memory: 98 us,
// most of it waiting at barriers for uneven warps and for stores.  Refilling each
// row's registers as soon as they are used: 86 us; three CTAs per SM with two rows
// each: 82.)  A warp leaves its piece's column sums in the workspace and a second
// launch adds an expert's pieces in order.

constexpr int kGradWarps = 8;
constexpr int kGradCols = 256;
constexpr int kGradCtas = 2;       // per SM
constexpr int kRowsAhead = 4;
constexpr int64_t kMostPieces = 4096;  // pieces are 16 rows, or more when there would be more of them than this

struct GradPieces {
    const int32_t *offsets, *counts;
    int64_t slots;
    int n_experts, piece;
    int64_t most;  // pieces that the workspace holds: all there can be, unless the ranges overlap
};

// An expert's range: first slot, live slots, end (the next expert's start; the buffer's end for the last).
struct SlotRange {
    int64_t begin, count, next;
    bool bad;
};

__device__ __forceinline__ SlotRange slot_range(const GradPieces& a, int e) {
    SlotRange r;
    r.begin = __ldg(a.offsets + e);
    r.count = __ldg(a.counts + e);
    r.next = e + 1 < a.n_experts ? (int64_t)__ldg(a.offsets + e + 1) : a.slots;
    r.bad = (e == 0 ? r.begin != 0 : r.begin < 0) || r.count < 0 || r.begin + r.count > r.next || r.next > a.slots;
    return r;
}

// Pieces before each expert, in shared memory; every thread of the block must call it.
__device__ __forceinline__ int piece_prefix(const GradPieces& a, int* s_prefix, long long* s_scratch, unsigned* d_err) {
    return block_prefix(
        a.n_experts, s_prefix, s_scratch,
        [&](int e) -> long long {
            const SlotRange r = slot_range(a, e);
            if (r.bad && blockIdx.x == 0 && d_err) atomicOr(d_err, QZ_DERR_SHAPE);
            return r.bad ? 0 : (r.next - r.begin + a.piece - 1) / a.piece;
        },
        d_err);
}

template <int ACT, bool GATED>
__global__ void __launch_bounds__(kGradWarps * 32, kGradCtas)
    act_grad_kernel(GradPieces a, const uint16_t* __restrict__ dout, int64_t ld_d, const uint16_t* __restrict__ pre,
                    int64_t ld_p, int64_t n, uint16_t* __restrict__ dpre, int64_t ld_q, float* __restrict__ sums,
                    unsigned* d_err) {
    extern __shared__ int s_prefix[];
    __shared__ long long s_scratch[33];
    cudaTriggerProgrammaticLaunchCompletion();  // the bias sums wait for this launch's end before they read
    const int lane = threadIdx.x & 31;
    const int blocks = (int)((n + kGradCols - 1) / kGradCols);
    const int64_t total = (int64_t)piece_prefix(a, s_prefix, s_scratch, d_err) * blocks;
    const int64_t warps = (int64_t)gridDim.x * kGradWarps;
    for (int64_t w = (int64_t)blockIdx.x * kGradWarps + (threadIdx.x >> 5); w < total; w += warps) {
        const int p = (int)(w / blocks);
        const int64_t c = (int64_t)(w - (int64_t)p * blocks) * kGradCols + 8 * lane;
        const int e = find_owner(s_prefix, a.n_experts, p);
        const SlotRange range = slot_range(a, e);
        const int64_t first = range.begin + (int64_t)(p - s_prefix[e]) * a.piece;
        const int64_t end = min(range.next, first + a.piece), live = min(end, range.begin + range.count);
        if (c >= n) continue;
        if (p >= a.most) {  // ranges that overlap
            if (d_err && lane == 0) atomicOr(d_err, QZ_DERR_SHAPE);
            continue;
        }
        float sz[8] = {0, 0, 0, 0, 0, 0, 0, 0}, su[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int64_t s0 = first; s0 < live; s0 += kRowsAhead) {
            uint4 vd[kRowsAhead], vz[kRowsAhead], vu[kRowsAhead];
#pragma unroll
            for (int k = 0; k < kRowsAhead; ++k) {
                const int64_t s = s0 + k;
                if (s >= live) continue;
                vd[k] = ld_stream(dout + s * ld_d + c);
                vz[k] = ld_stream(pre + s * ld_p + c);
                if (GATED) vu[k] = ld_stream(pre + s * ld_p + n + c);
            }
#pragma unroll
            for (int k = 0; k < kRowsAhead; ++k) {
                const int64_t s = s0 + k;
                if (s >= live) continue;
                float d[8], z[8], dz[8];
                unpack8(vd[k], d);
                unpack8(vz[k], z);
                if (GATED) {
                    float u[8], du[8];
                    unpack8(vu[k], u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const ActPair q = act_with_grad<ACT>(z[j]);
                        du[j] = d[j] * q.value;
                        dz[j] = d[j] * u[j] * q.grad;
                        su[j] += du[j];
                        sz[j] += dz[j];
                    }
                    st_v4(dpre + s * ld_q + n + c, pack8(du));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        dz[j] = d[j] * act_with_grad<ACT>(z[j]).grad;
                        sz[j] += dz[j];
                    }
                }
                st_v4(dpre + s * ld_q + c, pack8(dz));
            }
        }
        for (int64_t s = max(first, live); s < end; ++s) {
            st_v4(dpre + s * ld_q + c, make_uint4(0, 0, 0, 0));
            if (GATED) st_v4(dpre + s * ld_q + n + c, make_uint4(0, 0, 0, 0));
        }
        if (sums != nullptr) {
            if (live <= first) continue;  // no piece of a live row: not read either
            float* to = sums + (int64_t)p * (GATED ? 2 * n : n) + c;
#pragma unroll
            for (int h = 0; h < (GATED ? 2 : 1); ++h) {
                const float(&v)[8] = h ? su : sz;
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    st_v4(to + h * n + 4 * q, make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                                         __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])));
            }
        }
    }
}

// CTA (c, e): 128 columns of expert e's dbias, four per lane.  Warp w adds one
// eighth of the expert's pieces in order, then the eighths are added in order.
constexpr int kSumCols = 128;

__global__ void __launch_bounds__(kGradWarps * 32)
    bias_sum_kernel(GradPieces a, const float* sums, int64_t width, float* __restrict__ dbias) {
    __shared__ int s_before[kGradWarps];
    __shared__ float4 s_part[kGradWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.y;
    const int64_t c = (int64_t)blockIdx.x * kSumCols + 4 * lane;
    const SlotRange range = slot_range(a, e);
    if (range.bad) return;  // the same for the whole CTA
    int before = 0;         // pieces of the experts before this one
    for (int i = threadIdx.x; i < e; i += kGradWarps * 32) {
        const SlotRange r = slot_range(a, i);
        if (!r.bad) before += (int)((r.next - r.begin + a.piece - 1) / a.piece);
    }
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    if (lane == 0) s_before[warp] = before;
    __syncthreads();
    before = 0;
#pragma unroll
    for (int w = 0; w < kGradWarps; ++w) before += s_before[w];
    const int pieces = (int)((range.count + a.piece - 1) / a.piece);  // with live rows
    if (before + pieces > a.most) return;
    const int each = (pieces + kGradWarps - 1) / kGradWarps, end = min(pieces, (warp + 1) * each);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    cudaGridDependencySynchronize();
    if (c < width) {
        const float* from = sums + (int64_t)before * width + c;
#pragma unroll 4
        for (int p = warp * each; p < end; ++p) {
            const float4 u = ld_written_v4(from + (int64_t)p * width);
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
    }
    s_part[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < width) {
#pragma unroll
        for (int w = 1; w < kGradWarps; ++w) {
            const float4 u = s_part[w][lane];
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
        }
        float* to = dbias + (int64_t)e * width + c;  // only float-aligned
        to[0] = v.x;
        to[1] = v.y;
        to[2] = v.z;
        to[3] = v.w;
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

cudaError_t launch_combine(const uint16_t* y, int64_t ld_y, const int32_t* slots, int64_t T, int k, int64_t n_slots,
                           int64_t H, const float* weights, const uint16_t* residual, int64_t ld_r, uint16_t* out,
                           int64_t ld_o, cudaStream_t s) {
    const dim3 grid((unsigned)T, (unsigned)((H + kRowCols - 1) / kRowCols));
    combine_kernel<<<grid, kRowThreads, 0, s>>>(y, ld_y, slots, k, n_slots, H, weights, residual, ld_r, out, ld_o);
    return cudaGetLastError();
}

cudaError_t launch_dispatch(const uint16_t* x, int64_t ld_x, const int32_t* slots, const int32_t* rows, int64_t T,
                            int k, int64_t n_slots, int64_t H, const float* weights, uint16_t* y, int64_t ld_y,
                            const uint16_t* other, int64_t ld_o, float* dots, cudaStream_t s) {
    // a CTA per token, and enough of them for the unused slots when there are few tokens (16 tokens over
    // 128 experts padded to 128: 16,000 rows of zeros)
    const int64_t zeroing = (n_slots + kZeroSlots - 1) / kZeroSlots;
    const int64_t most = zeroing < kZeroCtas ? zeroing : kZeroCtas;
    const unsigned grid = (unsigned)(T > most ? T : most > 0 ? most : 1);
    if (other)
        dispatch_kernel<true><<<grid, kDispatchThreads, 0, s>>>(x, ld_x, slots, rows, T, k, n_slots, H, weights, y,
                                                                ld_y, other, ld_o, dots);
    else
        dispatch_kernel<false><<<grid, kDispatchThreads, 0, s>>>(x, ld_x, slots, rows, T, k, n_slots, H, weights, y,
                                                                 ld_y, nullptr, 0, nullptr);
    return cudaGetLastError();
}

static int grad_piece(int64_t slots) {
    int piece = 16;
    while ((slots + piece - 1) / piece > kMostPieces) piece *= 2;
    return piece;
}

// Each expert's last piece may be short.
static int64_t most_pieces(int64_t slots, int n_experts) { return slots / grad_piece(slots) + n_experts; }

size_t act_grad_bytes(int64_t slots, int64_t n, bool gated, int n_experts) {
    return (size_t)most_pieces(slots, n_experts) * (size_t)(gated ? 2 * n : n) * sizeof(float);
}

cudaError_t launch_act_grad(const uint16_t* dout, int64_t ld_d, const uint16_t* pre, int64_t ld_p, int64_t slots,
                            int64_t n, int act, bool gated, const int32_t* offsets, const int32_t* counts,
                            int n_experts, uint16_t* dpre, int64_t ld_q, float* dbias, float* sums, int sms, cudaStream_t s,
                            unsigned* d_err) {
    typedef void (*Kernel)(GradPieces, const uint16_t*, int64_t, const uint16_t*, int64_t, int64_t, uint16_t*, int64_t, float*,
                           unsigned*);
    static const Kernel kernels[4][2] = {
        {act_grad_kernel<QZ_ACT_NONE, false>, act_grad_kernel<QZ_ACT_NONE, true>},
        {act_grad_kernel<QZ_ACT_RELU, false>, act_grad_kernel<QZ_ACT_RELU, true>},
        {act_grad_kernel<QZ_ACT_SILU, false>, act_grad_kernel<QZ_ACT_SILU, true>},
        {act_grad_kernel<QZ_ACT_GELU, false>, act_grad_kernel<QZ_ACT_GELU, true>},
    };
    const GradPieces a = {offsets, counts, slots, n_experts, grad_piece(slots), most_pieces(slots, n_experts)};
    const int64_t ctas = (a.most * ((n + kGradCols - 1) / kGradCols) + kGradWarps - 1) / kGradWarps;
    const unsigned grid = (unsigned)(ctas < (int64_t)sms * kGradCtas ? ctas : (int64_t)sms * kGradCtas);
    const size_t smem = (size_t)(n_experts + 1) * sizeof(int);
    kernels[act][gated]<<<grid, kGradWarps * 32, smem, s>>>(a, dout, ld_d, pre, ld_p, n, dpre, ld_q,
                                                            dbias ? sums : nullptr, d_err);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || dbias == nullptr) return e;
    const int64_t width = gated ? 2 * n : n;
    cudaLaunchAttribute beside;  // its lists are read beside the first launch's end
    beside.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    beside.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3((unsigned)((width + kSumCols - 1) / kSumCols), (unsigned)n_experts);
    config.blockDim = dim3(kGradWarps * 32);
    config.stream = s;
    config.attrs = &beside;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, bias_sum_kernel, a, (const float*)sums, width, dbias);
}

}  // namespace qz
