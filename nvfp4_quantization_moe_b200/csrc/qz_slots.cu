// qz_slots.cu -- moves between token order and expert order (sm_100a): the
// weighted gather that ends a mixture-of-experts layer, its adjoint (the
// scatter with the routing weights' gradients), and the gradient of the
// experts' activation with the bias gradients.
//
// All three stream bf16 rows once and are bound by HBM; the arithmetic is fp32
// with one rounding to bf16 per output.  Sums that cross threads are formed in
// a fixed order (no atomics), so results repeat bit for bit.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/qz.h"
#include "qz_act.cuh"
#include "qz_device.cuh"

namespace qz {

namespace cg = cooperative_groups;

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
    constexpr int kU = 4;
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
// slots and forms the dot products with the slots' rows of `other`; it also
// zeroes the unused slots of its share of the slots.

constexpr int kDispatchThreads = 256;

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
            for (int j = 0; j < k; ++j) {
                const int64_t s = __ldg(slots + t * k + j);
                if (s < 0 || s >= n_slots) continue;  // the same for the whole CTA
                uint4 o = make_uint4(0, 0, 0, 0);
                if (DOTS && in) o = ld_stream(other + s * ld_o + c);
                if (in) {
                    if (weights) {
                        const float w = __ldg(weights + t * k + j);
                        float g[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) g[i] = w * f[i];
                        st_v4(y + s * ld_y + c, pack8(g));
                    } else {
                        st_v4(y + s * ld_y + c, raw);
                    }
                }
                if (DOTS) {
                    float g[8];
                    unpack8(o, g);
                    float d = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) d = fmaf(f[i], g[i], d);
#pragma unroll
                    for (int b = 16; b > 0; b >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, b);
                    if (lane == 0) s_dot[warp][j] += d;
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
    const int64_t end = min(n_slots, (t + 1) * share);
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
// CTA (c, r, e): 256 columns of the rows of expert e that cluster rank r owns.
// A warp takes one row at a time, 8 columns per lane, and keeps its columns'
// sums; the warps' sums, then the cluster's (through distributed shared
// memory), are added in a fixed order.  The cluster of 8 splits an expert's
// rows because there are too few (expert, column block) pairs to fill the GPU.

constexpr int kGradWarps = 8;
constexpr int kGradCols = 256;
constexpr int kGradSplit = 8;  // cluster size
constexpr int kRowsAhead = 2;

template <int ACT, bool GATED>
__global__ void __launch_bounds__(kGradWarps * 32, 3) __cluster_dims__(1, kGradSplit, 1)
    act_grad_kernel(const uint16_t* __restrict__ dout, int64_t ld_d, const uint16_t* __restrict__ pre, int64_t ld_p,
                    int64_t slots, int64_t n, const int32_t* __restrict__ offsets,
                    const int32_t* __restrict__ counts, int n_experts, uint16_t* __restrict__ dpre, int64_t ld_q,
                    float* __restrict__ dbias, unsigned* d_err) {
    __shared__ float s_sum[kGradWarps][(GATED ? 2 : 1) * kGradCols];
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.z, r = blockIdx.y;
    const int64_t c = (int64_t)blockIdx.x * kGradCols + 8 * lane;
    const int64_t begin = __ldg(offsets + e);
    int64_t count = __ldg(counts + e);
    // the rows up to the next expert's (the end of the buffer for the last) are this expert's to zero
    int64_t next = e + 1 < n_experts ? (int64_t)__ldg(offsets + e + 1) : slots;
    const bool bad = begin < 0 || count < 0 || begin + count > slots || next < begin + count || next > slots;
    if (bad) {
        if (d_err && r == 0 && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(d_err, QZ_DERR_SHAPE);
        count = 0;
        next = begin;
    }
    float sz[8] = {0, 0, 0, 0, 0, 0, 0, 0}, su[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (c < n) {
        // kRowsAhead rows' loads are in flight before the first is used
        constexpr int64_t kStep = kGradSplit * kGradWarps;
        for (int64_t i0 = r * kGradWarps + warp; i0 < count; i0 += kRowsAhead * kStep) {
            uint4 vd[kRowsAhead], vz[kRowsAhead], vu[kRowsAhead];
#pragma unroll
            for (int k = 0; k < kRowsAhead; ++k) {
                const int64_t s = begin + i0 + k * kStep;
                if (i0 + k * kStep >= count) continue;
                vd[k] = ld_stream(dout + s * ld_d + c);
                vz[k] = ld_stream(pre + s * ld_p + c);
                if (GATED) vu[k] = ld_stream(pre + s * ld_p + n + c);
            }
#pragma unroll
            for (int k = 0; k < kRowsAhead; ++k) {
                const int64_t s = begin + i0 + k * kStep;
                if (i0 + k * kStep >= count) continue;
                float d[8], z[8], dz[8];
                unpack8(vd[k], d);
                unpack8(vz[k], z);
                if (GATED) {
                    float u[8], du[8];
                    unpack8(vu[k], u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const ActPair p = act_with_grad<ACT>(z[j]);
                        du[j] = d[j] * p.value;
                        dz[j] = d[j] * u[j] * p.grad;
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
        for (int64_t s = begin + count + r * kGradWarps + warp; s < next; s += kGradSplit * kGradWarps) {
            st_v4(dpre + s * ld_q + c, make_uint4(0, 0, 0, 0));
            if (GATED) st_v4(dpre + s * ld_q + n + c, make_uint4(0, 0, 0, 0));
        }
    }
    if (dbias == nullptr) return;  // the same for every CTA of the cluster
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        s_sum[warp][8 * lane + j] = sz[j];
        if (GATED) s_sum[warp][kGradCols + 8 * lane + j] = su[j];
    }
    __syncthreads();
    const int width = (GATED ? 2 : 1) * kGradCols;
    for (int i = threadIdx.x; i < width; i += blockDim.x) {
        float v = 0.0f;
        for (int w = 0; w < kGradWarps; ++w) v += s_sum[w][i];
        s_sum[0][i] = v;
    }
    cluster.sync();
    if (r == 0) {
        for (int i = threadIdx.x; i < width; i += blockDim.x) {
            const int64_t col = (int64_t)blockIdx.x * kGradCols + (i % kGradCols);
            if (col >= n) continue;
            float v = 0.0f;
            for (int q = 0; q < kGradSplit; ++q) v += cluster.map_shared_rank(&s_sum[0][0], q)[i];
            if (!bad) dbias[(int64_t)e * (GATED ? 2 * n : n) + (i / kGradCols) * n + col] = v;
        }
    }
    cluster.sync();  // no CTA leaves while its sums may still be read
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
    const unsigned grid = (unsigned)(T > 0 ? T : 1);  // T == 0: one CTA zeroes every slot
    if (other)
        dispatch_kernel<true><<<grid, kDispatchThreads, 0, s>>>(x, ld_x, slots, rows, T, k, n_slots, H, weights, y,
                                                                ld_y, other, ld_o, dots);
    else
        dispatch_kernel<false><<<grid, kDispatchThreads, 0, s>>>(x, ld_x, slots, rows, T, k, n_slots, H, weights, y,
                                                                 ld_y, nullptr, 0, nullptr);
    return cudaGetLastError();
}

template <int ACT>
static cudaError_t act_grad_launch(bool gated, dim3 grid, const uint16_t* dout, int64_t ld_d, const uint16_t* pre, int64_t ld_p,
                                   int64_t slots, int64_t n, const int32_t* offsets, const int32_t* counts, int n_experts,
                                   uint16_t* dpre, int64_t ld_q, float* dbias, cudaStream_t s, unsigned* d_err) {
    if (gated)
        act_grad_kernel<ACT, true><<<grid, kGradWarps * 32, 0, s>>>(dout, ld_d, pre, ld_p, slots, n, offsets, counts, n_experts,
                                                                    dpre, ld_q, dbias, d_err);
    else
        act_grad_kernel<ACT, false><<<grid, kGradWarps * 32, 0, s>>>(dout, ld_d, pre, ld_p, slots, n, offsets, counts, n_experts,
                                                                     dpre, ld_q, dbias, d_err);
    return cudaGetLastError();
}

cudaError_t launch_act_grad(const uint16_t* dout, int64_t ld_d, const uint16_t* pre, int64_t ld_p, int64_t slots,
                            int64_t n, int act, bool gated, const int32_t* offsets, const int32_t* counts,
                            int n_experts, uint16_t* dpre, int64_t ld_q, float* dbias, cudaStream_t s,
                            unsigned* d_err) {
    const dim3 grid((unsigned)((n + kGradCols - 1) / kGradCols), kGradSplit, (unsigned)n_experts);
    switch (act) {
        case QZ_ACT_RELU:
            return act_grad_launch<QZ_ACT_RELU>(gated, grid, dout, ld_d, pre, ld_p, slots, n, offsets, counts, n_experts, dpre,
                                                ld_q, dbias, s, d_err);
        case QZ_ACT_SILU:
            return act_grad_launch<QZ_ACT_SILU>(gated, grid, dout, ld_d, pre, ld_p, slots, n, offsets, counts, n_experts, dpre,
                                                ld_q, dbias, s, d_err);
        case QZ_ACT_GELU:
            return act_grad_launch<QZ_ACT_GELU>(gated, grid, dout, ld_d, pre, ld_p, slots, n, offsets, counts, n_experts, dpre,
                                                ld_q, dbias, s, d_err);
        default:
            return act_grad_launch<QZ_ACT_NONE>(gated, grid, dout, ld_d, pre, ld_p, slots, n, offsets, counts, n_experts, dpre,
                                                ld_q, dbias, s, d_err);
    }
}

}  // namespace qz
