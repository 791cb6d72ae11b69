// qz_product.cu -- the experts' block-scaled matrix products (sm_100a).
//
// A tile of 64 slots x 64 columns per CTA: each step decodes 32 elements of
// every row to fp32 in shared memory and multiplies on the CUDA cores.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/qz.h"
#include "../../include/qz_quant.cuh"
#include "qz_act.cuh"
#include "qz_device.cuh"

namespace qz {

constexpr int kPT = 64;   // tile rows and columns
constexpr int kPK = 32;   // contraction elements per step

// Value of element i of a row of block-scaled codes without its second-level scale.
template <int FMT>
__device__ __forceinline__ float coded_value(const uint8_t* q, const uint8_t* sf, int64_t i, uint32_t scale) {
    if (FMT == QZ_FMT_MXFP8) {
        const uint32_t c = q[i];
        const float v = e4m3_value(c & 0x7Fu);
        const float p = scale == 0 ? 0x1p-127f : __uint_as_float(scale << 23);
        return ((c & 0x80u) ? -v : v) * p;
    }
    const uint32_t c = (q[i >> 1] >> ((i & 1) * 4)) & 15u;
    const uint32_t m = c & 7u;
    const float v = m < 2 ? 0.5f * (float)m : (float)((2u | (m & 1u)) << (m >> 1)) * 0.25f;
    return ((c & 8u) ? -v : v) * e4m3_value(scale);
}

__device__ __forceinline__ float activate(int act, float z) {
    if (act == QZ_ACT_RELU) return act_value<QZ_ACT_RELU>(z);
    if (act == QZ_ACT_SILU) return act_value<QZ_ACT_SILU>(z);
    if (act == QZ_ACT_GELU) return act_value<QZ_ACT_GELU>(z);
    return z;
}

__device__ __forceinline__ float decode_scale(const float* amax, int64_t i) {
    return amax ? __fdiv_rn(__ldg(amax + i), 2688.0f) : 1.0f;
}

// Which expert and which of its row tiles work item u is; false past the end.
__device__ __forceinline__ bool find_tile(const qz_product& p, int u, int& e, int64_t& first, int64_t& live) {
    for (e = 0; e < p.n_experts; ++e) {
        const int64_t off = __ldg(p.d_offsets + e), cnt = __ldg(p.d_counts + e);
        if (off < 0 || cnt <= 0 || off + cnt > p.slots) continue;
        const int64_t tiles = (cnt + kPT - 1) / kPT;
        if (u < tiles) {
            first = off + (int64_t)u * kPT;
            live = min((int64_t)kPT, cnt - (int64_t)u * kPT);
            return true;
        }
        u -= (int)tiles;
    }
    return false;
}

template <int FMT>
__global__ void __launch_bounds__(256) product_kernel(qz_product p, unsigned* d_err) {
    constexpr int BLOCK = FMT == QZ_FMT_MXFP8 ? 32 : 16;
    constexpr int EB = FMT == QZ_FMT_MXFP8 ? 1 : 2;  // elements per byte
    __shared__ float s_a[kPK][kPT + 1], s_b[2][kPK][kPT + 1];
    __shared__ int s_row[kPT];
    if (blockIdx.x == 0 && blockIdx.y == 0 && d_err) {
        for (int e = threadIdx.x; e < p.n_experts; e += blockDim.x) {
            const int64_t off = p.d_offsets[e], cnt = p.d_counts[e];
            if (off < 0 || cnt < 0 || off + cnt > p.slots) atomicOr(d_err, QZ_DERR_SHAPE);
        }
    }
    int e;
    int64_t first, live;
    if (!find_tile(p, blockIdx.y, e, first, live)) return;
    const int64_t n0 = (int64_t)blockIdx.x * kPT, kv = p.k / BLOCK;
    const bool gated = p.up_q != nullptr;
    if (threadIdx.x < kPT) {
        int r = -1;
        if (threadIdx.x < live) {
            r = p.d_rows ? __ldg(p.d_rows + first + threadIdx.x) : (int)(first + threadIdx.x);
            if (r < 0 || r >= p.x_rows) r = -1;
        }
        s_row[threadIdx.x] = r;
    }
    __syncthreads();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[2][4][4] = {};
    for (int64_t k0 = 0; k0 < p.k; k0 += kPK) {
        for (int i = threadIdx.x; i < kPT * kPK; i += blockDim.x) {
            const int r = i / kPK, c = i % kPK;
            const int64_t kk = k0 + c, row = s_row[r];
            float v = 0.0f;
            if (row >= 0)
                v = coded_value<FMT>(static_cast<const uint8_t*>(p.x_q) + row * (p.k / EB), nullptr, kk,
                                     p.x_sf[row * kv + kk / BLOCK]);
            s_a[c][r] = v;
            for (int h = 0; h < (gated ? 2 : 1); ++h) {
                const uint8_t* q = static_cast<const uint8_t*>(h ? p.up_q : p.w_q) + e * p.w_stride;
                const uint8_t* sf = (h ? p.up_sf : p.w_sf) + e * p.w_sf_stride;
                float w = 0.0f;
                if (n0 + r < p.n)
                    w = coded_value<FMT>(q + (n0 + r) * (p.k / EB), nullptr, kk, sf[swz_offset(n0 + r, kk / BLOCK, kv)]);
                s_b[h][c][r] = w;
            }
        }
        __syncthreads();
        for (int c = 0; c < kPK; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float av = s_a[c][ty * 4 + i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[0][i][j] = fmaf(av, s_b[0][c][tx * 4 + j], acc[0][i][j]);
                    if (gated) acc[1][i][j] = fmaf(av, s_b[1][c][tx * 4 + j], acc[1][i][j]);
                }
            }
        }
        __syncthreads();
    }
    // epilogue: out in place of s_a / s_b is not needed for bf16; the MXFP8 form
    // is made from the bf16 values once the tile is in shared memory
    __shared__ uint16_t s_o[kPT][kPT];
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        const int64_t s = first + r;
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx * 4 + j;
            float h = 0.0f;
            if (r < live && n < p.n) {
                const int row = s_row[r];
                const float ga = row >= 0 ? decode_scale(p.x_amax, p.x_amax_per_row ? row : 0) : 1.0f;
                float z = acc[0][i][j] * (ga * decode_scale(p.w_amax, e));
                if (p.bias) z += bf16_lo(static_cast<const uint16_t*>(p.bias)[e * p.n + n]);
                if (p.pre) static_cast<uint16_t*>(p.pre)[s * p.ld_pre + n] = (uint16_t)bf16x2_of(z, 0.0f);
                h = activate(p.activation, z);
                if (gated) {
                    float u = acc[1][i][j] * (ga * decode_scale(p.up_amax, e));
                    if (p.up_bias) u += bf16_lo(static_cast<const uint16_t*>(p.up_bias)[e * p.n + n]);
                    if (p.pre) static_cast<uint16_t*>(p.pre)[s * p.ld_pre + p.n + n] = (uint16_t)bf16x2_of(u, 0.0f);
                    h *= u;
                }
                if (p.residual) h += bf16_lo(static_cast<const uint16_t*>(p.residual)[s * p.ld_residual + n]);
                static_cast<uint16_t*>(p.out)[s * p.ld_out + n] = (uint16_t)bf16x2_of(h, 0.0f);
            }
            s_o[r][tx * 4 + j] = (uint16_t)bf16x2_of(h, 0.0f);
        }
    }
    if (!p.q) return;
    __syncthreads();
    if (threadIdx.x < 2 * kPT) {
        const int r = threadIdx.x >> 1, b = threadIdx.x & 1;
        const int64_t n = n0 + 32 * b;
        if (r < live && n < p.n) {
            uint32_t x[16], q[8];
            for (int i = 0; i < 16; ++i) x[i] = (uint32_t)s_o[r][32 * b + 2 * i] | ((uint32_t)s_o[r][32 * b + 2 * i + 1] << 16);
            const uint32_t sc = qzq::mxfp8_block(x, q);
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.q) + (first + r) * p.n + n);
            dst[0] = make_uint4(q[0], q[1], q[2], q[3]);
            dst[1] = make_uint4(q[4], q[5], q[6], q[7]);
            p.sf[(first + r) * (p.n / 32) + n / 32] = (uint8_t)sc;
        }
    }
}

template <int FMT>
__global__ void __launch_bounds__(256) weight_grad_kernel(qz_weight_grad p, unsigned* d_err) {
    constexpr int BLOCK = FMT == QZ_FMT_MXFP8 ? 32 : 16;
    constexpr int EB = FMT == QZ_FMT_MXFP8 ? 1 : 2;
    __shared__ float s_a[kPK][kPT + 1], s_b[kPK][kPT + 1];
    const int e = blockIdx.z;
    const int64_t off = __ldg(p.d_offsets + e), cnt = __ldg(p.d_counts + e);
    const bool shape = off < 0 || cnt < 0 || off + cnt > p.slots, align = (off & 127) != 0;
    if (shape || align) {
        if (d_err && threadIdx.x == 0) atomicOr(d_err, (shape ? QZ_DERR_SHAPE : 0u) | (align ? QZ_DERR_ALIGN : 0u));
        return;
    }
    const int64_t r0 = (int64_t)blockIdx.y * kPT, c0 = (int64_t)blockIdx.x * kPT, kv = p.slots / BLOCK;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < cnt; k0 += kPK) {
        for (int i = threadIdx.x; i < kPT * kPK; i += blockDim.x) {
            const int r = i / kPK, c = i % kPK;
            const int64_t s = off + k0 + c;
            float a = 0.0f, b = 0.0f;
            if (k0 + c < cnt) {
                if (r0 + r < p.n)
                    a = coded_value<FMT>(static_cast<const uint8_t*>(p.dz_q) + (r0 + r) * (p.slots / EB), nullptr, s,
                                         p.dz_sf[swz_offset(r0 + r, s / BLOCK, kv)]);
                if (c0 + r < p.k)
                    b = coded_value<FMT>(static_cast<const uint8_t*>(p.x_q) + (c0 + r) * (p.slots / EB), nullptr, s,
                                         p.x_sf[swz_offset(c0 + r, s / BLOCK, kv)]);
            }
            s_a[c][r] = a;
            s_b[c][r] = b;
        }
        __syncthreads();
        for (int c = 0; c < kPK; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s_a[c][ty * 4 + i], s_b[c][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
    const float g = decode_scale(p.dz_amax, 0) * decode_scale(p.x_amax, 0);
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + ty * 4 + i, c = c0 + tx * 4 + j;
            if (r >= p.n || c >= p.k) continue;
            const int64_t at = (e * p.n + r) * p.k + c;
            float v = acc[i][j] * g;
            if (p.out_type == QZ_TYPE_F32) {
                float* o = static_cast<float*>(p.out) + at;
                *o = p.accumulate ? *o + v : v;
            } else {
                uint16_t* o = static_cast<uint16_t*>(p.out) + at;
                if (p.accumulate) v += bf16_lo(*o);
                *o = (uint16_t)bf16x2_of(v, 0.0f);
            }
        }
    }
}

cudaError_t launch_product(const qz_product& p, cudaStream_t s, unsigned* d_err) {
    const int64_t most = (p.slots + kPT - 1) / kPT + p.n_experts;
    const dim3 grid((unsigned)((p.n + kPT - 1) / kPT), (unsigned)(most < 65535 ? most : 65535));
    if (p.fmt == QZ_FMT_MXFP8) product_kernel<QZ_FMT_MXFP8><<<grid, 256, 0, s>>>(p, d_err);
    else product_kernel<QZ_FMT_NVFP4><<<grid, 256, 0, s>>>(p, d_err);
    return cudaGetLastError();
}

cudaError_t launch_weight_grad(const qz_weight_grad& p, cudaStream_t s, unsigned* d_err) {
    const dim3 grid((unsigned)((p.k + kPT - 1) / kPT), (unsigned)((p.n + kPT - 1) / kPT), (unsigned)p.n_experts);
    if (p.fmt == QZ_FMT_MXFP8) weight_grad_kernel<QZ_FMT_MXFP8><<<grid, 256, 0, s>>>(p, d_err);
    else weight_grad_kernel<QZ_FMT_NVFP4><<<grid, 256, 0, s>>>(p, d_err);
    return cudaGetLastError();
}

}  // namespace qz
