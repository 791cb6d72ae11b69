// qz_api.cu -- the extern "C" entry points declared in include/qz.h.
//
// Host side only: argument checks that need no device memory, grid sizing
// (one wave of resident CTAs on every SM, cached per device), and the
// launches.  Nothing here allocates, synchronizes or reads device memory.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>
#include <mutex>

#include "../../include/qz.h"

namespace qz {
cudaError_t launch_mxfp8(const qz_expert* table, int n, int layout, int grid, cudaStream_t s, unsigned* d_err,
                         bool independent);
cudaError_t launch_nvfp4_tensor(const qz_expert* table, int n, int layout, bool compute_amax, int grid,
                                cudaStream_t s, unsigned* d_err, bool independent);
cudaError_t launch_nvfp4_rows(const qz_expert* table, int n, int layout, int grid, cudaStream_t s, unsigned* d_err);
cudaError_t launch_swizzle(const qz_sf_pair* table, int n, int grid, cudaStream_t s, unsigned* d_err);
cudaError_t launch_rmsnorm_quant(const uint16_t* x, const uint16_t* r, const uint16_t* g, float eps, int64_t T,
                                 int64_t H, uint16_t* y, uint16_t* h, int fmt, uint8_t* q, uint8_t* sf, int layout,
                                 const float* amax, cudaStream_t s, bool latency_mode);
cudaError_t launch_allreduce_norm_quant(const uint16_t* const* xs, int n_x, const uint16_t* r, const uint16_t* g,
                                        float eps, int64_t T, int64_t H, int64_t row_begin, int64_t row_end,
                                        const qz_norm_dest* dsts, int n_dst, int fmt, int layout, const float* amax,
                                        cudaStream_t s, bool latency_mode);
int grouped_blocks_per_sm(int which, int n);
size_t workspace_bytes(int n);
cudaError_t launch_nvfp4_compute_l2(const qz_expert* table, int n, int layout, int grid, unsigned* ws,
                                    cudaStream_t s, unsigned* d_err, long long wait_ns, unsigned test_flags);
cudaError_t launch_nvfp4_compute_l2_static(const qz_expert* table, int n, int layout, int grid, cudaStream_t s,
                                           unsigned* d_err, long long wait_ns, unsigned test_flags);
int rows_blocks_per_sm(int n);
cudaError_t launch_dequant(const qz_dq_expert* table, int n, int fmt, bool per_row, int layout, int grid,
                           cudaStream_t s, unsigned* d_err);
int dequant_blocks_per_sm(int n, int fmt);
cudaError_t launch_colwise(const qz_expert* table, int n, int fmt, int layout, int grid, cudaStream_t s,
                           unsigned* d_err);
int colwise_blocks_per_sm(int n, int fmt);
cudaError_t launch_split_fused(const qz_fused_split* table, int n, int fmt, int amax_kind, int src_layout,
                               int dst_layout, int grid, cudaStream_t s, unsigned* d_err);
int split_blocks_per_sm(int n);
cudaError_t launch_attention_merge(const float* O, const float* lse, int S, int64_t T, int64_t H, uint16_t* y,
                                   uint8_t* q, uint8_t* sf, int layout, cudaStream_t s);
cudaError_t launch_route(const void* logits, int type, int64_t T, int E, int64_t ld, const float* bias,
                         const qz_router& r, int32_t* ids, float* weights, cudaStream_t s);
cudaError_t launch_route_grad(const void* logits, int type, int64_t T, int E, int64_t ld, const qz_router& r,
                              const int32_t* ids, const float* dweights, void* dlogits, int64_t ldd, cudaStream_t s);
size_t plan_bytes(int64_t n, int E);
cudaError_t launch_plan(const int32_t* ids, int64_t T, int k, int E, int align, int64_t slots, int32_t* offsets,
                        int32_t* counts, int32_t* rows, int32_t* pair_slots, void* ws, cudaStream_t s);
size_t product_bytes(const qz_product& p);
cudaError_t launch_product(const qz_product& call, int ctas, cudaStream_t s, unsigned* d_err, void* ws);
cudaError_t launch_weight_grad(const qz_weight_grad& p, int ctas, cudaStream_t s, unsigned* d_err);
cudaError_t launch_act_grad(const uint16_t* dout, int64_t ld_d, const uint16_t* pre, int64_t ld_p, int64_t slots,
                            int64_t n, int act, bool gated, const int32_t* offsets, const int32_t* counts,
                            int n_experts, uint16_t* dpre, int64_t ld_q, float* dbias, float* sums, int sms, cudaStream_t s,
                            unsigned* d_err);
size_t act_grad_bytes(int64_t slots, int64_t n, bool gated, int n_experts);
cudaError_t launch_dispatch(const uint16_t* x, int64_t ld_x, const int32_t* slots, const int32_t* rows, int64_t T,
                            int k, int64_t n_slots, int64_t H, const float* weights, uint16_t* y, int64_t ld_y,
                            const uint16_t* other, int64_t ld_o, float* dots, cudaStream_t s);
cudaError_t launch_combine(const uint16_t* y, int64_t ld_y, const int32_t* slots, int64_t T, int k, int64_t n_slots,
                           int64_t H, const float* weights, const uint16_t* residual, int64_t ld_r, uint16_t* out,
                           int64_t ld_o, cudaStream_t s);
}  // namespace qz

namespace {

constexpr int kMaxDevices = 64;
constexpr int kKinds = 11;  // mxfp8, nvfp4 tile, swizzle, amax, rows, computed-amax L2 path, dequantize MXFP8,
                            // colwise MXFP8, fused split, dequantize NVFP4, colwise NVFP4

struct DeviceLimits {
    int sms = 0;
    int per_sm[kKinds] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
};

std::mutex g_mu;
DeviceLimits g_dev[kMaxDevices];

// One wave of resident CTAs for kernel `kind` on the current device.  The
// occupancy is taken once per device with the largest prefix table, so the
// cached value never over-subscribes a smaller call.
int wave_grid(int kind, const qz_launch_opts* opts) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    int grid;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        DeviceLimits& d = g_dev[dev];
        if (d.sms == 0) {
            int sms = 0;
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            d.sms = sms > 0 ? sms : 1;
        }
        if (d.per_sm[kind] == 0)
            d.per_sm[kind] = (kind == 4)   ? qz::rows_blocks_per_sm(QZ_MAX_EXPERTS)
                             : (kind == 6) ? qz::dequant_blocks_per_sm(QZ_MAX_EXPERTS, QZ_FMT_MXFP8)
                             : (kind == 9) ? qz::dequant_blocks_per_sm(QZ_MAX_EXPERTS, QZ_FMT_NVFP4)
                             : (kind == 7) ? qz::colwise_blocks_per_sm(QZ_MAX_EXPERTS, QZ_FMT_MXFP8)
                             : (kind == 10) ? qz::colwise_blocks_per_sm(QZ_MAX_EXPERTS, QZ_FMT_NVFP4)
                             : (kind == 8) ? qz::split_blocks_per_sm(QZ_MAX_EXPERTS)
                                           : qz::grouped_blocks_per_sm(kind, QZ_MAX_EXPERTS);
        grid = d.sms * d.per_sm[kind];
    }
    if (opts && opts->max_ctas > 0 && opts->max_ctas < grid) grid = opts->max_ctas;
    return grid;
}

// SM count of the current device (cached).
int device_sms() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceLimits& d = g_dev[dev];
    if (d.sms == 0) {
        int sms = 0;
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        d.sms = sms > 0 ? sms : 1;
    }
    return d.sms;
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

unsigned* err_word(const qz_launch_opts* opts) { return opts ? opts->d_err : nullptr; }
long long wait_limit(const qz_launch_opts* opts) { return opts ? (long long)opts->wait_limit_ns : 0; }
unsigned test_flags(const qz_launch_opts* opts) { return opts ? opts->test_flags : 0u; }
bool independent(const qz_launch_opts* opts) { return opts && (opts->launch_flags & QZ_OPT_INDEPENDENT) != 0u; }

qz_status check_table(const void* table, int n) {
    if (n < 0 || n > QZ_MAX_EXPERTS) return QZ_ERR_INVALID_ARG;
    if (n > 0 && table == nullptr) return QZ_ERR_INVALID_ARG;
    return QZ_OK;
}

bool valid_layout(int layout) { return layout == QZ_SF_LINEAR || layout == QZ_SF_SWIZZLED_128x4; }

qz_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QZ_OK : QZ_ERR_CUDA; }

// Grid of the MXFP8 tile kernels (quantize, dequantize): with an element
// count, about one CTA per kTilesPerCta tiles in whole waves (at most
// kMaxWaves), since the hardware's placement of many short CTAs streams a
// large call faster than one persistent wave (measured: 5.4 -> 6.6 TB/s on
// 128 experts of 3072 x 4096), and a call of fewer tiles than one wave
// launches one CTA per tile; a cap in opts->max_ctas still applies.  The
// NVFP4 kernels measured slower that way and keep one wave.
constexpr int64_t kTilesPerCta = 10;
constexpr int64_t kMaxWaves = 16;

int sized_grid(int kind, const qz_launch_opts* opts) {
    const int wave = wave_grid(kind, nullptr);
    int grid = wave;
    if (opts && opts->elems_hint > 0) {
        const int64_t tiles = (opts->elems_hint + 16383) / 16384;
        int64_t waves = (tiles + kTilesPerCta * wave / 2) / (kTilesPerCta * wave);  // rounded
        waves = waves < 1 ? 1 : (waves > kMaxWaves ? kMaxWaves : waves);
        grid = (int)(wave * waves);
        if (tiles < grid) grid = (int)tiles;  // a small call launches no idle CTAs
    }
    if (opts && opts->max_ctas > 0 && opts->max_ctas < grid) grid = opts->max_ctas;
    return grid;
}

constexpr int64_t kMaxIndex = 0x7FFFFFFFLL;  // slots, rows and tokens are int32 on the device

bool finite(float v) { return v - v == 0.0f; }

// The router arguments that the forward and the gradient share.
qz_status check_router(const void* logits, int type, int64_t T, int E, int64_t ld, const qz_router* r) {
    if (!r || (type != QZ_TYPE_BF16 && type != QZ_TYPE_F32)) return QZ_ERR_INVALID_ARG;
    if (T < 0 || T > kMaxIndex / QZ_MAX_TOP_K || E < 1 || E > QZ_MAX_ROUTE_EXPERTS || ld < E) return QZ_ERR_INVALID_ARG;
    if (r->score != QZ_SCORE_SOFTMAX && r->score != QZ_SCORE_SIGMOID) return QZ_ERR_INVALID_ARG;
    if (r->top_k < 1 || r->top_k > QZ_MAX_TOP_K || r->top_k > E || !finite(r->scale)) return QZ_ERR_INVALID_ARG;
    if (T > 0 && !logits) return QZ_ERR_INVALID_ARG;
    if (!aligned(logits, type == QZ_TYPE_BF16 ? 2 : 4)) return QZ_ERR_ALIGNMENT;
    return QZ_OK;
}

// A row stride of a bf16 matrix of `cols` columns read 16 bytes at a time.
bool valid_ld(int64_t ld, int64_t cols) { return ld >= cols && ld % 8 == 0 && ld <= QZ_MAX_LD; }

// CTAs of the product kernels: one per SM, or the call's cap.
int one_per_sm(const qz_launch_opts* opts) {
    const int sms = device_sms();
    return opts && opts->max_ctas > 0 && opts->max_ctas < sms ? opts->max_ctas : sms;
}

bool valid_activation(int a) { return a >= QZ_ACT_NONE && a <= QZ_ACT_GELU; }

qz_status check_rows(const void* a, const void* b, const int32_t* slots, int64_t T, int top_k, int64_t n_slots,
                     int64_t H) {
    if (T < 0 || T > kMaxIndex || n_slots < 0 || n_slots > kMaxIndex) return QZ_ERR_INVALID_ARG;
    if (top_k < 1 || top_k > QZ_MAX_TOP_K || H < 8 || H % 8 != 0 || H > QZ_MAX_LD) return QZ_ERR_INVALID_ARG;
    if ((T > 0 && !slots) || (T > 0 && !a) || (n_slots > 0 && !b)) return QZ_ERR_INVALID_ARG;
    return QZ_OK;
}

}  // namespace

extern "C" {

size_t qz_sf_bytes(int64_t rows, int64_t cols, int fmt, int layout) {
    if (fmt == QZ_FMT_FP8_BLOCK128) {
        if (layout != QZ_SF_LINEAR || rows <= 0 || cols <= 0) return 0;
        return (size_t)(4 * ((rows + 127) / 128) * ((cols + 127) / 128));
    }
    if (fmt != QZ_FMT_MXFP8 && fmt != QZ_FMT_NVFP4) return 0;
    if (!valid_layout(layout)) return 0;
    const int64_t block = fmt == QZ_FMT_MXFP8 ? 32 : 16;
    if (rows <= 0 || cols <= 0 || cols % block != 0) return 0;
    const int64_t kv = cols / block;
    if (layout == QZ_SF_LINEAR) return (size_t)(rows * kv);
    return (size_t)(((rows + 127) / 128) * 128 * ((kv + 3) / 4) * 4);
}

qz_status qz_quantize_grouped_mxfp8(const qz_expert* d_table, int n_experts, int layout, void* stream,
                                    const qz_launch_opts* opts) {
    qz_status st = check_table(d_table, n_experts);
    if (st != QZ_OK) return st;
    if (!valid_layout(layout)) return QZ_ERR_INVALID_ARG;
    if (n_experts == 0) return QZ_OK;
    return from_cuda(qz::launch_mxfp8(d_table, n_experts, layout, sized_grid(0, opts), (cudaStream_t)stream,
                                      err_word(opts), independent(opts)));
}

qz_status qz_quantize_grouped_nvfp4(const qz_expert* d_table, int n_experts, int mode, int layout, void* stream,
                                    const qz_launch_opts* opts) {
    qz_status st = check_table(d_table, n_experts);
    if (st != QZ_OK) return st;
    if (!valid_layout(layout)) return QZ_ERR_INVALID_ARG;
    if (mode != QZ_NVFP4_PER_TENSOR_GIVEN && mode != QZ_NVFP4_PER_TENSOR_COMPUTE && mode != QZ_NVFP4_PER_ROW)
        return QZ_ERR_INVALID_ARG;
    if (opts && opts->wait_limit_ns < 0) return QZ_ERR_INVALID_ARG;
    if (mode == QZ_NVFP4_PER_TENSOR_COMPUTE && opts && opts->d_workspace) {
        if (n_experts > 0 && opts->workspace_bytes < qz::workspace_bytes(n_experts)) return QZ_ERR_INVALID_ARG;
        if (!aligned(opts->d_workspace, 4)) return QZ_ERR_ALIGNMENT;
    }
    if (n_experts == 0) return QZ_OK;
    cudaStream_t s = (cudaStream_t)stream;
    if (mode == QZ_NVFP4_PER_TENSOR_COMPUTE && opts && opts->d_workspace)
        return from_cuda(qz::launch_nvfp4_compute_l2(d_table, n_experts, layout, wave_grid(5, opts),
                                                     static_cast<unsigned*>(opts->d_workspace), s, err_word(opts),
                                                     wait_limit(opts), test_flags(opts)));
    if (mode == QZ_NVFP4_PER_ROW)
        return from_cuda(qz::launch_nvfp4_rows(d_table, n_experts, layout, wave_grid(4, opts), s, err_word(opts)));
    return from_cuda(qz::launch_nvfp4_tensor(d_table, n_experts, layout, mode == QZ_NVFP4_PER_TENSOR_COMPUTE,
                                             wave_grid(1, opts), s, err_word(opts), independent(opts)));
}

qz_status qz_rmsnorm_quantize(const void* d_x, const void* d_residual, const void* d_gamma, float eps, int64_t T,
                              int64_t H, void* d_norm_out, void* d_residual_out, int fmt, void* d_q, uint8_t* d_sf,
                              int layout, const float* d_global_amax, void* stream) {
    if (fmt != QZ_FMT_MXFP8 && fmt != QZ_FMT_NVFP4) return QZ_ERR_INVALID_ARG;
    if (!valid_layout(layout)) return QZ_ERR_INVALID_ARG;
    const int64_t block = fmt == QZ_FMT_MXFP8 ? 32 : 16;
    if (T < 0 || H <= 0 || H > QZ_MAX_HIDDEN || H % block != 0) return QZ_ERR_INVALID_ARG;
    if (T > 0x7FFFFF00LL) return QZ_ERR_INVALID_ARG;
    if (layout == QZ_SF_SWIZZLED_128x4 && (H / block) % 4 != 0) return QZ_ERR_UNSUPPORTED;
    if (T == 0) return QZ_OK;
    if (!d_x || !d_residual || !d_gamma || !d_norm_out || !d_q || !d_sf) return QZ_ERR_INVALID_ARG;
    if (fmt == QZ_FMT_NVFP4 && !d_global_amax) return QZ_ERR_INVALID_ARG;
    if (!aligned(d_x, 16) || !aligned(d_residual, 16) || !aligned(d_gamma, 16) || !aligned(d_norm_out, 16) ||
        (d_residual_out && !aligned(d_residual_out, 16)))
        return QZ_ERR_ALIGNMENT;
    if (!aligned(d_q, 8) || !aligned(d_sf, layout == QZ_SF_SWIZZLED_128x4 ? 16 : 4)) return QZ_ERR_ALIGNMENT;
    if (d_global_amax && !aligned(d_global_amax, 4)) return QZ_ERR_ALIGNMENT;
    const bool latency_mode = T <= 2 * (int64_t)device_sms();
    return from_cuda(qz::launch_rmsnorm_quant(
        static_cast<const uint16_t*>(d_x), static_cast<const uint16_t*>(d_residual),
        static_cast<const uint16_t*>(d_gamma), eps, T, H, static_cast<uint16_t*>(d_norm_out),
        static_cast<uint16_t*>(d_residual_out), fmt, static_cast<uint8_t*>(d_q), d_sf, layout, d_global_amax,
        (cudaStream_t)stream, latency_mode));
}

qz_status qz_allreduce_rmsnorm_quantize(const void* const* rank_x, int n_ranks, const void* d_residual,
                                        const void* d_gamma, float eps, int64_t T, int64_t H, int64_t row_begin,
                                        int64_t row_end, const qz_norm_dest* dests, int n_dests, int fmt,
                                        int layout, const float* d_global_amax, void* stream) {
    if (fmt != QZ_FMT_MXFP8 && fmt != QZ_FMT_NVFP4) return QZ_ERR_INVALID_ARG;
    if (!valid_layout(layout)) return QZ_ERR_INVALID_ARG;
    if (n_ranks < 1 || n_ranks > QZ_MAX_RANKS || n_dests < 1 || n_dests > QZ_MAX_RANKS) return QZ_ERR_INVALID_ARG;
    if (!rank_x || !dests) return QZ_ERR_INVALID_ARG;
    const int64_t block = fmt == QZ_FMT_MXFP8 ? 32 : 16;
    if (T < 0 || H <= 0 || H > QZ_MAX_HIDDEN || H % block != 0) return QZ_ERR_INVALID_ARG;
    if (T > 0x7FFFFF00LL) return QZ_ERR_INVALID_ARG;
    if (row_begin < 0 || row_begin > row_end || row_end > T) return QZ_ERR_INVALID_ARG;
    if (layout == QZ_SF_SWIZZLED_128x4 && (H / block) % 4 != 0) return QZ_ERR_UNSUPPORTED;
    if (T == 0) return QZ_OK;
    if (!d_residual || !d_gamma || (fmt == QZ_FMT_NVFP4 && !d_global_amax)) return QZ_ERR_INVALID_ARG;
    for (int i = 0; i < n_ranks; ++i)
        if (!rank_x[i]) return QZ_ERR_INVALID_ARG;
    for (int d = 0; d < n_dests; ++d)
        if (!dests[d].norm_out || !dests[d].q || !dests[d].sf) return QZ_ERR_INVALID_ARG;
    if (!aligned(d_residual, 16) || !aligned(d_gamma, 16)) return QZ_ERR_ALIGNMENT;
    if (d_global_amax && !aligned(d_global_amax, 4)) return QZ_ERR_ALIGNMENT;
    for (int i = 0; i < n_ranks; ++i)
        if (!aligned(rank_x[i], 16)) return QZ_ERR_ALIGNMENT;
    for (int d = 0; d < n_dests; ++d) {
        const qz_norm_dest& o = dests[d];
        if (!aligned(o.norm_out, 16) || (o.residual_out && !aligned(o.residual_out, 16)) || !aligned(o.q, 8) ||
            !aligned(o.sf, layout == QZ_SF_SWIZZLED_128x4 ? 16 : 4))
            return QZ_ERR_ALIGNMENT;
    }
    const bool latency_mode = row_end - row_begin <= 2 * (int64_t)device_sms();
    return from_cuda(qz::launch_allreduce_norm_quant(
        reinterpret_cast<const uint16_t* const*>(rank_x), n_ranks, static_cast<const uint16_t*>(d_residual),
        static_cast<const uint16_t*>(d_gamma), eps, T, H, row_begin, row_end, dests, n_dests, fmt, layout,
        d_global_amax, (cudaStream_t)stream, latency_mode));
}

qz_status qz_swizzle_scales(const qz_sf_pair* d_table, int n, void* stream, const qz_launch_opts* opts) {
    qz_status st = check_table(d_table, n);
    if (st != QZ_OK) return st;
    if (n == 0) return QZ_OK;
    return from_cuda(qz::launch_swizzle(d_table, n, wave_grid(2, opts), (cudaStream_t)stream, err_word(opts)));
}

qz_status qz_quantize_grouped_nvfp4_compute_noalloc(const qz_expert* d_table, int n_experts, int layout,
                                                    void* stream, const qz_launch_opts* opts) {
    if (n_experts < 0 || n_experts > QZ_STATIC_WS_MAX_EXPERTS) return QZ_ERR_INVALID_ARG;
    if (n_experts > 0 && d_table == nullptr) return QZ_ERR_INVALID_ARG;
    if (opts && opts->wait_limit_ns < 0) return QZ_ERR_INVALID_ARG;
    if (!valid_layout(layout)) return QZ_ERR_INVALID_ARG;
    if (n_experts == 0) return QZ_OK;
    return from_cuda(qz::launch_nvfp4_compute_l2_static(d_table, n_experts, layout, wave_grid(5, opts),
                                                        (cudaStream_t)stream, err_word(opts), wait_limit(opts),
                                                        test_flags(opts)));
}

qz_status qz_dequantize_grouped(const qz_dq_expert* d_table, int n_experts, int fmt, int per_row, int layout,
                                void* stream, const qz_launch_opts* opts) {
    qz_status st = check_table(d_table, n_experts);
    if (st != QZ_OK) return st;
    if (!valid_layout(layout)) return QZ_ERR_INVALID_ARG;
    if (fmt != QZ_FMT_MXFP8 && fmt != QZ_FMT_NVFP4) return QZ_ERR_INVALID_ARG;
    if (n_experts == 0) return QZ_OK;
    return from_cuda(qz::launch_dequant(d_table, n_experts, fmt, per_row != 0, layout,
                                        fmt == QZ_FMT_MXFP8 ? sized_grid(6, opts) : wave_grid(9, opts),
                                        (cudaStream_t)stream, err_word(opts)));
}

qz_status qz_quantize_grouped_colwise(const qz_expert* d_table, int n_experts, int fmt, int layout, void* stream,
                                      const qz_launch_opts* opts) {
    qz_status st = check_table(d_table, n_experts);
    if (st != QZ_OK) return st;
    if (!valid_layout(layout)) return QZ_ERR_INVALID_ARG;
    if (fmt != QZ_FMT_MXFP8 && fmt != QZ_FMT_NVFP4) return QZ_ERR_INVALID_ARG;
    if (n_experts == 0) return QZ_OK;
    return from_cuda(qz::launch_colwise(d_table, n_experts, fmt, layout,
                                        wave_grid(fmt == QZ_FMT_MXFP8 ? 7 : 10, opts), (cudaStream_t)stream,
                                        err_word(opts)));
}

qz_status qz_attention_merge_quantize(const float* d_partial, const float* d_lse, int S, int64_t T, int64_t H,
                                      void* d_out, void* d_q, uint8_t* d_sf, int layout, void* stream) {
    if (S < 1 || S > QZ_MAX_SPLITS || T < 0 || T > 0x7FFFFFFFLL) return QZ_ERR_INVALID_ARG;
    if (H <= 0 || H % 32 != 0 || H > QZ_MAX_HIDDEN) return QZ_ERR_INVALID_ARG;
    if (!valid_layout(layout)) return QZ_ERR_INVALID_ARG;
    if (d_q && layout == QZ_SF_SWIZZLED_128x4 && (H / 32) % 4 != 0) return QZ_ERR_UNSUPPORTED;
    if (T == 0) return QZ_OK;
    if (!d_partial || !d_lse || !d_out || (d_q && !d_sf)) return QZ_ERR_INVALID_ARG;
    if (!aligned(d_partial, 16) || !aligned(d_out, 16)) return QZ_ERR_ALIGNMENT;
    if (d_q && (!aligned(d_q, 8) || (layout == QZ_SF_SWIZZLED_128x4 && !aligned(d_sf, 16)))) return QZ_ERR_ALIGNMENT;
    return from_cuda(qz::launch_attention_merge(d_partial, d_lse, S, T, H, static_cast<uint16_t*>(d_out),
                                                static_cast<uint8_t*>(d_q), d_sf, layout, (cudaStream_t)stream));
}

qz_status qz_split_fused_experts(const qz_fused_split* d_table, int n, int fmt, int amax_kind, int src_layout,
                                 int dst_layout, void* stream, const qz_launch_opts* opts) {
    qz_status st = check_table(d_table, n);
    if (st != QZ_OK) return st;
    if (fmt != QZ_FMT_MXFP8 && fmt != QZ_FMT_NVFP4 && fmt != QZ_FMT_FP8_BLOCK128) return QZ_ERR_INVALID_ARG;
    if (amax_kind != QZ_AMAX_NONE && amax_kind != QZ_AMAX_PER_TENSOR && amax_kind != QZ_AMAX_PER_ROW)
        return QZ_ERR_INVALID_ARG;
    if (fmt != QZ_FMT_NVFP4 && amax_kind != QZ_AMAX_NONE) return QZ_ERR_INVALID_ARG;
    if (!valid_layout(src_layout) || !valid_layout(dst_layout)) return QZ_ERR_INVALID_ARG;
    if (fmt == QZ_FMT_FP8_BLOCK128 && (src_layout != QZ_SF_LINEAR || dst_layout != QZ_SF_LINEAR))
        return QZ_ERR_UNSUPPORTED;
    if (n == 0) return QZ_OK;
    return from_cuda(qz::launch_split_fused(d_table, n, fmt, amax_kind, src_layout, dst_layout, wave_grid(8, opts),
                                            (cudaStream_t)stream, err_word(opts)));
}

qz_status qz_ipc_export(const void* d_ptr, qz_ipc_handle* out) {
    if (!d_ptr || !out) return QZ_ERR_INVALID_ARG;
    static_assert(sizeof(cudaIpcMemHandle_t) == sizeof(out->handle), "IPC handle size");
    // the allocation's start and size: the driver's address-range query,
    // reached through the runtime so the library needs no link to the driver
    typedef int (*AddressRange)(unsigned long long*, size_t*, unsigned long long);
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &fn, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess || !fn)
        return QZ_ERR_CUDA;
    unsigned long long base = 0;
    size_t size = 0;
    if (reinterpret_cast<AddressRange>(fn)(&base, &size, (unsigned long long)(uintptr_t)d_ptr) != 0) return QZ_ERR_CUDA;
    cudaIpcMemHandle_t h;
    if (cudaIpcGetMemHandle(&h, reinterpret_cast<void*>(base)) != cudaSuccess) return QZ_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QZ_ERR_CUDA;
    memcpy(out->handle, &h, sizeof(h));
    out->offset = (uint64_t)((uintptr_t)d_ptr - base);
    out->alloc_bytes = (uint64_t)size;
    out->device = dev;
    out->reserved = 0;
    return QZ_OK;
}

qz_status qz_ipc_import(const qz_ipc_handle* h, void** d_ptr_out) {
    if (!h || !d_ptr_out) return QZ_ERR_INVALID_ARG;
    cudaIpcMemHandle_t ipc;
    memcpy(&ipc, h->handle, sizeof(ipc));
    void* base = nullptr;
    if (cudaIpcOpenMemHandle(&base, ipc, cudaIpcMemLazyEnablePeerAccess) != cudaSuccess) return QZ_ERR_CUDA;
    *d_ptr_out = static_cast<char*>(base) + h->offset;
    return QZ_OK;
}

qz_status qz_ipc_close(void* d_ptr, const qz_ipc_handle* h) {
    if (!d_ptr || !h) return QZ_ERR_INVALID_ARG;
    return from_cuda(cudaIpcCloseMemHandle(static_cast<char*>(d_ptr) - h->offset));
}

qz_status qz_route_experts(const void* d_logits, int type, int64_t T, int E, int64_t ld, const float* d_bias,
                           const qz_router* router, int32_t* d_ids, float* d_weights, void* stream) {
    qz_status st = check_router(d_logits, type, T, E, ld, router);
    if (st != QZ_OK) return st;
    if (router->n_groups < 1 || router->n_groups > QZ_MAX_GROUPS || E % router->n_groups != 0) return QZ_ERR_INVALID_ARG;
    if (router->top_groups < 1 || router->top_groups > router->n_groups ||
        router->top_k > router->top_groups * (E / router->n_groups))
        return QZ_ERR_INVALID_ARG;
    if (T == 0) return QZ_OK;
    if (!d_ids || !d_weights) return QZ_ERR_INVALID_ARG;
    if (!aligned(d_ids, 4) || !aligned(d_weights, 4) || !aligned(d_bias, 4)) return QZ_ERR_ALIGNMENT;
    return from_cuda(qz::launch_route(d_logits, type, T, E, ld, d_bias, *router, d_ids, d_weights,
                                      (cudaStream_t)stream));
}

qz_status qz_route_experts_grad(const void* d_logits, int type, int64_t T, int E, int64_t ld, const qz_router* router,
                                const int32_t* d_ids, const float* d_dweights, void* d_dlogits, int64_t ldd,
                                void* stream) {
    qz_status st = check_router(d_logits, type, T, E, ld, router);
    if (st != QZ_OK) return st;
    if (ldd < E) return QZ_ERR_INVALID_ARG;
    if (T == 0) return QZ_OK;
    if (!d_ids || !d_dweights || !d_dlogits) return QZ_ERR_INVALID_ARG;
    if (!aligned(d_ids, 4) || !aligned(d_dweights, 4) || !aligned(d_dlogits, type == QZ_TYPE_BF16 ? 2 : 4))
        return QZ_ERR_ALIGNMENT;
    return from_cuda(qz::launch_route_grad(d_logits, type, T, E, ld, *router, d_ids, d_dweights, d_dlogits, ldd,
                                           (cudaStream_t)stream));
}

int64_t qz_plan_slots(int64_t T, int top_k, int E, int align) {
    if (T < 0 || T > kMaxIndex / QZ_MAX_TOP_K || top_k < 1 || top_k > QZ_MAX_TOP_K) return 0;
    if (E < 1 || E > QZ_MAX_ROUTE_EXPERTS || align < 1 || align > 1024 || (align & (align - 1)) != 0) return 0;
    const int64_t n = T * top_k;
    const int64_t s = (n + (E < n ? E : n) * (align - 1) + align - 1) / align * align;
    return s <= kMaxIndex ? s : 0;
}

size_t qz_plan_bytes(int64_t T, int top_k, int E) {
    if (T < 0 || T > kMaxIndex / QZ_MAX_TOP_K || top_k < 1 || top_k > QZ_MAX_TOP_K) return 0;
    if (E < 1 || E > QZ_MAX_ROUTE_EXPERTS) return 0;
    return qz::plan_bytes(T * top_k, E);
}

qz_status qz_plan_experts(const int32_t* d_ids, int64_t T, int top_k, int E, int align, int32_t* d_offsets,
                          int32_t* d_counts, int32_t* d_rows, int32_t* d_slots, void* d_workspace,
                          size_t workspace_bytes, void* stream) {
    if (T < 0 || T > kMaxIndex / QZ_MAX_TOP_K || top_k < 1 || top_k > QZ_MAX_TOP_K) return QZ_ERR_INVALID_ARG;
    if (E < 1 || E > QZ_MAX_ROUTE_EXPERTS || align < 1 || align > 1024 || (align & (align - 1)) != 0)
        return QZ_ERR_INVALID_ARG;
    const int64_t slots = qz_plan_slots(T, top_k, E, align);
    if (!d_offsets || !d_counts || (T > 0 && (slots == 0 || !d_ids || !d_rows || !d_slots))) return QZ_ERR_INVALID_ARG;
    const size_t need = qz::plan_bytes(T * top_k, E);
    if (need > 0 && (!d_workspace || workspace_bytes < need)) return QZ_ERR_INVALID_ARG;
    if (!aligned(d_ids, 4) || !aligned(d_offsets, 4) || !aligned(d_counts, 4) || !aligned(d_rows, 4) ||
        !aligned(d_slots, 4) || !aligned(d_workspace, 4))
        return QZ_ERR_ALIGNMENT;
    return from_cuda(qz::launch_plan(d_ids, T, top_k, E, align, slots, d_offsets, d_counts, d_rows, d_slots,
                                     d_workspace, (cudaStream_t)stream));
}

qz_status qz_expert_product(const qz_product* p, void* stream, const qz_launch_opts* opts) {
    if (!p) return QZ_ERR_INVALID_ARG;
    if (p->fmt != QZ_FMT_MXFP8 && p->fmt != QZ_FMT_NVFP4) return QZ_ERR_INVALID_ARG;
    if (!valid_activation(p->activation)) return QZ_ERR_INVALID_ARG;
    if (p->n_experts < 1 || p->n_experts > QZ_MAX_ROUTE_EXPERTS) return QZ_ERR_INVALID_ARG;
    if (p->n < 8 || p->n % 8 != 0 || p->n > QZ_MAX_LD || p->k < 32 || p->k % 32 != 0 || p->k > QZ_MAX_LD)
        return QZ_ERR_INVALID_ARG;
    if (p->x_rows < 0 || p->x_rows > kMaxIndex || p->slots < 0 || p->slots > kMaxIndex) return QZ_ERR_INVALID_ARG;
    const bool gated = p->up_q != nullptr, fp4 = p->fmt == QZ_FMT_NVFP4;
    const int64_t row_bytes = fp4 ? p->k / 2 : p->k;
    if (p->w_stride < p->n * row_bytes || p->w_stride % 16 != 0) return QZ_ERR_INVALID_ARG;
    if (p->w_sf_stride < (int64_t)qz_sf_bytes(p->n, p->k, p->fmt, QZ_SF_SWIZZLED_128x4) || p->w_sf_stride % 16 != 0)
        return QZ_ERR_INVALID_ARG;
    if (!valid_ld(p->ld_out, p->n) || (p->residual && !valid_ld(p->ld_residual, p->n)) ||
        (p->pre && !valid_ld(p->ld_pre, gated ? 2 * p->n : p->n)))
        return QZ_ERR_INVALID_ARG;
    if (!gated && (p->up_sf || p->up_amax || p->up_bias)) return QZ_ERR_INVALID_ARG;
    if (p->q && (p->n % 32 != 0 || !p->sf)) return QZ_ERR_INVALID_ARG;
    if (p->slots == 0) return QZ_OK;
    if (!p->d_offsets || !p->d_counts || !p->w_q || !p->w_sf || !p->out) return QZ_ERR_INVALID_ARG;
    if (p->x_rows > 0 && (!p->x_q || !p->x_sf || (fp4 && !p->x_amax))) return QZ_ERR_INVALID_ARG;
    if (gated && (!p->up_sf || (fp4 && !p->up_amax))) return QZ_ERR_INVALID_ARG;
    if (fp4 && !p->w_amax) return QZ_ERR_INVALID_ARG;
    if (!aligned(p->x_q, 16) || !aligned(p->w_q, 16) || !aligned(p->up_q, 16) || !aligned(p->w_sf, 16) ||
        !aligned(p->up_sf, 16) || !aligned(p->out, 16) || !aligned(p->residual, 16) || !aligned(p->pre, 16) ||
        !aligned(p->q, 16) || !aligned(p->bias, 16) || !aligned(p->up_bias, 16))
        return QZ_ERR_ALIGNMENT;
    if (!aligned(p->x_sf, 4) || !aligned(p->x_amax, 4) || !aligned(p->w_amax, 4) || !aligned(p->up_amax, 4) ||
        !aligned(p->d_rows, 4) || !aligned(p->d_offsets, 4) || !aligned(p->d_counts, 4))
        return QZ_ERR_ALIGNMENT;
    void* const ws = opts ? opts->d_workspace : nullptr;
    if (ws && opts->workspace_bytes < qz::product_bytes(*p)) return QZ_ERR_INVALID_ARG;
    if (!aligned(ws, 16)) return QZ_ERR_ALIGNMENT;
    return from_cuda(qz::launch_product(*p, one_per_sm(opts), (cudaStream_t)stream, err_word(opts), ws));
}

size_t qz_product_bytes(const qz_product* p) {
    if (!p || (p->fmt != QZ_FMT_MXFP8 && p->fmt != QZ_FMT_NVFP4) || p->k < 32 || p->k % 32 != 0 || p->k > QZ_MAX_LD ||
        p->slots < 0 || p->slots > kMaxIndex)
        return 0;
    return qz::product_bytes(*p);
}

qz_status qz_expert_weight_grad(const qz_weight_grad* p, void* stream, const qz_launch_opts* opts) {
    if (!p) return QZ_ERR_INVALID_ARG;
    if (p->fmt != QZ_FMT_MXFP8 && p->fmt != QZ_FMT_NVFP4) return QZ_ERR_INVALID_ARG;
    if (p->out_type != QZ_TYPE_BF16 && p->out_type != QZ_TYPE_F32) return QZ_ERR_INVALID_ARG;
    if (p->n_experts < 1 || p->n_experts > QZ_MAX_ROUTE_EXPERTS) return QZ_ERR_INVALID_ARG;
    if (p->n < 8 || p->n % 8 != 0 || p->n > QZ_MAX_LD || p->k < 8 || p->k % 8 != 0 || p->k > QZ_MAX_LD)
        return QZ_ERR_INVALID_ARG;
    if (p->slots < 0 || p->slots % 32 != 0 || p->slots > kMaxIndex) return QZ_ERR_INVALID_ARG;
    if (!p->d_offsets || !p->d_counts || !p->out) return QZ_ERR_INVALID_ARG;
    if (p->slots > 0 && (!p->dz_q || !p->dz_sf || !p->x_q || !p->x_sf)) return QZ_ERR_INVALID_ARG;
    if (p->slots > 0 && p->fmt == QZ_FMT_NVFP4 && (!p->dz_amax || !p->x_amax)) return QZ_ERR_INVALID_ARG;
    if (!aligned(p->dz_q, 16) || !aligned(p->x_q, 16) || !aligned(p->dz_sf, 16) || !aligned(p->x_sf, 16) ||
        !aligned(p->out, 16))
        return QZ_ERR_ALIGNMENT;
    if (!aligned(p->dz_amax, 4) || !aligned(p->x_amax, 4) || !aligned(p->d_offsets, 4) || !aligned(p->d_counts, 4))
        return QZ_ERR_ALIGNMENT;
    return from_cuda(qz::launch_weight_grad(*p, one_per_sm(opts), (cudaStream_t)stream, err_word(opts)));
}

size_t qz_activation_grad_bytes(int64_t slots, int64_t n, int gated, int n_experts) {
    if (slots < 0 || slots > kMaxIndex || n < 8 || n % 8 != 0 || n > QZ_MAX_LD || n_experts < 1 ||
        n_experts > QZ_MAX_ROUTE_EXPERTS)
        return 0;
    return qz::act_grad_bytes(slots, n, gated != 0, n_experts);
}

qz_status qz_expert_activation_grad(const void* d_dout, int64_t ld_dout, const void* d_pre, int64_t ld_pre,
                                    int64_t slots, int64_t n, int activation, int gated, const int32_t* d_offsets,
                                    const int32_t* d_counts, int n_experts, void* d_dpre, int64_t ld_dpre,
                                    float* d_dbias, void* stream, const qz_launch_opts* opts) {
    const int64_t width = gated ? 2 * n : n;
    if (!valid_activation(activation) || n_experts < 1 || n_experts > QZ_MAX_ROUTE_EXPERTS) return QZ_ERR_INVALID_ARG;
    if (slots < 0 || slots > kMaxIndex || n < 8 || n % 8 != 0 || n > QZ_MAX_LD) return QZ_ERR_INVALID_ARG;
    if (!valid_ld(ld_dout, n) || !valid_ld(ld_pre, width) || !valid_ld(ld_dpre, width)) return QZ_ERR_INVALID_ARG;
    if (!d_offsets || !d_counts || (slots > 0 && (!d_dout || !d_pre || !d_dpre))) return QZ_ERR_INVALID_ARG;
    if (!aligned(d_dout, 16) || !aligned(d_pre, 16) || !aligned(d_dpre, 16) || !aligned(d_dbias, 4) ||
        !aligned(d_offsets, 4) || !aligned(d_counts, 4))
        return QZ_ERR_ALIGNMENT;
    void* const ws = opts ? opts->d_workspace : nullptr;
    if (d_dbias && (!ws || opts->workspace_bytes < qz::act_grad_bytes(slots, n, gated != 0, n_experts)))
        return QZ_ERR_INVALID_ARG;
    if (!aligned(ws, 16)) return QZ_ERR_ALIGNMENT;
    return from_cuda(qz::launch_act_grad(static_cast<const uint16_t*>(d_dout), ld_dout,
                                         static_cast<const uint16_t*>(d_pre), ld_pre, slots, n, activation, gated != 0,
                                         d_offsets, d_counts, n_experts, static_cast<uint16_t*>(d_dpre), ld_dpre,
                                         d_dbias, static_cast<float*>(ws), device_sms(), (cudaStream_t)stream,
                                         err_word(opts)));
}

qz_status qz_dispatch_experts(const void* d_x, int64_t ld_x, const int32_t* d_slots, const int32_t* d_rows, int64_t T,
                              int top_k, int64_t slots, int64_t H, const float* d_weights, void* d_y, int64_t ld_y,
                              const void* d_other, int64_t ld_other, float* d_dots, void* stream) {
    qz_status st = check_rows(d_x, d_y, d_slots, T, top_k, slots, H);
    if (st != QZ_OK) return st;
    if (!valid_ld(ld_x, H) || !valid_ld(ld_y, H) || (d_other && !valid_ld(ld_other, H))) return QZ_ERR_INVALID_ARG;
    if ((d_other != nullptr) != (d_dots != nullptr) || (slots > 0 && !d_rows)) return QZ_ERR_INVALID_ARG;
    if (!aligned(d_x, 16) || !aligned(d_y, 16) || !aligned(d_other, 16) || !aligned(d_slots, 4) ||
        !aligned(d_rows, 4) || !aligned(d_weights, 4) || !aligned(d_dots, 4))
        return QZ_ERR_ALIGNMENT;
    if (T == 0 && slots == 0) return QZ_OK;
    return from_cuda(qz::launch_dispatch(static_cast<const uint16_t*>(d_x), ld_x, d_slots, d_rows, T, top_k, slots, H,
                                         d_weights, static_cast<uint16_t*>(d_y), ld_y,
                                         static_cast<const uint16_t*>(d_other), ld_other, d_dots,
                                         (cudaStream_t)stream));
}

qz_status qz_combine_experts(const void* d_y, int64_t ld_y, const int32_t* d_slots, int64_t T, int top_k,
                             int64_t slots, int64_t H, const float* d_weights, const void* d_residual,
                             int64_t ld_residual, void* d_out, int64_t ld_out, void* stream) {
    qz_status st = check_rows(d_out, d_y, d_slots, T, top_k, slots, H);
    if (st != QZ_OK) return st;
    if (!valid_ld(ld_y, H) || !valid_ld(ld_out, H) || (d_residual && !valid_ld(ld_residual, H)))
        return QZ_ERR_INVALID_ARG;
    if (!aligned(d_y, 16) || !aligned(d_out, 16) || !aligned(d_residual, 16) || !aligned(d_slots, 4) ||
        !aligned(d_weights, 4))
        return QZ_ERR_ALIGNMENT;
    if (T == 0) return QZ_OK;
    return from_cuda(qz::launch_combine(static_cast<const uint16_t*>(d_y), ld_y, d_slots, T, top_k, slots, H,
                                        d_weights, static_cast<const uint16_t*>(d_residual), ld_residual,
                                        static_cast<uint16_t*>(d_out), ld_out, (cudaStream_t)stream));
}

size_t qz_workspace_bytes(int n_experts) {
    if (n_experts < 1 || n_experts > QZ_MAX_EXPERTS) return 0;
    return qz::workspace_bytes(n_experts);
}

const char* qz_status_string(qz_status status) {
    switch (status) {
        case QZ_OK: return "QZ_OK";
        case QZ_ERR_INVALID_ARG: return "QZ_ERR_INVALID_ARG: invalid argument";
        case QZ_ERR_ALIGNMENT: return "QZ_ERR_ALIGNMENT: misaligned pointer or stride";
        case QZ_ERR_UNSUPPORTED: return "QZ_ERR_UNSUPPORTED: unsupported shape/format/layout combination";
        case QZ_ERR_CUDA: return "QZ_ERR_CUDA: CUDA launch error";
    }
    return "unknown qz_status";
}

int qz_version(void) { return 100; }

}  // extern "C"
