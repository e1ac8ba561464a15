// api.hip -- the extern "C" entry points of include/convmi.h: argument checking, kernel
// selection and launch.  No allocation, no synchronisation: every kernel goes on the
// caller's stream.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <string>

#include "../../include/convmi.h"
#include "internal.hpp"

using namespace convmi;

namespace {

thread_local std::string g_last_error;

convmi_status fail(convmi_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

convmi_status hip_fail(hipError_t e, const char* where) {
    return fail(CONVMI_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

constexpr int64_t kI32Max = 2147483647LL;
// pad_plan: one product's work from which channels are padded.  Both sides measured, whole call:
// 4.5 MFLOP bf16 26 us direct, 29 padded; 7.3: 30, 31; 7.8 fp32 108, 41; 19 bf16 79, 28; 54: 219,
// 31.  One limit for both types, between their break-even points: bf16 loses a microsecond
// just above it, fp32 would lose more below a higher one.
constexpr double kPadFlops = 6e6;

int64_t out_extent(int64_t in, int64_t k, int64_t s, int64_t p) {
    int64_t span = in + 2 * p - k;
    return span < 0 ? 0 : span / s + 1;
}

// Validate a descriptor; fills kernel dims.  `need_bn_params` checks momentum/eps.
convmi_status check_desc(const convmi_desc* d, ConvDims* out) {
    if (!d) return fail(CONVMI_ERR_INVALID_ARG, "desc is NULL");
    if (d->N < 1 || d->H < 1 || d->W < 1 || d->IC < 1 || d->OC < 1 || d->KH < 1 || d->KW < 1)
        return fail(CONVMI_ERR_INVALID_ARG, "sizes must be >= 1 (N=%lld H=%lld W=%lld IC=%lld OC=%lld KH=%lld KW=%lld)",
                    (long long)d->N, (long long)d->H, (long long)d->W, (long long)d->IC, (long long)d->OC,
                    (long long)d->KH, (long long)d->KW);
    if (d->stride_h < 1 || d->stride_w < 1) return fail(CONVMI_ERR_INVALID_ARG, "strides must be >= 1");
    if (d->pad_h < 0 || d->pad_w < 0) return fail(CONVMI_ERR_INVALID_ARG, "padding must be >= 0");
    if (d->dtype != CONVMI_F32 && d->dtype != CONVMI_BF16)
        return fail(CONVMI_ERR_INVALID_ARG, "unknown dtype %d", d->dtype);
    if (d->activation < CONVMI_ACT_IDENTITY || d->activation > CONVMI_ACT_GELU)
        return fail(CONVMI_ERR_INVALID_ARG, "unknown activation %d", d->activation);
    if (d->normalization < CONVMI_NORM_NONE || d->normalization > CONVMI_NORM_GROUP)
        return fail(CONVMI_ERR_INVALID_ARG, "unknown normalization %d", d->normalization);
    if (d->mode != CONVMI_MODE_TRAIN && d->mode != CONVMI_MODE_EVAL)
        return fail(CONVMI_ERR_INVALID_ARG, "unknown mode %d", d->mode);
    if (d->normalization == CONVMI_NORM_BATCH && !(d->momentum >= 0.0f && d->momentum <= 1.0f))
        return fail(CONVMI_ERR_INVALID_ARG, "momentum must be in [0, 1]");
    if (d->normalization != CONVMI_NORM_NONE && !(d->eps > 0.0f))
        return fail(CONVMI_ERR_INVALID_ARG, "eps must be > 0");
    if (d->normalization == CONVMI_NORM_GROUP && (d->groups < 1 || d->OC % d->groups != 0))
        return fail(CONVMI_ERR_INVALID_ARG, "groups (%d) must be >= 1 and divide OC (%lld)", d->groups,
                    (long long)d->OC);
    const int64_t OH = out_extent(d->H, d->KH, d->stride_h, d->pad_h);
    const int64_t OW = out_extent(d->W, d->KW, d->stride_w, d->pad_w);
    if (OH < 1 || OW < 1)
        return fail(CONVMI_ERR_INVALID_ARG, "kernel %lldx%lld does not fit the padded %lldx%lld input",
                    (long long)d->KH, (long long)d->KW, (long long)d->H, (long long)d->W);
    // Index arithmetic inside the kernels is int32 per image and for N*OH*OW rows.
    if (d->H * d->W * d->IC > kI32Max || OH * OW * d->OC > kI32Max || d->N * OH * OW > kI32Max ||
        d->N * d->H * d->W > kI32Max || d->OC * d->KH * d->KW * d->IC > kI32Max ||
        d->stride_h > 65535 || d->stride_w > 65535 || d->pad_h > 65535 || d->pad_w > 65535 ||
        d->H > kI32Max / 4 || d->W > kI32Max / 4)
        return fail(CONVMI_ERR_UNSUPPORTED, "problem exceeds the int32 index limits of the kernels");
    if (out) {
        *out = ConvDims{(int)d->N, (int)d->H, (int)d->W, (int)d->IC, (int)d->OC, (int)d->KH, (int)d->KW,
                        d->stride_h, d->stride_w, d->pad_h, d->pad_w, (int)OH, (int)OW};
    }
    return CONVMI_OK;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

convmi_status need(const void* p, const char* name) {
    if (!p) return fail(CONVMI_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, 16)) return fail(CONVMI_ERR_MISALIGNED, "%s is not 16-byte aligned", name);
    return CONVMI_OK;
}

convmi_status need_vec(const float* p, const char* name) {
    if (!p) return fail(CONVMI_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, 4)) return fail(CONVMI_ERR_MISALIGNED, "%s is not 4-byte aligned", name);
    return CONVMI_OK;
}

convmi_status check_ws(void* ws, size_t have, size_t want, const char* op) {
    if (want == 0) return CONVMI_OK;
    if (have < want || !ws)
        return fail(CONVMI_ERR_WORKSPACE, "%s needs %zu workspace bytes, got %zu%s", op, want, have,
                    ws ? "" : " (NULL)");
    if (!aligned(ws, 256)) return fail(CONVMI_ERR_MISALIGNED, "workspace is not 256-byte aligned");
    return CONVMI_OK;
}

#define CHECK(expr)                        \
    do {                                   \
        convmi_status _st = (expr);        \
        if (_st != CONVMI_OK) return _st;  \
    } while (0)

int64_t rows_of(const ConvDims& d) { return (int64_t)d.N * d.OH * d.OW; }

// Layer norm and group norm: per-sample statistics over channel groups.
bool per_sample_norm(const convmi_desc* desc) {
    return desc->normalization == CONVMI_NORM_LAYER || desc->normalization == CONVMI_NORM_GROUP;
}
int norm_groups(const convmi_desc* desc) { return desc->normalization == CONVMI_NORM_GROUP ? desc->groups : 1; }

// Per-tile batch-norm statistics of the fused training forward, after its weight copy.
size_t stats_offset(const convmi_desc* desc, const ConvDims& d) { return halo_fwd_ws_bytes(desc->dtype, d); }
size_t stats_bytes(const convmi_desc* desc, const ConvDims& d) {
    return align_up((size_t)halo_fwd_stat_tiles(desc->dtype, d) * 4 * d.OC * sizeof(float), 256);
}

size_t ws_forward(const convmi_desc* desc, const ConvDims& d) {
    size_t a = igemm_fwd_supported(desc->dtype, d) ? igemm_fwd_ws_bytes(desc->dtype, d) : 0;
    size_t b = 0;
    if (desc->normalization != CONVMI_NORM_NONE) {
        b = per_sample_norm(desc) ? grp_stats_ws_bytes(d.N, (int64_t)d.OH * d.OW, d.OC, desc->dtype)
                                  : bn_stats_ws_bytes(rows_of(d), d.OC, desc->dtype);
        if (halo_fwd_supported(desc->dtype, d)) {
            const size_t c = stats_offset(desc, d) + stats_bytes(desc, d);
            if (c > b) b = c;
        }
    }
    return a > b ? a : b;
}
size_t ws_backward_data(const convmi_desc* desc, const ConvDims& d) {
    return igemm_dx_supported(desc->dtype, d) ? igemm_dx_ws_bytes(desc->dtype, d) : 0;
}
size_t ws_backward_weight(const convmi_desc* desc, const ConvDims& d) {
    return igemm_dw_supported(desc->dtype, d) ? igemm_dw_ws_bytes(desc->dtype, d) : 0;
}
size_t ws_bn_stats(const convmi_desc* desc, const ConvDims& d) {
    if (per_sample_norm(desc)) return grp_stats_ws_bytes(d.N, (int64_t)d.OH * d.OW, d.OC, desc->dtype);
    return bn_stats_ws_bytes(rows_of(d), d.OC, desc->dtype);
}
size_t ws_act_bwd(const convmi_desc* desc, const ConvDims& d) {
    if (per_sample_norm(desc))
        return grp_bwd_ws_bytes(d.N, (int64_t)d.OH * d.OW, d.OC, norm_groups(desc), desc->dtype);
    return desc->normalization == CONVMI_NORM_BATCH ? bn_bwd_ws_bytes(rows_of(d), d.OC, desc->dtype) : 0;
}

// backward_full: dz (unless the activation is the identity), then the weight-gradient
// workspace, then the input-gradient one (the two products run concurrently, so they
// cannot share bytes).
size_t dz_bytes_full(const convmi_desc* desc, const ConvDims& d) {
    return desc->activation == CONVMI_ACT_IDENTITY ? 0
                                                   : align_up((size_t)rows_of(d) * d.OC * dtype_size(desc->dtype), 256);
}
size_t ws_backward_full(const convmi_desc* desc, const ConvDims& d) {
    return dz_bytes_full(desc, d) + align_up(ws_backward_weight(desc, d), 256) + ws_backward_data(desc, d);
}
// With x or the saved tensor kept in 8 bits: x unpacked behind the rest.  Layers whose
// channel counts the tiled products do not take would run the direct kernels; since x is
// copied anyway, one with enough work for it is computed on channels padded to counts
// that they take (x, dz and w in, dx, dw and db out).
struct PadPlan {
    bool on;
    ConvDims d;  // padded channels
    size_t x, dz, w, dx, dw, db, ws_dw, ws_dx, total;  // offsets behind the compact dz
};
PadPlan pad_plan(const convmi_desc* desc, const ConvDims& d) {
    PadPlan p{};
    const int vec = desc->dtype == CONVMI_BF16 ? 8 : 4;
    auto tiled = [&](const ConvDims& c) {
        return igemm_dx_supported(desc->dtype, c) && igemm_dw_supported(desc->dtype, c);
    };
    if (2.0 * rows_of(d) * d.OC * d.KH * d.KW * d.IC < kPadFlops || tiled(d)) return p;
    if (d.IC > (1 << 24) || d.OC > (1 << 24)) return p;  // 32-bit row lengths in bytes
    int64_t nw = 0;
    for (int m = vec; !p.on; m *= 2) {
        if (m > 8 * vec) return p;
        p.d = d;
        p.d.IC = (int)(ceil_div(d.IC, m) * m);
        p.d.OC = (int)(ceil_div(d.OC, m) * m);
        nw = (int64_t)p.d.OC * d.KH * d.KW * p.d.IC;
        if ((int64_t)d.H * d.W * p.d.IC > kI32Max || (int64_t)d.OH * d.OW * p.d.OC > kI32Max || nw > kI32Max) return p;
        p.on = tiled(p.d);
    }
    const int64_t xr = (int64_t)d.N * d.H * d.W;
    const size_t es = dtype_size(desc->dtype);
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t o = at; at = align_up(at + bytes, 256); return o; };
    p.x = take((size_t)xr * p.d.IC * es);
    p.dz = take((size_t)rows_of(d) * p.d.OC * es);
    p.w = take((size_t)nw * es);
    p.dx = take((size_t)xr * p.d.IC * es);
    p.dw = take((size_t)nw * 4);
    p.db = take((size_t)p.d.OC * 4);
    p.ws_dw = take(igemm_dw_ws_bytes(desc->dtype, p.d));
    p.ws_dx = take(igemm_dx_ws_bytes(desc->dtype, p.d));
    p.total = at;
    return p;
}
size_t ws_backward_full_mx8(const convmi_desc* desc, const ConvDims& d) {
    const PadPlan p = pad_plan(desc, d);
    const size_t full = align_up(ws_backward_full(desc, d), 256);
    if (p.on) {
        // without scales the call runs on the layer's own channels, whose dW may split further
        const size_t padded = dz_bytes_full(desc, d) + p.total;
        return padded > full ? padded : full;
    }
    return full + align_up((size_t)d.N * d.H * d.W * d.IC * dtype_size(desc->dtype), 256);
}

bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
    if (!a || !b) return false;
    uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + bn && b0 < a0 + an;
}

}  // namespace

#define CONVMI_API __attribute__((visibility("default")))

extern "C" {

CONVMI_API const char* convmi_last_error(void) { return g_last_error.c_str(); }

CONVMI_API const char* convmi_version(void) { return "convmi 0.1 (gfx950)"; }

CONVMI_API convmi_status convmi_output_dims(const convmi_desc* desc, int64_t* OH, int64_t* OW) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    if (!OH || !OW) return fail(CONVMI_ERR_INVALID_ARG, "OH/OW out-pointers are NULL");
    *OH = d.OH;
    *OW = d.OW;
    return CONVMI_OK;
}

CONVMI_API convmi_status convmi_workspace_size(const convmi_desc* desc, int32_t op, size_t* bytes) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    if (!bytes) return fail(CONVMI_ERR_INVALID_ARG, "bytes out-pointer is NULL");
    switch (op) {
    case CONVMI_OP_FORWARD: *bytes = ws_forward(desc, d); break;
    case CONVMI_OP_BACKWARD_DATA: *bytes = ws_backward_data(desc, d); break;
    case CONVMI_OP_BACKWARD_WEIGHT: *bytes = ws_backward_weight(desc, d); break;
    case CONVMI_OP_BN_STATS: *bytes = ws_bn_stats(desc, d); break;
    case CONVMI_OP_ACTIVATION_BACKWARD: *bytes = ws_act_bwd(desc, d); break;
    case CONVMI_OP_BACKWARD_FULL: *bytes = ws_backward_full(desc, d); break;
    case CONVMI_OP_BACKWARD_FULL_MX8: *bytes = ws_backward_full_mx8(desc, d); break;
    default: return fail(CONVMI_ERR_INVALID_ARG, "unknown op %d", op);
    }
    return CONVMI_OK;
}

CONVMI_API convmi_status convmi_plan_name(const convmi_desc* desc, int32_t op, char* buf, size_t len) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    if (!buf || len == 0) return fail(CONVMI_ERR_INVALID_ARG, "buf is NULL or len is 0");
    const int dt = desc->dtype;
    if (op == CONVMI_OP_FORWARD) {
        if (!halo_plan_text(dt, d, true, buf, len))
            snprintf(buf, len, "%s", igemm_fwd_supported(dt, d) ? "implicit gemm" : "direct");
    } else if (op == CONVMI_OP_BACKWARD_DATA) {
        if (!igemm_dx_supported(dt, d))
            snprintf(buf, len, "direct");
        else if (!halo_plan_text(dt, d, false, buf, len))
            snprintf(buf, len, "implicit gemm");
    } else {
        return fail(CONVMI_ERR_INVALID_ARG, "plan names cover the forward and the input gradient, not op %d", op);
    }
    return CONVMI_OK;
}

}  // extern "C"

namespace {

// conv2d_forward after the descriptor check; shared by the allocation-free variant,
// which passes its static scratch array as the workspace.
convmi_status forward_impl(const convmi_desc* desc, const ConvDims& d, const void* x, const void* w,
                           const float* bias, const float* gamma, const float* beta, float* running_mean,
                           float* running_var, float* save_mean, float* save_inv_std, void* z, void* y,
                           void* workspace, size_t workspace_bytes, void* stream) {
    CHECK(need(x, "x"));
    CHECK(need(w, "w"));
    CHECK(need(y, "y"));
    if (bias) CHECK(need_vec(bias, "bias"));
    const bool bn = desc->normalization == CONVMI_NORM_BATCH;
    const bool psn = per_sample_norm(desc);
    const size_t es = dtype_size(desc->dtype);
    const size_t ybytes = (size_t)rows_of(d) * d.OC * es;
    if (bn) {
        CHECK(need(z, "z (required with batch norm)"));
        CHECK(need_vec(gamma, "gamma"));
        CHECK(need_vec(beta, "beta"));
        CHECK(need_vec(save_mean, "save_mean"));
        CHECK(need_vec(save_inv_std, "save_inv_std"));
        if ((running_mean == nullptr) != (running_var == nullptr))
            return fail(CONVMI_ERR_INVALID_ARG, "running_mean and running_var must be both given or both NULL");
        if (desc->mode == CONVMI_MODE_EVAL && running_mean == nullptr)
            return fail(CONVMI_ERR_INVALID_ARG, "evaluation mode normalises with running_mean/running_var: both required");
        if (running_mean) {
            CHECK(need_vec(running_mean, "running_mean"));
            CHECK(need_vec(running_var, "running_var"));
        }
    } else if (psn) {
        CHECK(need(z, "z (required with layer / group norm)"));
        CHECK(need_vec(gamma, "gamma"));
        CHECK(need_vec(beta, "beta"));
        CHECK(need_vec(save_mean, "save_mean"));
        CHECK(need_vec(save_inv_std, "save_inv_std"));
        if (running_mean || running_var)
            return fail(CONVMI_ERR_INVALID_ARG, "layer / group norm keep no running statistics: pass NULL");
    } else if (z) {
        CHECK(need(z, "z"));
    }
    if (z && z == y) return fail(CONVMI_ERR_INVALID_ARG, "z and y must be distinct buffers");
    if (overlaps(y, ybytes, x, (size_t)d.N * d.H * d.W * d.IC * es) || overlaps(z, ybytes, x, (size_t)d.N * d.H * d.W * d.IC * es))
        return fail(CONVMI_ERR_INVALID_ARG, "outputs overlap x");
    CHECK(check_ws(workspace, workspace_bytes, ws_forward(desc, d), "conv2d_forward"));
    hipStream_t s = (hipStream_t)stream;
    const int act = desc->activation;
    hipError_t e;
    // Layer / group norm: z (with per-tile statistics from the stride-1 epilogue when that
    // path runs), the per-sample group statistics, then normalise + activate.
    if (psn) {
        const int G = norm_groups(desc);
        const int64_t S = (int64_t)d.OH * d.OW;
        if (halo_fwd_supported(desc->dtype, d)) {
            float* part = (float*)((char*)workspace + stats_offset(desc, d));
            e = launch_halo_fwd(desc->dtype, x, w, bias, z, nullptr, d, act, workspace, s, nullptr, part);
            if (e != hipSuccess) return hip_fail(e, "conv2d_forward: convolution launch");
            e = launch_grp_tiles_finalize(part, halo_fwd_stat_tiles(desc->dtype, d), d.N, d.OC, G, S, desc->eps,
                                          save_mean, save_inv_std, s);
        } else {
            e = igemm_fwd_supported(desc->dtype, d)
                    ? launch_igemm_fwd(desc->dtype, x, w, bias, z, nullptr, d, act, workspace, s)
                    : launch_conv_fwd_direct(desc->dtype, x, w, bias, z, nullptr, d, act, s);
            if (e != hipSuccess) return hip_fail(e, "conv2d_forward: convolution launch");
            e = launch_grp_stats(desc->dtype, z, d.N, S, d.OC, G, desc->eps, save_mean, save_inv_std, workspace, s);
        }
        if (e != hipSuccess) return hip_fail(e, "conv2d_forward: normalisation statistics launch");
        e = launch_grp_apply(desc->dtype, z, y, d.N, S, d.OC, G, act, gamma, beta, save_mean, save_inv_std, s);
        if (e != hipSuccess) return hip_fail(e, "conv2d_forward: normalise/activate launch");
        return CONVMI_OK;
    }
    // Without batch norm the activation is fused into the convolution's epilogue; so is
    // evaluation-mode batch norm on the input-tile-reuse path (its statistics are known
    // before the convolution runs).
    if (bn && desc->mode == CONVMI_MODE_EVAL && halo_fwd_supported(desc->dtype, d)) {
        e = launch_bn_eval_stats(running_mean, running_var, d.OC, desc->eps, save_mean, save_inv_std, s);
        if (e != hipSuccess) return hip_fail(e, "conv2d_forward: batch-norm statistics launch");
        const float* bn_eval[4] = {save_mean, save_inv_std, gamma, beta};
        e = launch_halo_fwd(desc->dtype, x, w, bias, z, y, d, act, workspace, s, bn_eval);
        if (e != hipSuccess) return hip_fail(e, "conv2d_forward: convolution launch");
        return CONVMI_OK;
    }
    // Training-mode batch norm on the input-tile-reuse path: the convolution's epilogue
    // also reduces per-tile statistics of the stored z, so z is not read again for them.
    if (bn && desc->mode == CONVMI_MODE_TRAIN && halo_fwd_supported(desc->dtype, d)) {
        float* part = (float*)((char*)workspace + stats_offset(desc, d));
        e = launch_halo_fwd(desc->dtype, x, w, bias, z, nullptr, d, act, workspace, s, nullptr, part);
        if (e != hipSuccess) return hip_fail(e, "conv2d_forward: convolution launch");
        e = launch_bn_tiles_finalize(part, halo_fwd_stat_tiles(desc->dtype, d), (int)d.OC, rows_of(d),
                                     desc->momentum, desc->eps, save_mean, save_inv_std, running_mean, running_var, s);
        if (e != hipSuccess) return hip_fail(e, "conv2d_forward: batch-norm statistics launch");
        e = launch_apply_act(desc->dtype, z, y, rows_of(d), d.OC, act, 1, gamma, beta, save_mean, save_inv_std, s);
        if (e != hipSuccess) return hip_fail(e, "conv2d_forward: normalise/activate launch");
        return CONVMI_OK;
    }
    void* conv_y = bn ? nullptr : y;
    if (igemm_fwd_supported(desc->dtype, d))
        e = launch_igemm_fwd(desc->dtype, x, w, bias, z, conv_y, d, act, workspace, s);
    else
        e = launch_conv_fwd_direct(desc->dtype, x, w, bias, z, conv_y, d, act, s);
    if (e != hipSuccess) return hip_fail(e, "conv2d_forward: convolution launch");
    if (bn) {
        if (desc->mode == CONVMI_MODE_EVAL)  // running statistics, left unchanged
            e = launch_bn_eval_stats(running_mean, running_var, d.OC, desc->eps, save_mean, save_inv_std, s);
        else
            e = launch_bn_stats(desc->dtype, z, rows_of(d), d.OC, desc->momentum, desc->eps, save_mean,
                                save_inv_std, running_mean, running_var, workspace, s);
        if (e != hipSuccess) return hip_fail(e, "conv2d_forward: batch-norm statistics launch");
        e = launch_apply_act(desc->dtype, z, y, rows_of(d), d.OC, act, 1, gamma, beta, save_mean, save_inv_std, s);
        if (e != hipSuccess) return hip_fail(e, "conv2d_forward: normalise/activate launch");
    }
    return CONVMI_OK;
}

// Scratch for conv2d_forward_noalloc: one copy per GPU, held until the process ends.
// Host code never passes `scratch` itself to a kernel (in host code the name is a
// host-side stand-in): it uses the device address hipGetSymbolAddress returns, looked
// up once per device.
constexpr size_t kScratchBytes = CONVMI_NOALLOC_SCRATCH_BYTES;
__device__ __align__(256) unsigned char scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

// Device address of this device's `scratch`, resolved on the first call made with the
// device current.
convmi_status scratch_for_current_device(void** out) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "conv2d_forward_noalloc: hipGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(CONVMI_ERR_UNSUPPORTED, "device %d beyond %d", dev, kMaxDevices);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return hip_fail(e, "conv2d_forward_noalloc: hipGetSymbolAddress(scratch)");
        if (!p || !aligned(p, 256)) return fail(CONVMI_ERR_HIP, "scratch array has no usable device address");
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return CONVMI_OK;
}

// A second stream per device for conv2d_backward_full: the weight gradient runs there
// while the input gradient runs on the caller's stream, forked and joined with events
// (default priority, non-blocking; created on the device's first such call and kept
// until the process ends).  The mutex covers the whole fork-join enqueue, so the shared
// events are never recorded by two calls at once.
struct SideStream {
    hipStream_t s = nullptr;
    hipEvent_t fork = nullptr, join = nullptr;
    std::mutex mu;
};
std::mutex g_side_mu;
SideStream g_side[kMaxDevices];

convmi_status side_stream_for_current_device(SideStream** out) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "conv2d_backward_full: hipGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(CONVMI_ERR_UNSUPPORTED, "device %d beyond %d", dev, kMaxDevices);
    std::lock_guard<std::mutex> lock(g_side_mu);
    SideStream& ss = g_side[dev];
    if (!ss.join) {
        if (!ss.s && (e = hipStreamCreateWithFlags(&ss.s, hipStreamNonBlocking)) != hipSuccess)
            return hip_fail(e, "conv2d_backward_full: creating the weight-gradient stream");
        if (!ss.fork && (e = hipEventCreateWithFlags(&ss.fork, hipEventDisableTiming)) != hipSuccess)
            return hip_fail(e, "conv2d_backward_full: creating an event");
        if ((e = hipEventCreateWithFlags(&ss.join, hipEventDisableTiming)) != hipSuccess)
            return hip_fail(e, "conv2d_backward_full: creating an event");
    }
    *out = &ss;
    return CONVMI_OK;
}

}  // namespace

extern "C" {

CONVMI_API convmi_status conv2d_forward(const convmi_desc* desc, const void* x, const void* w, const float* bias,
                             const float* gamma, const float* beta, float* running_mean, float* running_var,
                             float* save_mean, float* save_inv_std, void* z, void* y,
                             void* workspace, size_t workspace_bytes, void* stream) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    return forward_impl(desc, d, x, w, bias, gamma, beta, running_mean, running_var, save_mean, save_inv_std, z, y,
                        workspace, workspace_bytes, stream);
}

CONVMI_API convmi_status conv2d_forward_noalloc(const convmi_desc* desc, const void* x, const void* w,
                                                const float* bias, const float* gamma, const float* beta,
                                                float* running_mean, float* running_var, float* save_mean,
                                                float* save_inv_std, void* z, void* y, void* stream) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    const size_t want = ws_forward(desc, d);
    if (want > kScratchBytes)
        return fail(CONVMI_ERR_WORKSPACE,
                    "conv2d_forward_noalloc: this layer needs %zu bytes of scratch, above the static limit of %zu; "
                    "use conv2d_forward with a caller-owned workspace",
                    want, kScratchBytes);
    void* ws = nullptr;
    if (want > 0) CHECK(scratch_for_current_device(&ws));
    return forward_impl(desc, d, x, w, bias, gamma, beta, running_mean, running_var, save_mean, save_inv_std, z, y,
                        ws, want, stream);
}

CONVMI_API convmi_status conv2d_backward_data(const convmi_desc* desc, const void* dz, const void* w, void* dx,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    CHECK(need(dz, "dz"));
    CHECK(need(w, "w"));
    CHECK(need(dx, "dx"));
    const size_t es = dtype_size(desc->dtype);
    const size_t dxb = (size_t)d.N * d.H * d.W * d.IC * es;
    if (overlaps(dx, dxb, dz, (size_t)rows_of(d) * d.OC * es) || overlaps(dx, dxb, w, (size_t)d.OC * d.KH * d.KW * d.IC * es))
        return fail(CONVMI_ERR_INVALID_ARG, "dx overlaps an input");
    CHECK(check_ws(workspace, workspace_bytes, ws_backward_data(desc, d), "conv2d_backward_data"));
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = igemm_dx_supported(desc->dtype, d)
                       ? launch_igemm_dx(desc->dtype, dz, w, dx, d, workspace, s)
                       : launch_conv_dx_direct(desc->dtype, dz, w, dx, d, s);
    if (e != hipSuccess) return hip_fail(e, "conv2d_backward_data launch");
    return CONVMI_OK;
}

CONVMI_API convmi_status conv2d_backward_weight(const convmi_desc* desc, const void* x, const void* dz, float* dw,
                                     float* db, int32_t accumulate, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    CHECK(need(x, "x"));
    CHECK(need(dz, "dz"));
    CHECK(need(dw, "dw"));
    if (db) CHECK(need_vec(db, "db"));
    if (accumulate != 0 && accumulate != 1) return fail(CONVMI_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    CHECK(check_ws(workspace, workspace_bytes, ws_backward_weight(desc, d), "conv2d_backward_weight"));
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = igemm_dw_supported(desc->dtype, d)
                       ? launch_igemm_dw(desc->dtype, x, dz, dw, db, accumulate, d, workspace, s)
                       : launch_conv_dw_direct(desc->dtype, x, dz, dw, db, accumulate, d, s);
    if (e != hipSuccess) return hip_fail(e, "conv2d_backward_weight launch");
    return CONVMI_OK;
}

CONVMI_API convmi_status bn_stats_training(const convmi_desc* desc, const void* z, float* save_mean, float* save_inv_std,
                                float* running_mean, float* running_var,
                                void* workspace, size_t workspace_bytes, void* stream) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    if (desc->normalization == CONVMI_NORM_NONE)
        return fail(CONVMI_ERR_INVALID_ARG, "bn_stats_training needs a normalization");
    if (per_sample_norm(desc)) {
        CHECK(need(z, "z"));
        CHECK(need_vec(save_mean, "save_mean"));
        CHECK(need_vec(save_inv_std, "save_inv_std"));
        if (running_mean || running_var)
            return fail(CONVMI_ERR_INVALID_ARG, "layer / group norm keep no running statistics: pass NULL");
        CHECK(check_ws(workspace, workspace_bytes, ws_bn_stats(desc, d), "bn_stats_training"));
        hipError_t e = launch_grp_stats(desc->dtype, z, d.N, (int64_t)d.OH * d.OW, d.OC, norm_groups(desc), desc->eps,
                                        save_mean, save_inv_std, workspace, (hipStream_t)stream);
        if (e != hipSuccess) return hip_fail(e, "bn_stats_training launch");
        return CONVMI_OK;
    }
    if (desc->mode != CONVMI_MODE_TRAIN)
        return fail(CONVMI_ERR_INVALID_ARG,
                    "bn_stats_training computes training statistics; in evaluation mode conv2d_forward uses the "
                    "running statistics");
    CHECK(need(z, "z"));
    CHECK(need_vec(save_mean, "save_mean"));
    CHECK(need_vec(save_inv_std, "save_inv_std"));
    if ((running_mean == nullptr) != (running_var == nullptr))
        return fail(CONVMI_ERR_INVALID_ARG, "running_mean and running_var must be both given or both NULL");
    if (running_mean) {
        CHECK(need_vec(running_mean, "running_mean"));
        CHECK(need_vec(running_var, "running_var"));
    }
    CHECK(check_ws(workspace, workspace_bytes, ws_bn_stats(desc, d), "bn_stats_training"));
    hipError_t e = launch_bn_stats(desc->dtype, z, rows_of(d), d.OC, desc->momentum, desc->eps, save_mean,
                                   save_inv_std, running_mean, running_var, workspace, (hipStream_t)stream);
    if (e != hipSuccess) return hip_fail(e, "bn_stats_training launch");
    return CONVMI_OK;
}

CONVMI_API convmi_status activation_backward(const convmi_desc* desc, const void* z, const void* dy,
                                  const float* gamma, const float* beta,
                                  const float* save_mean, const float* save_inv_std,
                                  void* dz, float* dgamma, float* dbeta, int32_t accumulate,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    CHECK(need(z, "z"));
    CHECK(need(dy, "dy"));
    CHECK(need(dz, "dz"));
    if (accumulate != 0 && accumulate != 1) return fail(CONVMI_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    const size_t bytes = (size_t)rows_of(d) * d.OC * dtype_size(desc->dtype);
    if (dz != dy && overlaps(dz, bytes, dy, bytes)) return fail(CONVMI_ERR_INVALID_ARG, "dz partially overlaps dy");
    if (overlaps(dz, bytes, z, bytes)) return fail(CONVMI_ERR_INVALID_ARG, "dz overlaps z");
    hipStream_t s = (hipStream_t)stream;
    hipError_t e;
    if (per_sample_norm(desc)) {
        CHECK(need_vec(gamma, "gamma"));
        CHECK(need_vec(beta, "beta"));
        CHECK(need_vec(save_mean, "save_mean"));
        CHECK(need_vec(save_inv_std, "save_inv_std"));
        if (dgamma) CHECK(need_vec(dgamma, "dgamma"));
        if (dbeta) CHECK(need_vec(dbeta, "dbeta"));
        CHECK(check_ws(workspace, workspace_bytes, ws_act_bwd(desc, d), "activation_backward"));
        e = launch_grp_bwd(desc->dtype, z, dy, dz, d.N, (int64_t)d.OH * d.OW, d.OC, norm_groups(desc),
                           desc->activation, gamma, beta, save_mean, save_inv_std, dgamma, dbeta, accumulate,
                           workspace, s);
    } else if (desc->normalization == CONVMI_NORM_BATCH) {
        CHECK(need_vec(gamma, "gamma"));
        CHECK(need_vec(beta, "beta"));
        CHECK(need_vec(save_mean, "save_mean"));
        CHECK(need_vec(save_inv_std, "save_inv_std"));
        if (dgamma) CHECK(need_vec(dgamma, "dgamma"));
        if (dbeta) CHECK(need_vec(dbeta, "dbeta"));
        CHECK(check_ws(workspace, workspace_bytes, ws_act_bwd(desc, d), "activation_backward"));
        e = launch_bn_bwd(desc->dtype, z, dy, dz, rows_of(d), d.OC, desc->activation, gamma, beta, save_mean,
                          save_inv_std, dgamma, dbeta, accumulate, desc->mode == CONVMI_MODE_EVAL ? 1 : 0,
                          workspace, s);
    } else {
        e = launch_act_bwd(desc->dtype, z, dy, dz, rows_of(d), d.OC, desc->activation, s);
    }
    if (e != hipSuccess) return hip_fail(e, "activation_backward launch");
    return CONVMI_OK;
}

}  // extern "C"

namespace {

int64_t mx8_blocks(int64_t cols) { return ceil_div(cols, 32); }

// conv2d_backward_full (both scale pointers NULL: dense tensors) and its variant with x
// and / or the saved tensor kept in 8 bits.
convmi_status backward_full_impl(const char* op, const convmi_desc* desc, const void* x, const void* x_scales,
                                 const void* w, const void* saved, const void* saved_scales, int32_t saved_is_output,
                                 const void* dy, void* dx, float* dw, float* db, int32_t accumulate, size_t want,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    if (desc->normalization != CONVMI_NORM_NONE)
        return fail(CONVMI_ERR_UNSUPPORTED,
                    "conv2d_backward_full takes unnormalised layers; with a normalisation call activation_backward, "
                    "then conv2d_backward_data and conv2d_backward_weight");
    if (saved_is_output != 0 && saved_is_output != 1)
        return fail(CONVMI_ERR_INVALID_ARG, "saved_is_output must be 0 or 1");
    if (saved_is_output && desc->activation == CONVMI_ACT_GELU)
        return fail(CONVMI_ERR_INVALID_ARG, "the GELU derivative is not a function of its output: pass z");
    CHECK(need(x, "x"));
    CHECK(need(w, "w"));
    CHECK(need(saved, saved_is_output ? "y" : "z"));
    CHECK(need(dy, "dy"));
    CHECK(need(dw, "dw"));
    if (dx) CHECK(need(dx, "dx"));
    if (db) CHECK(need_vec(db, "db"));
    if (accumulate != 0 && accumulate != 1) return fail(CONVMI_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    const size_t es = dtype_size(desc->dtype);
    const int64_t xrows = (int64_t)d.N * d.H * d.W;
    const size_t xb = (size_t)xrows * d.IC * es, yb = (size_t)rows_of(d) * d.OC * es;
    if (dx && (overlaps(dx, xb, x, x_scales ? xb / es : xb) || overlaps(dx, xb, dy, yb) ||
               overlaps(dx, xb, saved, saved_scales ? yb / es : yb) ||
               overlaps(dx, xb, w, (size_t)d.OC * d.KH * d.KW * d.IC * es)))
        return fail(CONVMI_ERR_INVALID_ARG, "dx overlaps an input");
    if (x_scales) {
        CHECK(need(x_scales, "x_scales"));
        if (dx && overlaps(dx, xb, x_scales, (size_t)xrows * mx8_blocks(d.IC)))
            return fail(CONVMI_ERR_INVALID_ARG, "dx overlaps an input");
    }
    if (saved_scales) {
        CHECK(need(saved_scales, "saved_scales"));
        if (dx && overlaps(dx, xb, saved_scales, (size_t)rows_of(d) * mx8_blocks(d.OC)))
            return fail(CONVMI_ERR_INVALID_ARG, "dx overlaps an input");
    }
    CHECK(check_ws(workspace, workspace_bytes, want, op));
    hipStream_t s = (hipStream_t)stream;
    hipError_t e = hipSuccess;
    const void* dz = dy;  // identity: act' = 1
    const size_t zb = dz_bytes_full(desc, d);
    const PadPlan pad = x_scales || saved_scales ? pad_plan(desc, d) : PadPlan{};
    if (x_scales && !pad.on) {
        void* xu = (char*)workspace + align_up(ws_backward_full(desc, d), 256);
        if ((e = launch_mx8_unpack(desc->dtype, x, x_scales, xrows, d.IC, xu, s)) != hipSuccess)
            return hip_fail(e, "conv2d_backward_full_mx8: unpack launch");
        x = xu;
    }
    if (zb) {
        dz = workspace;
        e = saved_scales ? launch_mx8_act_bwd(desc->dtype, saved, saved_scales, saved_is_output, dy, workspace,
                                              rows_of(d), d.OC, desc->activation, s)
            : saved_is_output
                ? launch_act_bwd_from_output(desc->dtype, saved, dy, workspace, rows_of(d), d.OC, desc->activation, s)
                : launch_act_bwd(desc->dtype, saved, dy, workspace, rows_of(d), d.OC, desc->activation, s);
        if (e != hipSuccess) return hip_fail(e, "conv2d_backward_full: activation backward launch");
    }
    void* ws_dw = (char*)workspace + zb;
    void* ws_dx = (char*)ws_dw + align_up(ws_backward_weight(desc, d), 256);
    Compact out{};
    if (pad.on) {  // from here on everything is the padded layer's
        char* at = (char*)workspace + zb;
        const int64_t taps = (int64_t)d.KH * d.KW;
        Prep in{};
        add_prep(in, x, x_scales, at + pad.x, xrows, x_scales ? d.IC : d.IC * es, (int)es, pad.d.IC * es);
        add_prep(in, dz, nullptr, at + pad.dz, rows_of(d), d.OC * es, (int)es, pad.d.OC * es);
        add_prep(in, w, nullptr, at + pad.w, d.OC * taps, d.IC * es, (int)es, pad.d.IC * es,
                 (pad.d.OC - d.OC) * taps);
        if ((e = launch_prep(in, desc->dtype, s)) != hipSuccess)
            return hip_fail(e, "conv2d_backward_full_mx8: padding launch");
        if (dx) out.seg[out.n++] = CompactSeg{at + pad.dx, dx, xrows, d.IC, pad.d.IC, desc->dtype, 0};
        out.seg[out.n++] = CompactSeg{at + pad.dw, dw, d.OC * taps, d.IC, pad.d.IC, CONVMI_F32, accumulate};
        if (db) out.seg[out.n++] = CompactSeg{at + pad.db, db, 1, d.OC, d.OC, CONVMI_F32, accumulate};
        x = at + pad.x;
        dz = at + pad.dz;
        w = at + pad.w;
        if (dx) dx = at + pad.dx;
        dw = (float*)(at + pad.dw);
        if (db) db = (float*)(at + pad.db);
        ws_dw = at + pad.ws_dw;
        ws_dx = at + pad.ws_dx;
        accumulate = 0;
        d = pad.d;
    }
    auto finish = [&]() {
        if (out.n && (e = launch_compact(out, s)) != hipSuccess)
            return hip_fail(e, "conv2d_backward_full_mx8: compaction launch");
        return CONVMI_OK;
    };
    auto weight_gradient = [&](hipStream_t st) {
        return igemm_dw_supported(desc->dtype, d) ? launch_igemm_dw(desc->dtype, x, dz, dw, db, accumulate, d, ws_dw, st)
                                                  : launch_conv_dw_direct(desc->dtype, x, dz, dw, db, accumulate, d, st);
    };
    auto input_gradient = [&](hipStream_t st) {
        return igemm_dx_supported(desc->dtype, d) ? launch_igemm_dx(desc->dtype, dz, w, dx, d, ws_dx, st)
                                                  : launch_conv_dx_direct(desc->dtype, dz, w, dx, d, st);
    };
    if (!dx || !dw_leaves_room(desc->dtype, d)) {
        if ((e = weight_gradient(s)) != hipSuccess) return hip_fail(e, "conv2d_backward_full: weight-gradient launch");
        if (dx && (e = input_gradient(s)) != hipSuccess)
            return hip_fail(e, "conv2d_backward_full: input-gradient launch");
        return finish();
    }
    // Fork: the weight gradient on the side stream, after everything before it on `s`
    // (dz included); the input gradient on `s`.  Join: `s` waits for the side stream, so
    // work the caller enqueues later sees both products.  Only where the weight-gradient
    // workgroups leave room on a CU do the two kernels fill each other's idle slots
    // (c5's backward 105 -> 91 us); elsewhere the fork and join cost more than they save.
    SideStream* side = nullptr;
    CHECK(side_stream_for_current_device(&side));
    std::lock_guard<std::mutex> lock(side->mu);
    if ((e = hipEventRecord(side->fork, s)) != hipSuccess) return hip_fail(e, "conv2d_backward_full: fork event");
    if ((e = hipStreamWaitEvent(side->s, side->fork, 0)) != hipSuccess)
        return hip_fail(e, "conv2d_backward_full: fork wait");
    const hipError_t ew = weight_gradient(side->s);
    // the join is enqueued even when a launch failed, so `s` never runs ahead of the side stream
    const hipError_t ex = input_gradient(s);
    if ((e = hipEventRecord(side->join, side->s)) != hipSuccess) return hip_fail(e, "conv2d_backward_full: join event");
    if ((e = hipStreamWaitEvent(s, side->join, 0)) != hipSuccess) return hip_fail(e, "conv2d_backward_full: join wait");
    if (ew != hipSuccess) return hip_fail(ew, "conv2d_backward_full: weight-gradient launch");
    if (ex != hipSuccess) return hip_fail(ex, "conv2d_backward_full: input-gradient launch");
    return finish();
}

// ---------------------------------------------------------------- linear layer, RMS norm, MX8
convmi_status check_dtype(int32_t dtype) {
    if (dtype != CONVMI_F32 && dtype != CONVMI_BF16) return fail(CONVMI_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    return CONVMI_OK;
}
convmi_status check_flag(int32_t v, const char* name) {
    if (v != 0 && v != 1) return fail(CONVMI_ERR_INVALID_ARG, "%s must be 0 or 1", name);
    return CONVMI_OK;
}

convmi_status check_mx8(int64_t rows, int64_t cols, int32_t dtype) {
    if (rows < 0 || cols < 1)
        return fail(CONVMI_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1 (rows=%lld cols=%lld)", (long long)rows,
                    (long long)cols);
    CHECK(check_dtype(dtype));
    if (cols > kI32Max - 32 || (rows > 0 && cols > (1LL << 40) / rows))
        return fail(CONVMI_ERR_UNSUPPORTED, "tensor of %lld x %lld exceeds the index limits", (long long)rows,
                    (long long)cols);
    return CONVMI_OK;
}

convmi_status check_rms(const convmi_rms_desc* d) {
    if (!d) return fail(CONVMI_ERR_INVALID_ARG, "desc is NULL");
    if (d->rows < 0 || d->cols < 1)
        return fail(CONVMI_ERR_INVALID_ARG, "rows must be >= 0 and cols >= 1 (rows=%lld cols=%lld)",
                    (long long)d->rows, (long long)d->cols);
    CHECK(check_dtype(d->dtype));
    if (!(d->eps > 0.0f)) return fail(CONVMI_ERR_INVALID_ARG, "eps must be > 0");
    if (d->cols > (1LL << 24) || (d->rows > 0 && d->cols > (1LL << 40) / d->rows))
        return fail(CONVMI_ERR_UNSUPPORTED, "tensor of %lld x %lld exceeds the index limits", (long long)d->rows,
                    (long long)d->cols);
    return CONVMI_OK;
}

convmi_status check_linear(const convmi_linear_desc* d, LinearDims* out) {
    if (!d) return fail(CONVMI_ERR_INVALID_ARG, "desc is NULL");
    if (d->M < 0 || d->K < 1 || d->N < 1)
        return fail(CONVMI_ERR_INVALID_ARG, "M must be >= 0, K and N >= 1 (M=%lld K=%lld N=%lld)", (long long)d->M,
                    (long long)d->K, (long long)d->N);
    CHECK(check_dtype(d->dtype));
    if (d->activation < CONVMI_ACT_IDENTITY || d->activation > CONVMI_ACT_GELU)
        return fail(CONVMI_ERR_INVALID_ARG, "unknown activation %d", d->activation);
    CHECK(check_flag(d->x_mx8, "x_mx8"));
    CHECK(check_flag(d->z_mx8, "z_mx8"));
    if (d->K > (1LL << 20) || d->N > (1LL << 20) || d->M > kI32Max || !linear_fits(d->M, d->K, d->N))
        return fail(CONVMI_ERR_UNSUPPORTED, "problem exceeds the index limits of the kernels");
    *out = LinearDims{d->M, d->K, d->N, d->activation, d->dtype, d->x_mx8, d->z_mx8};
    return CONVMI_OK;
}
// An 8-bit tensor's scales: needed exactly when the descriptor says so.
convmi_status check_scales(const void* scales, int32_t mx8, const char* name, const char* flag) {
    if (mx8) return need(scales, name);
    if (scales) return fail(CONVMI_ERR_INVALID_ARG, "%s given without %s", name, flag);
    return CONVMI_OK;
}
// Output `o` against an input or another output; `same` allows o == i exactly.
convmi_status apart(const char* on, const void* o, size_t ob, const char* in, const void* i, size_t ib,
                    bool same = false) {
    if (!overlaps(o, ob, i, ib) || (same && o == i)) return CONVMI_OK;
    return fail(CONVMI_ERR_INVALID_ARG, "%s overlaps %s", on, in);
}
convmi_status check_linear_op(int32_t op) {
    if (op < CONVMI_LINEAR_FORWARD || op > CONVMI_LINEAR_BACKWARD_WEIGHT)
        return fail(CONVMI_ERR_INVALID_ARG, "unknown linear op %d", op);
    return CONVMI_OK;
}
// Products of MX8 operands have bf16 outputs.
convmi_status check_linear_fwd(const LinearDims& d) {
    if (d.x_mx8 && d.dtype != CONVMI_BF16)
        return fail(CONVMI_ERR_UNSUPPORTED, "linear_forward with x_mx8 has bf16 outputs: dtype must be BF16");
    return CONVMI_OK;
}

}  // namespace

extern "C" {

CONVMI_API convmi_status conv2d_backward_full(const convmi_desc* desc, const void* x, const void* w, const void* saved,
                                              int32_t saved_is_output, const void* dy, void* dx, float* dw, float* db,
                                              int32_t accumulate, void* workspace, size_t workspace_bytes,
                                              void* stream) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    return backward_full_impl("conv2d_backward_full", desc, x, nullptr, w, saved, nullptr, saved_is_output, dy, dx, dw,
                              db, accumulate, ws_backward_full(desc, d), workspace, workspace_bytes, stream);
}

CONVMI_API convmi_status conv2d_backward_full_mx8(const convmi_desc* desc, const void* x, const void* x_scales,
                                                  const void* w, const void* saved, const void* saved_scales,
                                                  int32_t saved_is_output, const void* dy, void* dx, float* dw,
                                                  float* db, int32_t accumulate, void* workspace,
                                                  size_t workspace_bytes, void* stream) {
    ConvDims d;
    CHECK(check_desc(desc, &d));
    return backward_full_impl("conv2d_backward_full_mx8", desc, x, x_scales, w, saved, saved_scales, saved_is_output,
                              dy, dx, dw, db, accumulate, ws_backward_full_mx8(desc, d), workspace, workspace_bytes,
                              stream);
}

CONVMI_API convmi_status mx8_pack(int64_t rows, int64_t cols, int32_t dtype, const void* x, void* codes, void* scales,
                                  void* stream) {
    CHECK(check_mx8(rows, cols, dtype));
    if (rows == 0) return CONVMI_OK;
    CHECK(need(x, "x"));
    CHECK(need(codes, "codes"));
    CHECK(need(scales, "scales"));
    const size_t n = (size_t)rows * cols, xb = n * dtype_size(dtype), sb = (size_t)rows * mx8_blocks(cols);
    CHECK(apart("codes", codes, n, "x", x, xb));
    CHECK(apart("scales", scales, sb, "x", x, xb));
    CHECK(apart("scales", scales, sb, "codes", codes, n));
    const hipError_t e = launch_mx8_pack(dtype, x, rows, (int)cols, codes, scales, (hipStream_t)stream);
    return e == hipSuccess ? CONVMI_OK : hip_fail(e, "mx8_pack launch");
}

CONVMI_API convmi_status mx8_unpack(int64_t rows, int64_t cols, int32_t dtype, const void* codes, const void* scales,
                                    void* x, void* stream) {
    CHECK(check_mx8(rows, cols, dtype));
    if (rows == 0) return CONVMI_OK;
    CHECK(need(codes, "codes"));
    CHECK(need(scales, "scales"));
    CHECK(need(x, "x"));
    const size_t n = (size_t)rows * cols, xb = n * dtype_size(dtype);
    CHECK(apart("x", x, xb, "codes", codes, n));
    CHECK(apart("x", x, xb, "scales", scales, (size_t)rows * mx8_blocks(cols)));
    const hipError_t e = launch_mx8_unpack(dtype, codes, scales, rows, (int)cols, x, (hipStream_t)stream);
    return e == hipSuccess ? CONVMI_OK : hip_fail(e, "mx8_unpack launch");
}

CONVMI_API convmi_status rms_norm_workspace_size(const convmi_rms_desc* desc, size_t* bytes) {
    CHECK(check_rms(desc));
    if (!bytes) return fail(CONVMI_ERR_INVALID_ARG, "bytes out-pointer is NULL");
    *bytes = rms_bwd_ws_bytes(desc->rows, (int)desc->cols);
    return CONVMI_OK;
}

CONVMI_API convmi_status rms_norm_forward(const convmi_rms_desc* desc, const void* x, const void* residual,
                                          const float* gamma, void* h, void* y, void* y8, void* y8_scales,
                                          float* save_inv_rms, void* stream) {
    CHECK(check_rms(desc));
    if ((y8 == nullptr) != (y8_scales == nullptr))
        return fail(CONVMI_ERR_INVALID_ARG, "y8 and y8_scales must be both given or both NULL");
    if (desc->rows == 0) return CONVMI_OK;
    CHECK(need(x, "x"));
    CHECK(need_vec(gamma, "gamma"));
    if (!y && !y8) return fail(CONVMI_ERR_INVALID_ARG, "y is NULL and there is no y8");
    if (residual) CHECK(need(residual, "residual"));
    if (h) CHECK(need(h, "h"));
    if (y) CHECK(need(y, "y"));
    if (y8) CHECK(need(y8, "y8"));
    if (y8) CHECK(need(y8_scales, "y8_scales"));
    if (save_inv_rms) CHECK(need_vec(save_inv_rms, "save_inv_rms"));
    const size_t n = (size_t)desc->rows * desc->cols, b = n * dtype_size(desc->dtype);
    const size_t sb = (size_t)desc->rows * mx8_blocks(desc->cols), gb = (size_t)desc->cols * 4, ib = (size_t)desc->rows * 4;
    struct Out { const char* name; void* p; size_t bytes; };
    const Out outs[5] = {{"h", h, b}, {"y", y, b}, {"y8", y8, n}, {"y8_scales", y8_scales, sb},
                         {"save_inv_rms", save_inv_rms, ib}};
    for (int i = 0; i < 5; ++i) {
        CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, "x", x, b, i == 0));
        CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, "residual", residual, b, i == 0));
        CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, "gamma", gamma, gb));
        for (int j = 0; j < i; ++j)
            CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, outs[j].name, outs[j].p, outs[j].bytes));
    }
    const hipError_t e = launch_rms_fwd(desc->dtype, x, residual, gamma, h, y, y8, y8_scales, save_inv_rms, desc->rows,
                                        (int)desc->cols, desc->eps, (hipStream_t)stream);
    return e == hipSuccess ? CONVMI_OK : hip_fail(e, "rms_norm_forward launch");
}

CONVMI_API convmi_status rms_norm_backward(const convmi_rms_desc* desc, const void* h, const float* gamma,
                                           const float* save_inv_rms, const void* dy, const void* dh, void* dx,
                                           float* dgamma, int32_t accumulate, void* workspace, size_t workspace_bytes,
                                           void* stream) {
    CHECK(check_rms(desc));
    CHECK(check_flag(accumulate, "accumulate"));
    const size_t b = (size_t)desc->rows * desc->cols * dtype_size(desc->dtype);
    if (desc->rows > 0) {
        CHECK(need(h, "h"));
        CHECK(need_vec(gamma, "gamma"));
        CHECK(need_vec(save_inv_rms, "save_inv_rms"));
        CHECK(need(dy, "dy"));
        if (dh) CHECK(need(dh, "dh"));
        CHECK(need(dx, "dx"));
        CHECK(apart("dx", dx, b, "h", h, b));
        CHECK(apart("dx", dx, b, "dy", dy, b, true));
        CHECK(apart("dx", dx, b, "dh", dh, b, true));
        CHECK(apart("dx", dx, b, "gamma", gamma, (size_t)desc->cols * 4));
        CHECK(apart("dx", dx, b, "save_inv_rms", save_inv_rms, (size_t)desc->rows * 4));
    }
    if (dgamma) {
        CHECK(need_vec(dgamma, "dgamma"));
        CHECK(apart("dgamma", dgamma, (size_t)desc->cols * 4, "gamma", gamma, (size_t)desc->cols * 4));
        if (desc->rows > 0) {
            const size_t gb = (size_t)desc->cols * 4;
            CHECK(apart("dgamma", dgamma, gb, "dx", dx, b));
            CHECK(apart("dgamma", dgamma, gb, "h", h, b));
            CHECK(apart("dgamma", dgamma, gb, "dy", dy, b));
            CHECK(apart("dgamma", dgamma, gb, "dh", dh, b));
            CHECK(apart("dgamma", dgamma, gb, "save_inv_rms", save_inv_rms, (size_t)desc->rows * 4));
        }
        CHECK(check_ws(workspace, workspace_bytes, rms_bwd_ws_bytes(desc->rows, (int)desc->cols),
                       "rms_norm_backward"));
    }
    const hipError_t e = launch_rms_bwd(desc->dtype, h, gamma, save_inv_rms, dy, dh, dx, dgamma, accumulate,
                                        desc->rows, (int)desc->cols, workspace, (hipStream_t)stream);
    return e == hipSuccess ? CONVMI_OK : hip_fail(e, "rms_norm_backward launch");
}

CONVMI_API convmi_status linear_workspace_size(const convmi_linear_desc* desc, int32_t op, size_t* bytes) {
    LinearDims d;
    CHECK(check_linear(desc, &d));
    CHECK(check_linear_op(op));
    if (op == CONVMI_LINEAR_FORWARD) CHECK(check_linear_fwd(d));
    if (!bytes) return fail(CONVMI_ERR_INVALID_ARG, "bytes out-pointer is NULL");
    *bytes = linear_ws_bytes(d, op);
    return CONVMI_OK;
}

CONVMI_API convmi_status linear_plan_name(const convmi_linear_desc* desc, int32_t op, char* buf, size_t len) {
    LinearDims d;
    CHECK(check_linear(desc, &d));
    CHECK(check_linear_op(op));
    if (op == CONVMI_LINEAR_FORWARD) CHECK(check_linear_fwd(d));
    if (!buf || len == 0) return fail(CONVMI_ERR_INVALID_ARG, "buf is NULL or len is 0");
    linear_plan_text(d, op, buf, len);
    return CONVMI_OK;
}

CONVMI_API convmi_status linear_forward(const convmi_linear_desc* desc, const void* x, const void* x_scales,
                                        const void* w, const void* w_scales, const float* bias, const void* residual,
                                        void* z, void* z_scales, void* y, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    LinearDims d;
    CHECK(check_linear(desc, &d));
    CHECK(check_linear_fwd(d));
    if (d.M == 0) return CONVMI_OK;
    CHECK(need(x, "x"));
    CHECK(need(w, "w"));
    CHECK(need(y, "y"));
    CHECK(check_scales(x_scales, d.x_mx8, "x_scales", "x_mx8"));
    CHECK(check_scales(w_scales, d.x_mx8, "w_scales", "x_mx8"));
    CHECK(check_scales(z_scales, d.z_mx8 && z, "z_scales", "an 8-bit z"));
    if (bias) CHECK(need_vec(bias, "bias"));
    if (residual) CHECK(need(residual, "residual"));
    if (z) CHECK(need(z, "z"));
    const size_t es = dtype_size(d.dtype), ws_ = d.x_mx8 ? 1 : es;
    const size_t xb = (size_t)d.M * d.K * ws_, wb = (size_t)d.N * d.K * ws_, yn = (size_t)d.M * d.N, yb = yn * es;
    const size_t kb = (size_t)mx8_blocks(d.K);
    struct Out { const char* name; void* p; size_t bytes; };
    const Out outs[3] = {{"y", y, yb}, {"z", z, d.z_mx8 ? yn : yb}, {"z_scales", z_scales, (size_t)d.M * mx8_blocks(d.N)}};
    for (int i = 0; i < 3; ++i) {
        CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, "x", x, xb));
        CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, "w", w, wb));
        CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, "x_scales", x_scales, (size_t)d.M * kb));
        CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, "w_scales", w_scales, (size_t)d.N * kb));
        CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, "bias", bias, (size_t)d.N * 4));
        CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, "residual", residual, yb, i == 0));
        for (int j = 0; j < i; ++j)
            CHECK(apart(outs[i].name, outs[i].p, outs[i].bytes, outs[j].name, outs[j].p, outs[j].bytes));
    }
    CHECK(check_ws(workspace, workspace_bytes, linear_ws_bytes(d, LIN_FORWARD), "linear_forward"));
    const hipError_t e = launch_linear_fwd(d, x, x_scales, w, w_scales, bias, residual, z, z_scales, y, workspace,
                                           (hipStream_t)stream);
    return e == hipSuccess ? CONVMI_OK : hip_fail(e, "linear_forward launch");
}

CONVMI_API convmi_status linear_activation_backward(const convmi_linear_desc* desc, const void* z,
                                                    const void* z_scales, const void* dy, void* dz, void* stream) {
    LinearDims d;
    CHECK(check_linear(desc, &d));
    if (d.M == 0) return CONVMI_OK;
    CHECK(need(z, "z"));
    CHECK(check_scales(z_scales, d.z_mx8, "z_scales", "z_mx8"));
    CHECK(need(dy, "dy"));
    CHECK(need(dz, "dz"));
    const size_t n = (size_t)d.M * d.N, b = n * dtype_size(d.dtype);
    CHECK(apart("dz", dz, b, "dy", dy, b, true));
    CHECK(apart("dz", dz, b, "z", z, d.z_mx8 ? n : b));
    CHECK(apart("dz", dz, b, "z_scales", z_scales, (size_t)d.M * mx8_blocks(d.N)));
    const hipError_t e = d.z_mx8 ? launch_mx8_act_bwd(d.dtype, z, z_scales, 0, dy, dz, d.M, (int)d.N, d.act,
                                                      (hipStream_t)stream)
                                 : launch_act_bwd(d.dtype, z, dy, dz, d.M, (int)d.N, d.act, (hipStream_t)stream);
    return e == hipSuccess ? CONVMI_OK : hip_fail(e, "linear_activation_backward launch");
}

CONVMI_API convmi_status linear_backward_data(const convmi_linear_desc* desc, const void* dz, const void* w, void* dx,
                                              void* workspace, size_t workspace_bytes, void* stream) {
    LinearDims d;
    CHECK(check_linear(desc, &d));
    if (d.M == 0) return CONVMI_OK;
    CHECK(need(dz, "dz"));
    CHECK(need(w, "w"));
    CHECK(need(dx, "dx"));
    const size_t es = dtype_size(d.dtype), xb = (size_t)d.M * d.K * es;
    CHECK(apart("dx", dx, xb, "dz", dz, (size_t)d.M * d.N * es));
    CHECK(apart("dx", dx, xb, "w", w, (size_t)d.N * d.K * es));
    CHECK(check_ws(workspace, workspace_bytes, linear_ws_bytes(d, LIN_BACKWARD_DATA), "linear_backward_data"));
    const hipError_t e = launch_linear_dx(d, dz, w, dx, workspace, (hipStream_t)stream);
    return e == hipSuccess ? CONVMI_OK : hip_fail(e, "linear_backward_data launch");
}

CONVMI_API convmi_status linear_backward_weight(const convmi_linear_desc* desc, const void* x, const void* x_scales,
                                                const void* dz, float* dw, float* db, int32_t accumulate,
                                                void* workspace, size_t workspace_bytes, void* stream) {
    LinearDims d;
    CHECK(check_linear(desc, &d));
    CHECK(check_flag(accumulate, "accumulate"));
    const size_t es = dtype_size(d.dtype), wb = (size_t)d.N * d.K * 4, nb = (size_t)d.N * 4;
    CHECK(need(dw, "dw"));
    if (db) CHECK(need_vec(db, "db"));
    if (d.M > 0) {
        CHECK(need(x, "x"));
        CHECK(check_scales(x_scales, d.x_mx8, "x_scales", "x_mx8"));
        CHECK(need(dz, "dz"));
        const size_t xb = (size_t)d.M * d.K * (d.x_mx8 ? 1 : es), zb = (size_t)d.M * d.N * es;
        CHECK(apart("dw", dw, wb, "x", x, xb));
        CHECK(apart("dw", dw, wb, "x_scales", x_scales, (size_t)d.M * mx8_blocks(d.K)));
        CHECK(apart("dw", dw, wb, "dz", dz, zb));
        CHECK(apart("db", db, nb, "x", x, xb));
        CHECK(apart("db", db, nb, "x_scales", x_scales, (size_t)d.M * mx8_blocks(d.K)));
        CHECK(apart("db", db, nb, "dz", dz, zb));
    }
    CHECK(apart("db", db, nb, "dw", dw, wb));
    CHECK(check_ws(workspace, workspace_bytes, linear_ws_bytes(d, LIN_BACKWARD_WEIGHT), "linear_backward_weight"));
    const hipError_t e = launch_linear_dw(d, x, x_scales, dz, dw, db, accumulate, workspace, (hipStream_t)stream);
    return e == hipSuccess ? CONVMI_OK : hip_fail(e, "linear_backward_weight launch");
}

}  // extern "C"
