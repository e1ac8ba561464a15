// internal.hpp -- host-side interface between the C-ABI front end (api.hip) and the
// kernel translation units.  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.hpp"
#include "seq.hpp"

namespace convmi {

enum DType : int { DT_F32 = 0, DT_BF16 = 1 };

inline size_t dtype_size(int dt) { return dt == DT_BF16 ? 2 : 4; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// A launch counts its threads in 32 bits.
inline bool grid_fits(int64_t blocks, int threads) { return blocks <= (int64_t)UINT32_MAX / threads; }
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// ---------------------------------------------------------------- direct kernels
// General-shape kernels (any IC, stride, padding): one thread per output element.
// They serve small layers and shapes the tiled MFMA kernels do not take.
hipError_t launch_conv_fwd_direct(int dt, const void* x, const void* w, const float* bias, void* z, void* y,
                                  const ConvDims& d, int act, hipStream_t s);
hipError_t launch_conv_dx_direct(int dt, const void* dz, const void* w, void* dx, const ConvDims& d,
                                 hipStream_t s);
hipError_t launch_conv_dw_direct(int dt, const void* x, const void* dz, float* dw, float* db, int accumulate,
                                 const ConvDims& d, hipStream_t s);

// ---------------------------------------------------------------- row reductions
// Per-channel reductions over the M = N*OH*OW rows of a [M][C] tensor are split into
// row slabs (one workgroup each) that write fp32 partials, then merged per channel in
// a fixed order.  The plan depends only on (M, C, dtype), so the workspace size and the
// summation order are reproducible.
struct RowPlan {
    int vec;              // elements per vector access (16 bytes, or 1 when C is not a multiple)
    int tpr;              // threads per row slice
    int rpi;              // rows per iteration of a workgroup
    int chunks;           // channel slices (grid.y)
    int64_t rows_per_block;
    int blocks;           // row slabs (grid.x)
    int bps;              // slabs per segment (all of them for batch norm)
    int64_t seg;          // rows per segment: 0 = all M rows (batch norm), S (per-sample norms)
};
RowPlan row_plan(int64_t M, int C, int dt);
// Layer / group norm: each sample's S = OH*OW rows are a segment of their own.
RowPlan seg_plan(int N, int64_t S, int C, int dt);
size_t bn_stats_ws_bytes(int64_t M, int C, int dt);
size_t bn_bwd_ws_bytes(int64_t M, int C, int dt);

hipError_t launch_bn_stats(int dt, const void* z, int64_t M, int C, float momentum, float eps, float* mean,
                           float* inv_std, float* run_mean, float* run_var, void* ws, hipStream_t s);
// y = act(a), a = z (norm 0) or the batch-norm affine (norm 1).
hipError_t launch_apply_act(int dt, const void* z, void* y, int64_t M, int C, int act, int norm,
                            const float* gamma, const float* beta, const float* mean, const float* inv_std,
                            hipStream_t s);
// dz = act'(z) * dy (no norm).
hipError_t launch_act_bwd(int dt, const void* z, const void* dy, void* dz, int64_t M, int C, int act,
                          hipStream_t s);
// dz = act'(a) * dy with the derivative taken from the output y = act(a) (no norm;
// identity, relu, tanh, sigmoid).
hipError_t launch_act_bwd_from_output(int dt, const void* y, const void* dy, void* dz, int64_t M, int C, int act,
                                      hipStream_t s);
// Batch-norm training backward (+ activation derivative), dgamma/dbeta optional.
hipError_t launch_bn_bwd(int dt, const void* z, const void* dy, void* dz, int64_t M, int C, int act,
                         const float* gamma, const float* beta, const float* mean, const float* inv_std,
                         float* dgamma, float* dbeta, int accumulate, int evaluation, void* ws, hipStream_t s);
hipError_t launch_bn_eval_stats(const float* run_mean, const float* run_var, int C, float eps, float* mean,
                                float* inv_std, hipStream_t s);

// Layer norm (G = 1) and group norm: statistics per sample n and group of C/G
// consecutive channels over the sample's S = OH*OW rows of z [N][S][C], stored at
// [n*G + g]; gamma/beta per channel.
size_t grp_stats_ws_bytes(int N, int64_t S, int C, int dt);
size_t grp_bwd_ws_bytes(int N, int64_t S, int C, int G, int dt);
hipError_t launch_grp_stats(int dt, const void* z, int N, int64_t S, int C, int G, float eps, float* mean,
                            float* inv_std, void* ws, hipStream_t s);
// From the per-tile statistics of the stride-1 forward's epilogue (tiles of one image
// are consecutive, ntiles / N of them per image).
hipError_t launch_grp_tiles_finalize(const float* part, int ntiles, int N, int C, int G, int64_t S, float eps,
                                     float* mean, float* inv_std, hipStream_t s);
hipError_t launch_grp_apply(int dt, const void* z, void* y, int N, int64_t S, int C, int G, int act,
                            const float* gamma, const float* beta, const float* mean, const float* inv_std,
                            hipStream_t s);
hipError_t launch_grp_bwd(int dt, const void* z, const void* dy, void* dz, int N, int64_t S, int C, int G, int act,
                          const float* gamma, const float* beta, const float* mean, const float* inv_std,
                          float* dgamma, float* dbeta, int accumulate, void* ws, hipStream_t s);

// ---------------------------------------------------------------- MFMA implicit GEMM
// Returns false (and launches nothing) when the shape is outside what the tiled
// kernels take; the caller then uses the direct kernels.
bool igemm_fwd_supported(int dt, const ConvDims& d);
bool igemm_dx_supported(int dt, const ConvDims& d);
bool igemm_dw_supported(int dt, const ConvDims& d);
size_t igemm_fwd_ws_bytes(int dt, const ConvDims& d);
size_t igemm_dx_ws_bytes(int dt, const ConvDims& d);
size_t igemm_dw_ws_bytes(int dt, const ConvDims& d);
// True when the weight-gradient kernel's workgroups leave room on a CU for others.
bool dw_leaves_room(int dt, const ConvDims& d);
hipError_t launch_igemm_fwd(int dt, const void* x, const void* w, const float* bias, void* z, void* y,
                            const ConvDims& d, int act, void* ws, hipStream_t s);
hipError_t launch_igemm_dx(int dt, const void* dz, const void* w, void* dx, const ConvDims& d, void* ws,
                           hipStream_t s);
hipError_t launch_igemm_dw(int dt, const void* x, const void* dz, float* dw, float* db, int accumulate,
                           const ConvDims& d, void* ws, hipStream_t s);

// ---------------------------------------------------------------- stride-1 input-tile reuse
// Forward and input gradient of stride-1 layers whose gathered channels fill 128-byte
// chunks: each input tile + halo is copied to LDS once per chunk and shared by all taps.
// bf16 rearranges the weights into MFMA fragment order in the workspace first (ws bytes
// below); fp32 reads w (forward) or the rearranged input-gradient weights of the generic
// path (backward, passed as w) directly.
bool halo_fwd_supported(int dt, const ConvDims& d);
bool halo_dx_supported(int dt, const ConvDims& d);
// Text naming the stride-1 tile plan (block, fragments, tile, halo buffers, paired bands),
// written into buf (at most len bytes, NUL-terminated); false when the layer takes no
// tile plan.
bool halo_plan_text(int dt, const ConvDims& d, bool fwd, char* buf, size_t len);
size_t halo_fwd_ws_bytes(int dt, const ConvDims& d);
size_t halo_dx_ws_bytes(int dt, const ConvDims& d);
// bn_eval: null, or {mean, inv_std, gamma, beta} of evaluation-mode batch norm, applied
// before the activation in the epilogue (y = act(gamma*(z - mean)*inv_std + beta)).
// stats_part: null, or room for 4 * C * halo_fwd_stat_tiles floats of per-tile training
// batch-norm statistics of z; then only z is written (y and act are ignored) and
// launch_bn_tiles_finalize turns the statistics into the batch mean and inverse std.
hipError_t launch_halo_fwd(int dt, const void* x, const void* w, const float* bias, void* z, void* y,
                           const ConvDims& d, int act, void* ws, hipStream_t s,
                           const float* const* bn_eval = nullptr, float* stats_part = nullptr);
int halo_fwd_stat_tiles(int dt, const ConvDims& d);  // spatial tiles of the forward (0: path not taken)
// part[(c*4 + q)*ntiles + tile], q = S1, S2, shift, count (see the forward epilogue).
hipError_t launch_bn_tiles_finalize(const float* part, int ntiles, int C, int64_t M, float momentum, float eps,
                                    float* mean, float* inv_std, float* run_mean, float* run_var, hipStream_t s);
hipError_t launch_halo_dx(int dt, const void* dz, const void* w, void* dx, const ConvDims& d, void* ws,
                          hipStream_t s);

// ---------------------------------------------------------------- 8-bit activations
// MX8 tensors (mx8.hpp): codes [rows][cols], scale bytes [rows][ceil(cols/32)].
hipError_t launch_mx8_pack(int dt, const void* x, int64_t rows, int cols, void* q, void* scales, hipStream_t s);
hipError_t launch_mx8_unpack(int dt, const void* q, const void* scales, int64_t rows, int cols, void* x,
                             hipStream_t s);
// dz = act'(v) * dy at the kept values v = z, or written in terms of v = y; dz may be dy.
hipError_t launch_mx8_act_bwd(int dt, const void* q, const void* scales, int from_output, const void* dy, void* dz,
                              int64_t rows, int cols, int act, hipStream_t s);

// Rows made readable for the tile kernels: copied to a pitch of whole 16-byte chunks with
// zeros behind them, MX8 tensors (scales given) unpacked to the launch's data type on the
// way; up to four tensors in one launch.
struct PrepSeg {
    const char* src;
    const uint8_t* scales;
    char* dst;
    int64_t chunks, src_chunks;  // 16-byte chunks of the copy; those that have a source row
    int row_bytes, per_row;      // of src; chunks per row of dst
    int nb;                      // scale bytes per row
    FastDiv fdr;                 // by per_row, for counts below 2^31
};
struct Prep {
    PrepSeg seg[4];
    int n;
};
// `rows` rows of row_bytes (MX8: codes, unpacked to es-byte values) into a copy at dst whose
// rows take `pitch` bytes (0: the next whole chunk), then zero_rows rows of zeros.
void add_prep(Prep& p, const void* src, const void* scales, void* dst, int64_t rows, int64_t row_bytes, int es,
              int64_t pitch = 0, int64_t zero_rows = 0);
hipError_t launch_prep(const Prep& p, int dt, hipStream_t s);
// The reverse for results: the first cols of every pitch values of src, copied to dst
// [rows][cols] or added to it.
struct CompactSeg {
    const void* src;
    void* dst;
    int64_t rows;
    int cols, pitch, dt, add;
};
struct Compact {
    CompactSeg seg[3];
    int n;
};
hipError_t launch_compact(const Compact& p, hipStream_t s);

// ---------------------------------------------------------------- RMS norm
hipError_t launch_rms_fwd(int dt, const void* x, const void* residual, const float* gamma, void* h, void* y, void* y8,
                          void* y8_scales, float* inv_rms, int64_t rows, int cols, float eps, hipStream_t s);
size_t rms_bwd_ws_bytes(int64_t rows, int cols);
hipError_t launch_rms_bwd(int dt, const void* h, const float* gamma, const float* inv_rms, const void* dy,
                          const void* dh, void* dx, float* dgamma, int accumulate, int64_t rows, int cols, void* ws,
                          hipStream_t s);

// ---------------------------------------------------------------- layer norm
hipError_t launch_layer_norm_fwd(int dt, const void* x, const void* residual, const float* gamma, const float* beta,
                                 void* h, void* y, void* y8, void* y8_scales, float* mean, float* inv_std, int64_t rows,
                                 int cols, float eps, hipStream_t s);
size_t layer_norm_bwd_ws_bytes(int64_t rows, int cols);
hipError_t launch_layer_norm_bwd(int dt, const void* h, const float* gamma, const float* mean, const float* inv_std,
                                 const void* dy, const void* dh, void* dx, float* dgamma, float* dbeta, int accumulate,
                                 int64_t rows, int cols, void* ws, hipStream_t s);

// ---------------------------------------------------------------- causal convolution
struct CausalConvDims {
    Seqs q;
    const void *x, *w;
    const float* bias;    // nullable
    const void* initial;  // nullable
    int D, taps, act, dtype;
    int64_t pitch;  // of x and dx
};
bool causal_conv_fits(int64_t rows, int64_t batch, int D, int taps, int dtype);
bool causal_conv_step_fits(int64_t rows, int D, int dtype);
size_t causal_conv_ws_bytes(int64_t rows, int D, int taps);
hipError_t launch_causal_conv_fwd(const CausalConvDims& d, void* y, void* final, hipStream_t s);
hipError_t launch_causal_conv_bwd(const CausalConvDims& d, const void* dy, const void* dfinal, void* dx, void* dinitial,
                                  float* dw, float* db, int accumulate, void* ws, hipStream_t s);
hipError_t launch_causal_conv_step(const CausalConvDims& d, const Slots& sl, void* state, void* y, hipStream_t s);

// ---------------------------------------------------------------- selective scan
struct ScanDims {
    Seqs q;
    const void *x, *dt, *B, *C, *z;  // z nullable
    const float *dt_bias, *A, *D;    // dt_bias, D nullable
    const float* initial;            // nullable
    int ch, N, G, dtype, softplus;
    int64_t xp, dtp, zp, bcp;
};
struct ScanGrads {
    const float* saved;
    const void* dy;
    const float* dfinal;  // nullable
    void *dx, *ddt, *dB, *dC, *dz;
    float *dA, *dD, *ddt_bias, *dinitial;  // nullable
    int accumulate;
};
bool scan_fits(const ScanDims& d);
bool scan_step_fits(const ScanDims& d);
size_t scan_saved_bytes(const ScanDims& d);
size_t scan_ws_bytes(const ScanDims& d, bool backward);
hipError_t launch_scan_fwd(const ScanDims& d, void* y, float* final, float* saved, void* ws, hipStream_t s);
hipError_t launch_scan_bwd(const ScanDims& d, const ScanGrads& g, void* ws, hipStream_t s);
hipError_t launch_scan_step(const ScanDims& d, const Slots& sl, float* state, void* y, hipStream_t s);

// ---------------------------------------------------------------- linear layer
enum LinOp : int { LIN_FORWARD = 0, LIN_BACKWARD_DATA = 1, LIN_BACKWARD_WEIGHT = 2 };
// Sizes validated on the host: M below 2^31, K and N at most 2^20.
struct LinearDims {
    int64_t M, K, N;
    int act, dtype, x_mx8, z_mx8;
};
// Whether the results of all three operations are few enough 128 x 128 tiles for a launch.
bool linear_fits(int64_t M, int64_t K, int64_t N);
size_t linear_ws_bytes(const LinearDims& d, int op);
void linear_plan_text(const LinearDims& d, int op, char* buf, size_t len);
hipError_t launch_linear_fwd(const LinearDims& d, const void* x, const void* x_sc, const void* w, const void* w_sc,
                             const float* bias, const void* residual, void* z, void* z8_scales, void* y, void* ws,
                             hipStream_t s);
hipError_t launch_linear_dx(const LinearDims& d, const void* dz, const void* w, void* dx, void* ws, hipStream_t s);
hipError_t launch_linear_dw(const LinearDims& d, const void* x, const void* x_sc, const void* dz, float* dw, float* db,
                            int accumulate, void* ws, hipStream_t s);

}  // namespace convmi
