// k_rms.hip -- root-mean-square norm with the residual's addition, and its backward pass.
//
//   forward   h = x + residual;  inv[r] = 1/sqrt(mean_c h^2 + eps);  y = gamma h inv
//   backward  hhat = h inv;  g = gamma dy;  m[r] = mean_c(g hhat)
//             dx = dh + inv (g - hhat m);   dgamma = sum_r dy hhat
//
// Both are one pass over memory (the row stays in registers between its sum and its use),
// bound by HBM: 8192 x 4096 bf16, forward with residual, h and 8-bit y 51 us (4.6 TB/s),
// backward with dh and dgamma 58 us (4.7 TB/s); a plain 1 GiB copy runs at 5.1.  Batches of
// some thousand short rows are bound by latency instead: 2049 x 1003 fp32, dx alone 7.2 us (the
// least a call takes is 3.8, the bytes 4.8; rows that start off 16 bytes cost 0.7, the last,
// nearly empty turn of the workgroups 0.25), dgamma's partial rows and second launch 4.7
// more.  A row belongs to TPR threads, each holding NV pieces of 8 consecutive
// values, piece i of thread t at column 8*(t + i*TPR): whole cache lines per access, and
// the four lanes of a 32-value block side by side for the 8-bit output.  The row sum is a
// fixed butterfly over lanes, then over waves in LDS, so results do not depend on the
// launch.  Rows longer than kMaxRow (kMaxRowBwd) values are read twice instead of held:
// 400 x 65536 bf16 forward 37 us (21 if every byte moved once), backward 74 (31), which reads
// h and dy a third time for dgamma.
//
// dgamma: a thread's columns are the same in every row, so it keeps its share of the sum
// in registers while its workgroup walks over rows; one partial row per workgroup goes to
// the workspace and a second kernel adds those in a fixed order in fp64.
#include "internal.hpp"
#include "lane_sums.hpp"
#include "mx8.hpp"

namespace convmi {
namespace {

constexpr int kThreads = 256;

// Sum over the TPR threads of a row; every thread gets it.  red: one float per wave of
// the workgroup, all of whose threads take part.
template <int TPR> __device__ __forceinline__ float row_sum(float v, float* red) {
    if constexpr (TPR == 16) {
        for (int k = 8; k >= 1; k >>= 1) v += dpp_ror(v, k);
        return v;
    } else {
        v = wave_class_sum(v, 1);
        if constexpr (TPR > 64) {
            __syncthreads();  // the last row's sums have been read
            if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
            __syncthreads();
            const float* mine = red + threadIdx.x / TPR * (TPR / 64);
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < TPR / 64; ++w) s += mine[w];
            return s;
        }
        return v;
    }
}

struct RmsArgs {
    const void *x, *residual;  // residual may be null
    const float* gamma;
    void *h, *y;               // nullable
    uint8_t *y8, *y8_scales;   // nullable
    float* inv_rms;            // nullable
    int64_t rows;
    int cols, nb;              // nb = ceil(cols / 32)
    float eps;
};

template <typename T> __device__ __forceinline__ void rms_load(const RmsArgs& a, int64_t at, int n, float (&v)[kPiece]) {
    load_piece((const T*)a.x + at, n, v);
    if (a.residual) {
        float r[kPiece];
        load_piece((const T*)a.residual + at, n, r);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[j] += r[j];
    }
}
// y (in the data type and / or in 8 bits) and h of one piece; all four lanes of a block
// take part, those past the row's end with zeros.
template <typename T>
__device__ __forceinline__ void rms_store(const RmsArgs& a, int64_t row, int col, int n, const float (&v)[kPiece],
                                          const float (&g)[kPiece], float inv) {
    const int64_t at = row * a.cols + col;
    float y[kPiece];
#pragma unroll
    for (int j = 0; j < kPiece; ++j) y[j] = g[j] * (v[j] * inv);
    if (a.h && n > 0) store_piece((T*)a.h + at, n, v);
    if (a.y && n > 0) store_piece((T*)a.y + at, n, y);
    if (a.y8) {
        uint32_t e;
        const uint2 c = mx_pack(y, e);
        if (n > 0) {
            store_codes(a.y8 + at, n, c);
            if ((threadIdx.x & 3) == 0) a.y8_scales[row * a.nb + col / kMxBlock] = (uint8_t)e;
        }
    }
}

template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void rms_fwd(RmsArgs a) {
    constexpr int RPB = TPR < kThreads ? kThreads / TPR : 1;
    __shared__ float red[(TPR > kThreads ? TPR : kThreads) / 64];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    float g[NV][kPiece];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (t + i * TPR) * kPiece;
        load_piece(a.gamma + col, a.cols - col, g[i]);
    }
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB) {
        const int64_t row = r0 + sub;
        const bool live = row < a.rows;  // whole rows, so whole lane groups, idle together
        float v[NV][kPiece], ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + i * TPR) * kPiece;
            rms_load<T>(a, row * a.cols + col, live ? a.cols - col : 0, v[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) ss = __builtin_fmaf(v[i][j], v[i][j], ss);
        ss = row_sum<TPR>(ss, red);
        const float inv = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
        if (a.inv_rms && live && t == 0) a.inv_rms[row] = inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + i * TPR) * kPiece;
            rms_store<T>(a, row, col, live ? a.cols - col : 0, v[i], g[i], inv);
        }
    }
}

// Rows of any length: the row is read once for its sum and once more for the outputs.
template <typename T> __global__ __launch_bounds__(1024) void rms_fwd_long(RmsArgs a) {
    __shared__ float red[16];
    const int end = a.nb * kMxBlock;  // whole blocks, so that four lanes stay together
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float ss = 0.0f;
        for (int col = threadIdx.x * kPiece; col < a.cols; col += 1024 * kPiece) {
            float v[kPiece];
            rms_load<T>(a, row * a.cols + col, a.cols - col, v);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) ss = __builtin_fmaf(v[j], v[j], ss);
        }
        ss = row_sum<1024>(ss, red);
        const float inv = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
        if (a.inv_rms && threadIdx.x == 0) a.inv_rms[row] = inv;
        for (int col = threadIdx.x * kPiece; col < end; col += 1024 * kPiece) {
            float v[kPiece], g[kPiece];
            rms_load<T>(a, row * a.cols + col, a.cols - col, v);
            load_piece(a.gamma + col, a.cols - col, g);
            rms_store<T>(a, row, col, a.cols - col, v, g, inv);
        }
    }
}

struct RmsBwdArgs {
    const void* h;
    const float *gamma, *inv_rms;
    const void *dy, *dh;  // dh may be null; dx may be dy or dh
    void* dx;
    float* part;          // [gridDim.x][cols] partial dgamma (of one workgroup: dgamma itself), or null
    int add;              // one workgroup: add to what is there
    int64_t rows;
    int cols;
};

template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void rms_bwd(RmsBwdArgs a) {
    constexpr bool AHEAD = TPR < 1024;  // 1024 threads have no registers for the next row
    constexpr int RPB = TPR < kThreads ? kThreads / TPR : 1;
    __shared__ float red[(TPR > kThreads ? TPR : kThreads) / 64];
    __shared__ float cs[RPB > 1 ? RPB * TPR * NV * kPiece : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    float g[NV][kPiece], dg[NV][kPiece];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (t + i * TPR) * kPiece;
        load_piece(a.gamma + col, a.cols - col, g[i]);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) dg[i][j] = 0.0f;
    }
    // The next row's loads are on their way while a row is worked on.
    RawPiece<T> ph[NV], py[NV], pd[NV];
    float pinv = 0.0f;
    auto fetch = [&](int64_t row) {
        const bool live = row < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + i * TPR) * kPiece, n = live ? a.cols - col : 0;
            ph[i] = load_raw((const T*)a.h + row * a.cols + col, n);
            py[i] = load_raw((const T*)a.dy + row * a.cols + col, n);
            pd[i] = load_raw((const T*)a.dh + row * a.cols + col, a.dh ? n : 0);
        }
        pinv = live ? a.inv_rms[row] : 0.0f;
    };
    if (AHEAD) fetch((int64_t)blockIdx.x * RPB + sub);
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB) {
        const int64_t row = r0 + sub;
        const bool live = row < a.rows;
        float hh[NV][kPiece], dy[NV][kPiece], d[NV][kPiece], dot = 0.0f;
        if (!AHEAD) fetch(row);
        const float inv = pinv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            widen(ph[i], hh[i]);
            widen(py[i], dy[i]);
            widen(pd[i], d[i]);
        }
        if (AHEAD) fetch(row + (int64_t)gridDim.x * RPB);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                hh[i][j] *= inv;
                dg[i][j] = __builtin_fmaf(dy[i][j], hh[i][j], dg[i][j]);
                dy[i][j] *= g[i][j];
                dot = __builtin_fmaf(dy[i][j], hh[i][j], dot);
            }
        const float m = row_sum<TPR>(dot, red) / (float)a.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + i * TPR) * kPiece, n = live ? a.cols - col : 0;
            float o[kPiece];
#pragma unroll
            for (int j = 0; j < kPiece; ++j) o[j] = inv * __builtin_fmaf(-hh[i][j], m, dy[i][j]) + d[i][j];
            if (n > 0) store_piece((T*)a.dx + row * a.cols + col, n, o);
        }
    }
    if (!a.part) return;
    if constexpr (RPB > 1) {  // the workgroup's row groups, in order
        constexpr int W = TPR * NV * kPiece;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) cs[sub * W + (t + i * TPR) * kPiece + j] = dg[i][j];
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += kThreads) {
            float s = 0.0f;
            for (int r = 0; r < RPB; ++r) s += cs[r * W + c];
            float* o = a.part + (int64_t)blockIdx.x * a.cols + c;
            *o = a.add ? *o + s : s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + i * TPR) * kPiece;
            if (col >= a.cols) continue;
            float* o = a.part + (int64_t)blockIdx.x * a.cols + col;
            if (a.add) {
                float old[kPiece];
                load_piece(o, a.cols - col, old);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) dg[i][j] += old[j];
            }
            store_piece(o, a.cols - col, dg[i]);
        }
    }
}

// Rows of any length, dx only: two passes over the row (dgamma comes from col_sums).
template <typename T> __global__ __launch_bounds__(1024) void rms_bwd_long(RmsBwdArgs a) {
    __shared__ float red[16];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float inv = a.inv_rms[row];
        float dot = 0.0f;
        for (int col = threadIdx.x * kPiece; col < a.cols; col += 1024 * kPiece) {
            const int64_t at = row * a.cols + col;
            float h[kPiece], dy[kPiece], g[kPiece];
            load_piece((const T*)a.h + at, a.cols - col, h);
            load_piece((const T*)a.dy + at, a.cols - col, dy);
            load_piece(a.gamma + col, a.cols - col, g);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) dot = __builtin_fmaf(dy[j] * g[j], h[j] * inv, dot);
        }
        const float m = row_sum<1024>(dot, red) / (float)a.cols;
        for (int col = threadIdx.x * kPiece; col < a.cols; col += 1024 * kPiece) {
            const int64_t at = row * a.cols + col;
            float h[kPiece], dy[kPiece], g[kPiece], d[kPiece];
            load_piece((const T*)a.h + at, a.cols - col, h);
            load_piece((const T*)a.dy + at, a.cols - col, dy);
            load_piece(a.gamma + col, a.cols - col, g);
            if (a.dh) load_piece((const T*)a.dh + at, a.cols - col, d);
            float o[kPiece];
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                o[j] = inv * __builtin_fmaf(-(h[j] * inv), m, dy[j] * g[j]);
                if (a.dh) o[j] += d[j];
            }
            store_piece((T*)a.dx + at, a.cols - col, o);
        }
    }
}

// ---------------------------------------------------------------- column sums
// dgamma of long rows: part[slab][c] = sum over the slab's rows of dy[r][c] h[r][c] inv[r].  A
// workgroup owns TX pieces of 8 columns and a slab of rows, its 256 / TX row groups
// taking every (256 / TX)-th row; they are added in order at the end.
template <typename T>
__global__ __launch_bounds__(kThreads) void col_sums(const T* __restrict__ dy, const T* __restrict__ h,
                                                     const float* __restrict__ inv, int64_t rows, int cols, int tx_log,
                                                     int64_t slab_rows, float* __restrict__ part) {
    __shared__ float cs[kThreads * kPiece];
    const int tx = 1 << tx_log, ty = kThreads >> tx_log;
    const int x = threadIdx.x & (tx - 1), y = threadIdx.x >> tx_log;
    const int col = (blockIdx.x * tx + x) * kPiece, n = cols - col;
    const int64_t begin = blockIdx.y * slab_rows, end = begin + slab_rows < rows ? begin + slab_rows : rows;
    float s[kPiece] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    constexpr int U = 8;  // rows whose loads are in flight together
    for (int64_t r = begin + y; r < end; r += (int64_t)ty * U) {
        float v[U][kPiece], w[U][kPiece], k[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = r + (int64_t)u * ty;
            const int m = row < end ? n : 0;
            load_piece(dy + row * cols + col, m, v[u]);
            load_piece(h + row * cols + col, m, w[u]);
            k[u] = row < end ? inv[row] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) s[j] = __builtin_fmaf(v[u][j], w[u][j] * k[u], s[j]);
    }
#pragma unroll
    for (int j = 0; j < kPiece; ++j) cs[threadIdx.x * kPiece + j] = s[j];
    __syncthreads();
    const int width = tx * kPiece, c0 = blockIdx.x * width;
    for (int c = threadIdx.x; c < width && c0 + c < cols; c += kThreads) {
        float t = 0.0f;
        for (int g = 0; g < ty; ++g) t += cs[g * width + c];
        part[(int64_t)blockIdx.y * cols + c0 + c] = t;
    }
}

// out[c] (+)= sum over the slabs, in fp64: 16 slab groups of 16 columns per workgroup, each
// adding every sixteenth slab (16 loads in flight), then the groups in order.
__global__ __launch_bounds__(kThreads) void col_sums_merge(const float* __restrict__ part, int slabs, int cols,
                                                           int accumulate, float* __restrict__ out) {
    constexpr int G = 16, U = 16;
    __shared__ double cs[G][kThreads / G];
    const int x = threadIdx.x % (kThreads / G), y = threadIdx.x / (kThreads / G);
    const int c = blockIdx.x * (kThreads / G) + x;
    double s = 0.0;
    if (c < cols) {
        int k = y;
        for (; k + G * (U - 1) < slabs; k += G * U) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = part[(int64_t)(k + G * u) * cols + c];
#pragma unroll
            for (int u = 0; u < U; ++u) s += (double)v[u];
        }
        for (; k < slabs; k += G) s += (double)part[(int64_t)k * cols + c];
    }
    cs[y][x] = s;
    __syncthreads();
    if (y == 0 && c < cols) {
        for (int g = 1; g < G; ++g) s += cs[g][x];
        out[c] = accumulate ? (float)((double)out[c] + s) : (float)s;
    }
}

// ---------------------------------------------------------------- host side
// Threads and pieces per row.  16 or 64 threads keep the sum inside a wave, so short
// rows need no barrier; more spread long rows until a thread's values fit the registers:
// 32 of them in the forward (1024 threads have 128 registers each), 16 in the backward,
// which keeps gamma, the dgamma sums and, up to 512 threads, the next row beside them
// (8192 x 4096 bf16, when the step was made: 65 us without the next row's loads ahead, 58
// with).
constexpr int kMaxRow = 1024 * 4 * kPiece, kMaxRowBwd = 1024 * 2 * kPiece;
#define CONVMI_RMS_SWITCH(cols, TPR, NV, ...)                                                        \
    do {                                                                                             \
        if ((cols) <= 16 * kPiece) { constexpr int TPR = 16, NV = 1; __VA_ARGS__; }                  \
        else if ((cols) <= 64 * kPiece) { constexpr int TPR = 64, NV = 1; __VA_ARGS__; }             \
        else if ((cols) <= 128 * kPiece) { constexpr int TPR = 64, NV = 2; __VA_ARGS__; }            \
        else if ((cols) <= 256 * kPiece) { constexpr int TPR = 256, NV = 1; __VA_ARGS__; }           \
        else if ((cols) <= 512 * kPiece) { constexpr int TPR = 256, NV = 2; __VA_ARGS__; }           \
        else if ((cols) <= 1024 * kPiece) { constexpr int TPR = 256, NV = 4; __VA_ARGS__; }          \
        else if ((cols) <= 2048 * kPiece) { constexpr int TPR = 1024, NV = 2; __VA_ARGS__; }         \
        else { constexpr int TPR = 1024, NV = 4; __VA_ARGS__; }                                      \
    } while (0)
#define CONVMI_RMS_BWD_SWITCH(cols, TPR, NV, ...)                                                    \
    do {                                                                                             \
        if ((cols) <= 16 * kPiece) { constexpr int TPR = 16, NV = 1; __VA_ARGS__; }                  \
        else if ((cols) <= 64 * kPiece) { constexpr int TPR = 64, NV = 1; __VA_ARGS__; }             \
        else if ((cols) <= 128 * kPiece) { constexpr int TPR = 128, NV = 1; __VA_ARGS__; }           \
        else if ((cols) <= 256 * kPiece) { constexpr int TPR = 256, NV = 1; __VA_ARGS__; }           \
        else if ((cols) <= 512 * kPiece) { constexpr int TPR = 512, NV = 1; __VA_ARGS__; }           \
        else if ((cols) <= 1024 * kPiece) { constexpr int TPR = 512, NV = 2; __VA_ARGS__; }          \
        else { constexpr int TPR = 1024, NV = 2; __VA_ARGS__; }                                      \
    } while (0)

// Workgroups of a row kernel whose rows take tpr threads: as many as the rows fill, at most
// `waves` waves.
int rms_blocks(int64_t rows, int tpr, int waves) {
    const int threads = tpr > kThreads ? tpr : kThreads;
    const int64_t need = ceil_div(rows, threads / tpr);
    const int cap = waves / (threads / 64);
    return (int)(need < cap ? need : cap);
}
// The backward's partial dgamma rows are one per workgroup: half as many waves with the next
// row ahead are as fast (8192 x 4096 bf16: 57.3 us with 2048, 57.0 with 4096, 61.4 with
// 6144) and leave less to merge (16384 x 512: 17.3, 18.1, 20.4).  1024-thread rows, which do
// not load ahead, need 4096 (2000 x 16384: 63.6 against 72.2).
constexpr int kFwdWaves = 8192, kBwdWaves = 2048, kBwdWavesLong = 4096;
int rms_fwd_blocks(int64_t rows, int cols) {
    int tpr = 1024;
    if (cols <= kMaxRow) CONVMI_RMS_SWITCH(cols, TPR, NV, { tpr = TPR; (void)NV; });
    return rms_blocks(rows, tpr, kFwdWaves);
}
// Few rows: one workgroup walks over all of them, and dgamma needs no second launch.
int rms_bwd_blocks(int64_t rows, int cols) {
    int tpr = 1024;
    if (cols <= kMaxRowBwd) CONVMI_RMS_BWD_SWITCH(cols, TPR, NV, { tpr = TPR; (void)NV; });
    const int per_pass = tpr < kThreads ? kThreads / tpr : 1;
    return cols <= kMaxRowBwd && rows <= 3 * per_pass ? 1 : rms_blocks(rows, tpr, tpr < 1024 ? kBwdWaves : kBwdWavesLong);
}

struct ColPlan {
    int tx_log, gx, slabs;
    int64_t slab_rows;
};
// Enough workgroups to keep loads in flight on every CU, but slabs of at least 8 rows
// per row group, so that the partial rows stay few beside the data.
ColPlan col_plan(int64_t rows, int cols) {
    ColPlan p;
    p.tx_log = 0;
    while (p.tx_log < 6 && (kPiece << p.tx_log) < cols) ++p.tx_log;
    p.gx = (int)ceil_div(cols, kPiece << p.tx_log);
    const int ty = kThreads >> p.tx_log;
    int64_t slabs = ceil_div(1024, p.gx);
    const int64_t most = ceil_div(rows, (int64_t)ty * 8);
    if (slabs > most) slabs = most;
    if (slabs > 512) slabs = 512;
    if (slabs < 1) slabs = 1;
    p.slab_rows = ceil_div(rows > 0 ? rows : 1, slabs);
    p.slabs = (int)ceil_div(rows > 0 ? rows : 1, p.slab_rows);
    return p;
}

template <typename T>
hipError_t launch_cols(const void* dy, const void* h, const float* inv, int64_t rows, int cols, float* out,
                       int accumulate, void* ws, hipStream_t s) {
    const ColPlan p = col_plan(rows, cols);
    col_sums<T><<<dim3(p.gx, p.slabs), kThreads, 0, s>>>((const T*)dy, (const T*)h, inv, rows, cols, p.tx_log,
                                                         p.slab_rows, (float*)ws);
    col_sums_merge<<<(unsigned)ceil_div(cols, 16), kThreads, 0, s>>>((const float*)ws, p.slabs, cols, accumulate, out);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_fwd(int dt, const void* x, const void* residual, const float* gamma, void* h, void* y, void* y8,
                          void* y8_scales, float* inv_rms, int64_t rows, int cols, float eps, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    const RmsArgs a{x,  residual, gamma, h, y, (uint8_t*)y8, (uint8_t*)y8_scales, inv_rms, rows, cols,
                    (int)ceil_div(cols, kMxBlock), eps};
    const int blocks = rms_fwd_blocks(rows, cols);
    if (cols > kMaxRow) {
        if (dt == DT_BF16) rms_fwd_long<bf16><<<blocks, 1024, 0, s>>>(a);
        else rms_fwd_long<float><<<blocks, 1024, 0, s>>>(a);
        return hipGetLastError();
    }
    CONVMI_RMS_SWITCH(cols, TPR, NV, {
        constexpr int threads = TPR > kThreads ? TPR : kThreads;
        if (dt == DT_BF16) rms_fwd<bf16, TPR, NV><<<blocks, threads, 0, s>>>(a);
        else rms_fwd<float, TPR, NV><<<blocks, threads, 0, s>>>(a);
    });
    return hipGetLastError();
}

size_t rms_bwd_ws_bytes(int64_t rows, int cols) {
    if (cols > kMaxRowBwd || rows == 0)
        return align_up((size_t)col_plan(rows, cols).slabs * cols * sizeof(float), 256);
    return align_up((size_t)rms_bwd_blocks(rows, cols) * cols * sizeof(float), 256);
}

hipError_t launch_rms_bwd(int dt, const void* h, const float* gamma, const float* inv_rms, const void* dy,
                          const void* dh, void* dx, float* dgamma, int accumulate, int64_t rows, int cols, void* ws,
                          hipStream_t s) {
    const bool held = cols <= kMaxRowBwd && rows > 0;
    // dgamma first where it has its own pass: dx may overwrite dy.
    if (dgamma && !held) {
        const hipError_t e = dt == DT_BF16
                                 ? launch_cols<bf16>(dy, h, inv_rms, rows, cols, dgamma, accumulate, ws, s)
                                 : launch_cols<float>(dy, h, inv_rms, rows, cols, dgamma, accumulate, ws, s);
        if (e != hipSuccess) return e;
    }
    if (rows == 0) return hipSuccess;
    const int blocks = rms_bwd_blocks(rows, cols);
    float* part = !held || !dgamma ? nullptr : blocks == 1 ? dgamma : (float*)ws;
    const RmsBwdArgs a{h, gamma, inv_rms, dy, dh, dx, part, blocks == 1 && accumulate, rows, cols};
    if (!held) {
        if (dt == DT_BF16) rms_bwd_long<bf16><<<blocks, 1024, 0, s>>>(a);
        else rms_bwd_long<float><<<blocks, 1024, 0, s>>>(a);
        return hipGetLastError();
    }
    CONVMI_RMS_BWD_SWITCH(cols, TPR, NV, {
        constexpr int threads = TPR > kThreads ? TPR : kThreads;
        if (dt == DT_BF16) rms_bwd<bf16, TPR, NV><<<blocks, threads, 0, s>>>(a);
        else rms_bwd<float, TPR, NV><<<blocks, threads, 0, s>>>(a);
    });
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && dgamma && blocks > 1) {
        col_sums_merge<<<(unsigned)ceil_div(cols, 16), kThreads, 0, s>>>((const float*)ws, blocks, cols, accumulate,
                                                                         dgamma);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace convmi
