// k_rms.hip -- root-mean-square norm and layer norm with the residual's addition, and their backward
// passes.
//
//   forward   h = x + residual;  inv[r] = 1/sqrt(mean_c h^2 + eps);  y = gamma h inv
//   backward  hhat = h inv;  g = gamma dy;  m[r] = mean_c(g hhat)
//             dx = dh + inv (g - hhat m);   dgamma = sum_r dy hhat
// Layer norm (LN) takes the row's mean off first:
//   forward   c = h - mean;  inv[r] = 1/sqrt(mean_c c^2 + eps);  y = gamma c inv + beta
//   backward  hhat = c inv;  dx = dh + inv (g - mean_c(g) - hhat m);  dbeta = sum_r dy
// The squares are taken around the mean, from the registers that hold the row; both sums of the
// backward go through the same barriers.  8192 x 4096 bf16: forward with residual and h 53 us
// (5.1 TB/s), backward with dh, dgamma and dbeta 60 (4.5 TB/s, the merge of the sums 6.7 of it).
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

// Both sums of the row's threads, through the same barriers.  red: two floats per wave.
template <int TPR> __device__ __forceinline__ void row_sum2(float& a, float& b, float* red) {
    if constexpr (TPR <= 64) {
        a = row_sum<TPR>(a, red);
        b = row_sum<TPR>(b, red);
    } else {
        a = wave_class_sum(a, 1);
        b = wave_class_sum(b, 1);
        __syncthreads();  // the last row's sums have been read
        if ((threadIdx.x & 63) == 0) {
            red[threadIdx.x >> 6 << 1] = a;
            red[(threadIdx.x >> 6 << 1) + 1] = b;
        }
        __syncthreads();
        const float* mine = red + threadIdx.x / TPR * (TPR / 32);
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) {
            a += mine[2 * w];
            b += mine[2 * w + 1];
        }
    }
}

// Squares of v's first n values around the row's mean, added to s.
__device__ __forceinline__ float add_squares(const float (&v)[kPiece], int n, float mean, float s) {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
        const float c = j < n ? v[j] - mean : 0.0f;
        s = __builtin_fmaf(c, c, s);
    }
    return s;
}

struct RmsArgs {
    const void *x, *residual;  // residual may be null
    const float *gamma, *beta; // beta: layer norm, may be null
    void *h, *y;               // nullable
    uint8_t *y8, *y8_scales;   // nullable
    float *mean, *inv;         // nullable; mean: layer norm
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
// take part, those past the row's end with zeros (gamma and beta are loaded as 0 there).
template <typename T, bool LN>
__device__ __forceinline__ void rms_store(const RmsArgs& a, int64_t row, int col, int n, const float (&v)[kPiece],
                                          const float (&g)[kPiece], const float (&b)[kPiece], float mean, float inv) {
    const int64_t at = row * a.cols + col;
    float y[kPiece];
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
        if constexpr (LN) y[j] = __builtin_fmaf(g[j], (v[j] - mean) * inv, b[j]);
        else y[j] = g[j] * (v[j] * inv);
    }
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

template <typename T, int TPR, int NV, bool LN>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void rms_fwd(RmsArgs a) {
    constexpr int RPB = TPR < kThreads ? kThreads / TPR : 1;
    __shared__ float red[(TPR > kThreads ? TPR : kThreads) / 64];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    constexpr bool HOLD = !LN || TPR * NV < 4096;  // 1024 threads have no registers for gamma and beta beside four pieces
    float g[NV][kPiece], b[NV][kPiece];
    auto affine = [&](int i) {
        const int col = (t + i * TPR) * kPiece;
        load_piece(a.gamma + col, a.cols - col, g[i]);
        if constexpr (LN) load_piece(a.beta + col, a.beta ? a.cols - col : 0, b[i]);
    };
    if constexpr (HOLD) {
#pragma unroll
        for (int i = 0; i < NV; ++i) affine(i);
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
        float mean = 0.0f;
        if constexpr (LN) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < kPiece; ++j) mean += v[i][j];
            mean = row_sum<TPR>(mean, red) / (float)a.cols;
#pragma unroll
            for (int i = 0; i < NV; ++i) ss = add_squares(v[i], a.cols - (t + i * TPR) * kPiece, mean, ss);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < kPiece; ++j) ss = __builtin_fmaf(v[i][j], v[i][j], ss);
        }
        ss = row_sum<TPR>(ss, red);
        const float inv = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
        if (a.inv && live && t == 0) a.inv[row] = inv;
        if (LN && a.mean && live && t == 0) a.mean[row] = mean;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + i * TPR) * kPiece;
            if constexpr (!HOLD) affine(i);
            rms_store<T, LN>(a, row, col, live ? a.cols - col : 0, v[i], g[i], b[i], mean, inv);
        }
    }
}

// Rows of any length: the row is read once for each sum (the mean's and the squares' around
// it; RMS: the squares') and once more for the outputs.
template <typename T, bool LN> __global__ __launch_bounds__(1024) void rms_fwd_long(RmsArgs a) {
    __shared__ float red[16];
    const int end = a.nb * kMxBlock;  // whole blocks, so that four lanes stay together
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float ss = 0.0f, mean = 0.0f;
        if constexpr (LN) {
            for (int col = threadIdx.x * kPiece; col < a.cols; col += 1024 * kPiece) {
                float v[kPiece];
                rms_load<T>(a, row * a.cols + col, a.cols - col, v);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) mean += v[j];
            }
            mean = row_sum<1024>(mean, red) / (float)a.cols;
            if (a.mean && threadIdx.x == 0) a.mean[row] = mean;
        }
        for (int col = threadIdx.x * kPiece; col < a.cols; col += 1024 * kPiece) {
            float v[kPiece];
            rms_load<T>(a, row * a.cols + col, a.cols - col, v);
            if constexpr (LN) {
                ss = add_squares(v, a.cols - col, mean, ss);
            } else {
#pragma unroll
                for (int j = 0; j < kPiece; ++j) ss = __builtin_fmaf(v[j], v[j], ss);
            }
        }
        ss = row_sum<1024>(ss, red);
        const float inv = 1.0f / sqrtf(ss / (float)a.cols + a.eps);
        if (a.inv && threadIdx.x == 0) a.inv[row] = inv;
        for (int col = threadIdx.x * kPiece; col < end; col += 1024 * kPiece) {
            float v[kPiece], g[kPiece], b[kPiece];
            rms_load<T>(a, row * a.cols + col, a.cols - col, v);
            load_piece(a.gamma + col, a.cols - col, g);
            if constexpr (LN) load_piece(a.beta + col, a.beta ? a.cols - col : 0, b);
            rms_store<T, LN>(a, row, col, a.cols - col, v, g, b, mean, inv);
        }
    }
}

struct RmsBwdArgs {
    const void* h;
    const float *gamma, *mean, *inv;  // mean: layer norm
    const void *dy, *dh;  // dh may be null; dx may be dy or dh
    void* dx;
    float* part;          // [gridDim.x][cols] partial dgamma (of one workgroup: dgamma itself), or null
    float* part_b;        // layer norm: dbeta's likewise, or null
    int add;              // one workgroup: add to what is there
    int64_t rows;
    int cols;
};

// A thread's sums over the workgroup's rows, of its columns: into row blockIdx.x of part.
template <int TPR, int NV>
__device__ __forceinline__ void put_sums(float (&d)[NV][kPiece], float* part, int cols, int add, float* cs) {
    constexpr int RPB = TPR < kThreads ? kThreads / TPR : 1;
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    part += (int64_t)blockIdx.x * cols;
    if constexpr (RPB > 1) {  // the workgroup's row groups, in order
        constexpr int W = TPR * NV * kPiece;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) cs[sub * W + (t + i * TPR) * kPiece + j] = d[i][j];
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += kThreads) {
            float s = 0.0f;
            for (int r = 0; r < RPB; ++r) s += cs[r * W + c];
            part[c] = add ? part[c] + s : s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + i * TPR) * kPiece;
            if (col >= cols) continue;
            if (add) {
                float old[kPiece];
                load_piece(part + col, cols - col, old);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) d[i][j] += old[j];
            }
            store_piece(part + col, cols - col, d[i]);
        }
    }
}

template <typename T, int TPR, int NV, bool LN>
__global__ __launch_bounds__(TPR > kThreads ? TPR : kThreads) void rms_bwd(RmsBwdArgs a) {
    constexpr bool AHEAD = TPR < 1024;  // 1024 threads have no registers for the next row
    constexpr int RPB = TPR < kThreads ? kThreads / TPR : 1;
    __shared__ float red[(TPR > kThreads ? TPR : kThreads) / 32];
    __shared__ float cs[RPB > 1 ? RPB * TPR * NV * kPiece : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    constexpr bool HOLD = !LN || TPR < 1024;  // gamma in registers
    float g[NV][kPiece], dg[NV][kPiece], db[LN ? NV : 1][kPiece];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (t + i * TPR) * kPiece;
        if (HOLD) load_piece(a.gamma + col, a.cols - col, g[i]);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
            dg[i][j] = 0.0f;
            if (LN) db[i][j] = 0.0f;
        }
    }
    // The next row's loads are on their way while a row is worked on.
    RawPiece<T> ph[NV], py[NV], pd[NV];
    float pinv = 0.0f, pmean = 0.0f;
    auto fetch = [&](int64_t row) {
        const bool live = row < a.rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + i * TPR) * kPiece, n = live ? a.cols - col : 0;
            ph[i] = load_raw((const T*)a.h + row * a.cols + col, n);
            py[i] = load_raw((const T*)a.dy + row * a.cols + col, n);
            pd[i] = load_raw((const T*)a.dh + row * a.cols + col, a.dh ? n : 0);
        }
        pinv = live ? a.inv[row] : 0.0f;
        if (LN) pmean = live ? a.mean[row] : 0.0f;
    };
    if (AHEAD) fetch((int64_t)blockIdx.x * RPB + sub);
    for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB) {
        const int64_t row = r0 + sub;
        const bool live = row < a.rows;
        float hh[NV][kPiece], dy[NV][kPiece], d[NV][kPiece], dot = 0.0f;
        if (!AHEAD) fetch(row);
        const float inv = pinv, mean = pmean;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            widen(ph[i], hh[i]);
            widen(py[i], dy[i]);
            widen(pd[i], d[i]);
        }
        if (AHEAD) fetch(row + (int64_t)gridDim.x * RPB);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + i * TPR) * kPiece;
            if (!HOLD) load_piece(a.gamma + col, a.cols - col, g[i]);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                if constexpr (LN) {
                    hh[i][j] = (hh[i][j] - mean) * inv;
                    db[i][j] += dy[i][j];
                } else {
                    hh[i][j] *= inv;
                }
                dg[i][j] = __builtin_fmaf(dy[i][j], hh[i][j], dg[i][j]);
                dy[i][j] *= g[i][j];
                dot = __builtin_fmaf(dy[i][j], hh[i][j], dot);
                if (LN) sum += dy[i][j];
            }
        }
        if constexpr (LN) row_sum2<TPR>(dot, sum, red);
        else dot = row_sum<TPR>(dot, red);
        const float m = dot / (float)a.cols, m1 = sum / (float)a.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (t + i * TPR) * kPiece, n = live ? a.cols - col : 0;
            float o[kPiece];
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
                o[j] = inv * __builtin_fmaf(-hh[i][j], m, LN ? dy[i][j] - m1 : dy[i][j]) + d[i][j];
            if (n > 0) store_piece((T*)a.dx + row * a.cols + col, n, o);
        }
    }
    if (a.part) put_sums<TPR, NV>(dg, a.part, a.cols, a.add, cs);
    if constexpr (LN) {
        if (a.part_b) put_sums<TPR, NV>(db, a.part_b, a.cols, a.add, cs);
    }
}

// Rows of any length, dx only: two passes over the row (dgamma and dbeta come from col_sums).
template <typename T, bool LN> __global__ __launch_bounds__(1024) void rms_bwd_long(RmsBwdArgs a) {
    __shared__ float red[32];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float inv = a.inv[row], mean = LN ? a.mean[row] : 0.0f;
        float dot = 0.0f, sum = 0.0f;
        for (int col = threadIdx.x * kPiece; col < a.cols; col += 1024 * kPiece) {
            const int64_t at = row * a.cols + col;
            float h[kPiece], dy[kPiece], g[kPiece];
            load_piece((const T*)a.h + at, a.cols - col, h);
            load_piece((const T*)a.dy + at, a.cols - col, dy);
            load_piece(a.gamma + col, a.cols - col, g);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                const float w = dy[j] * g[j];
                dot = __builtin_fmaf(w, (LN ? h[j] - mean : h[j]) * inv, dot);
                if (LN) sum += w;
            }
        }
        if constexpr (LN) row_sum2<1024>(dot, sum, red);
        else dot = row_sum<1024>(dot, red);
        const float m = dot / (float)a.cols, m1 = sum / (float)a.cols;
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
                const float w = dy[j] * g[j];
                o[j] = inv * __builtin_fmaf(-((LN ? h[j] - mean : h[j]) * inv), m, LN ? w - m1 : w);
                if (a.dh) o[j] += d[j];
            }
            store_piece((T*)a.dx + at, a.cols - col, o);
        }
    }
}

// ---------------------------------------------------------------- column sums
// dgamma of long rows: part[slab][c] = sum over the slab's rows of dy[r][c] hhat[r][c], and for
// layer norm dbeta's sums of dy[r][c] in part_b.  A workgroup owns TX pieces of 8 columns and
// a slab of rows, its 256 / TX row groups taking every (256 / TX)-th row; they are added in
// order at the end.
template <typename T, bool LN>
__global__ __launch_bounds__(kThreads) void col_sums(const T* __restrict__ dy, const T* __restrict__ h,
                                                     const float* __restrict__ mean, const float* __restrict__ inv,
                                                     int64_t rows, int cols, int tx_log, int64_t slab_rows,
                                                     float* __restrict__ part, float* __restrict__ part_b) {
    __shared__ float cs[kThreads * kPiece];
    const int tx = 1 << tx_log, ty = kThreads >> tx_log;
    const int x = threadIdx.x & (tx - 1), y = threadIdx.x >> tx_log;
    const int col = (blockIdx.x * tx + x) * kPiece, n = cols - col;
    const int64_t begin = blockIdx.y * slab_rows, end = begin + slab_rows < rows ? begin + slab_rows : rows;
    float s[kPiece] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sb[kPiece] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    constexpr int U = 8;  // rows whose loads are in flight together
    for (int64_t r = begin + y; r < end; r += (int64_t)ty * U) {
        float v[U][kPiece], w[U][kPiece], k[U], mu[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = r + (int64_t)u * ty;
            const int m = row < end ? n : 0;
            load_piece(dy + row * cols + col, m, v[u]);
            load_piece(h + row * cols + col, m, w[u]);
            k[u] = row < end ? inv[row] : 0.0f;
            mu[u] = LN && row < end ? mean[row] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                s[j] = __builtin_fmaf(v[u][j], (LN ? w[u][j] - mu[u] : w[u][j]) * k[u], s[j]);
                if (LN) sb[j] += v[u][j];
            }
    }
    const int width = tx * kPiece, c0 = blockIdx.x * width;
    for (int q = 0; q < (LN ? 2 : 1); ++q) {
        if (q) __syncthreads();
#pragma unroll
        for (int j = 0; j < kPiece; ++j) cs[threadIdx.x * kPiece + j] = q ? sb[j] : s[j];
        __syncthreads();
        float* out = q ? part_b : part;
        for (int c = threadIdx.x; c < width && c0 + c < cols; c += kThreads) {
            float t = 0.0f;
            for (int g = 0; g < ty; ++g) t += cs[g * width + c];
            out[(int64_t)blockIdx.y * cols + c0 + c] = t;
        }
    }
}

// out[c] (+)= sum over the slabs, in fp64: 16 slab groups of 16 columns per workgroup, each
// adding every sixteenth slab (16 loads in flight), then the groups in order.  The second
// workgroup row does the same for layer norm's dbeta.
__global__ __launch_bounds__(kThreads) void col_sums_merge(const float* __restrict__ part0, const float* __restrict__ part1,
                                                           int slabs, int cols, int accumulate, float* __restrict__ out0,
                                                           float* __restrict__ out1) {
    const float* __restrict__ part = blockIdx.y ? part1 : part0;
    float* __restrict__ out = blockIdx.y ? out1 : out0;
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
// Layer norm, with twice the sums, takes 59.9 + 4.9 us (8192 x 4096 bf16, rows and merge) with two
// waves a SIMD, 53.2 + 6.7 with three, 56.8 + 6.6 with four.
constexpr int kSimds = 1024;
constexpr int kFwdWaves = 8192, kBwdWaves = 2048, kBwdWavesMean = 3 * kSimds, kBwdWavesLong = 4096;
int rms_fwd_blocks(int64_t rows, int cols) {
    int tpr = 1024;
    if (cols <= kMaxRow) CONVMI_RMS_SWITCH(cols, TPR, NV, { tpr = TPR; (void)NV; });
    return rms_blocks(rows, tpr, kFwdWaves);
}
// Few rows: one workgroup walks over all of them, and dgamma needs no second launch.
int rms_bwd_blocks(int64_t rows, int cols, bool ln) {
    int tpr = 1024;
    if (cols <= kMaxRowBwd) CONVMI_RMS_BWD_SWITCH(cols, TPR, NV, { tpr = TPR; (void)NV; });
    const int per_pass = tpr < kThreads ? kThreads / tpr : 1;
    if (cols <= kMaxRowBwd && rows <= 3 * per_pass) return 1;
    return rms_blocks(rows, tpr, tpr >= 1024 ? kBwdWavesLong : ln ? kBwdWavesMean : kBwdWaves);
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

// Where the partial sums of dgamma and, behind them, of dbeta lie in the workspace.
struct Sums {
    float *dgamma, *dbeta;  // nullable
    float *part_g, *part_b;
    int slabs;
};
void launch_merge(const Sums& o, int cols, int accumulate, hipStream_t s) {
    const unsigned blocks = (unsigned)ceil_div(cols, 16);
    if (o.dgamma && o.dbeta)
        col_sums_merge<<<dim3(blocks, 2), kThreads, 0, s>>>(o.part_g, o.part_b, o.slabs, cols, accumulate, o.dgamma,
                                                            o.dbeta);
    else if (o.dgamma)
        col_sums_merge<<<blocks, kThreads, 0, s>>>(o.part_g, nullptr, o.slabs, cols, accumulate, o.dgamma, nullptr);
    else
        col_sums_merge<<<blocks, kThreads, 0, s>>>(o.part_b, nullptr, o.slabs, cols, accumulate, o.dbeta, nullptr);
}

template <typename T, bool LN>
hipError_t launch_cols(const RmsBwdArgs& a, const Sums& o, const ColPlan& p, int accumulate, hipStream_t s) {
    col_sums<T, LN><<<dim3(p.gx, p.slabs), kThreads, 0, s>>>((const T*)a.dy, (const T*)a.h, a.mean, a.inv, a.rows,
                                                             a.cols, p.tx_log, p.slab_rows, o.part_g, o.part_b);
    launch_merge(o, a.cols, accumulate, s);
    return hipGetLastError();
}

template <typename T, bool LN> hipError_t launch_fwd(const RmsArgs& a, hipStream_t s) {
    const int blocks = rms_fwd_blocks(a.rows, a.cols);
    if (a.cols > kMaxRow) {
        rms_fwd_long<T, LN><<<blocks, 1024, 0, s>>>(a);
        return hipGetLastError();
    }
    CONVMI_RMS_SWITCH(a.cols, TPR, NV, {
        constexpr int threads = TPR > kThreads ? TPR : kThreads;
        rms_fwd<T, TPR, NV, LN><<<blocks, threads, 0, s>>>(a);
    });
    return hipGetLastError();
}

// Rows of the partial sums in the workspace.
int bwd_slabs(int64_t rows, int cols, bool ln) {
    return cols > kMaxRowBwd || rows == 0 ? col_plan(rows, cols).slabs : rms_bwd_blocks(rows, cols, ln);
}

template <typename T, bool LN>
hipError_t launch_bwd(RmsBwdArgs a, float* dgamma, float* dbeta, int accumulate, void* ws, hipStream_t s) {
    const bool held = a.cols <= kMaxRowBwd && a.rows > 0, sums = dgamma || dbeta;
    const int slabs = bwd_slabs(a.rows, a.cols, LN);
    const Sums o{dgamma, dbeta, (float*)ws, (float*)ws + (LN ? (int64_t)slabs * a.cols : 0), slabs};
    // The sums first where they have their own pass: dx may overwrite dy.
    if (sums && !held) {
        const hipError_t e = launch_cols<T, LN>(a, o, col_plan(a.rows, a.cols), accumulate, s);
        if (e != hipSuccess) return e;
    }
    if (a.rows == 0) return hipSuccess;
    const int blocks = rms_bwd_blocks(a.rows, a.cols, LN);
    if (!held) {
        rms_bwd_long<T, LN><<<blocks, 1024, 0, s>>>(a);
        return hipGetLastError();
    }
    a.part = !dgamma ? nullptr : blocks == 1 ? dgamma : o.part_g;
    a.part_b = !dbeta ? nullptr : blocks == 1 ? dbeta : o.part_b;
    a.add = blocks == 1 && accumulate;
    CONVMI_RMS_BWD_SWITCH(a.cols, TPR, NV, {
        constexpr int threads = TPR > kThreads ? TPR : kThreads;
        rms_bwd<T, TPR, NV, LN><<<blocks, threads, 0, s>>>(a);
    });
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && sums && blocks > 1) {
        launch_merge(o, a.cols, accumulate, s);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace

hipError_t launch_rms_fwd(int dt, const void* x, const void* residual, const float* gamma, void* h, void* y, void* y8,
                          void* y8_scales, float* inv_rms, int64_t rows, int cols, float eps, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    const RmsArgs a{x, residual, gamma, nullptr, h, y, (uint8_t*)y8, (uint8_t*)y8_scales, nullptr, inv_rms, rows, cols,
                    (int)ceil_div(cols, kMxBlock), eps};
    return dt == DT_BF16 ? launch_fwd<bf16, false>(a, s) : launch_fwd<float, false>(a, s);
}

size_t rms_bwd_ws_bytes(int64_t rows, int cols) {
    return align_up((size_t)bwd_slabs(rows, cols, false) * cols * sizeof(float), 256);
}

hipError_t launch_rms_bwd(int dt, const void* h, const float* gamma, const float* inv_rms, const void* dy,
                          const void* dh, void* dx, float* dgamma, int accumulate, int64_t rows, int cols, void* ws,
                          hipStream_t s) {
    const RmsBwdArgs a{h, gamma, nullptr, inv_rms, dy, dh, dx, nullptr, nullptr, 0, rows, cols};
    return dt == DT_BF16 ? launch_bwd<bf16, false>(a, dgamma, nullptr, accumulate, ws, s)
                         : launch_bwd<float, false>(a, dgamma, nullptr, accumulate, ws, s);
}

hipError_t launch_layer_norm_fwd(int dt, const void* x, const void* residual, const float* gamma, const float* beta,
                                 void* h, void* y, void* y8, void* y8_scales, float* mean, float* inv_std, int64_t rows,
                                 int cols, float eps, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    const RmsArgs a{x, residual, gamma, beta, h, y, (uint8_t*)y8, (uint8_t*)y8_scales, mean, inv_std, rows, cols,
                    (int)ceil_div(cols, kMxBlock), eps};
    return dt == DT_BF16 ? launch_fwd<bf16, true>(a, s) : launch_fwd<float, true>(a, s);
}

size_t layer_norm_bwd_ws_bytes(int64_t rows, int cols) {
    return align_up((size_t)bwd_slabs(rows, cols, true) * cols * 2 * sizeof(float), 256);
}

hipError_t launch_layer_norm_bwd(int dt, const void* h, const float* gamma, const float* mean, const float* inv_std,
                                 const void* dy, const void* dh, void* dx, float* dgamma, float* dbeta, int accumulate,
                                 int64_t rows, int cols, void* ws, hipStream_t s) {
    const RmsBwdArgs a{h, gamma, mean, inv_std, dy, dh, dx, nullptr, nullptr, 0, rows, cols};
    return dt == DT_BF16 ? launch_bwd<bf16, true>(a, dgamma, dbeta, accumulate, ws, s)
                         : launch_bwd<float, true>(a, dgamma, dbeta, accumulate, ws, s);
}

}  // namespace convmi
