// k_cconv.hip -- short causal convolution along the rows of each sequence, channel by channel.
//
//   forward   z_t = bias + sum_k w_k x_(t-W+1+k);  y = act(z)
//   backward  dz = act'(z) dy (z is formed again);  dx_t = sum_k w_k dz_(t+W-1-k)
//             dw_k = sum_t dz_t x_(t-W+1+k);  db = sum_t dz_t
//   one token z = bias + sum_k w_k s_k, s = (state, x);  state <- s without its first row
//
// What lies before a sequence's first row is its initial state (W-1 rows) or zero; its last W-1
// rows, the initial state's among them where it is shorter, are its final state.
//
// Bound by HBM: x is read and y (dx) written once, neighbouring threads' rows come from the cache.
// 6151 x 4096 bf16, four taps, SiLU, ragged: forward 23 us (4.3 TB/s, floor 20 at a copy's 5.0);
// 8192 x 4096 backward 51 us (3.9 TB/s, floor 40), of it the kernel 50 with the vector ALU busy three
// quarters of the time, the merge of dw and db 5 behind it.  Rows and columns beyond the edge are
// not skipped but clamped to ones that exist, so that the loops have no branches: with a second path at
// every load the forward took 31 us, the backward 80.  The backward forms z again from x rather
// than reading it: 2 W operations against 2 bytes.
#include "internal.hpp"
#include "seq.hpp"
#include "vec.hpp"

namespace convmi {
namespace {

constexpr int kThreads = 256;

// v <- act(v), or with SLOPE its derivative act'(v); the branch on act is the same for all lanes.
template <int ACT, bool SLOPE, int V> __device__ __forceinline__ void act_all(float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if constexpr (ACT == ACT_SILU) v[j] = SLOPE ? silu_slope(v[j]) : silu(v[j]);
        else v[j] = SLOPE ? act_slope<ACT>(v[j]) : act_fwd<ACT>(v[j]);
    }
}
template <bool SLOPE, int V> __device__ __forceinline__ void activate(int act, float (&v)[V]) {
    if (act == ACT_SILU) act_all<ACT_SILU, SLOPE, V>(v);
    else CONVMI_ACT_SWITCH(act, A, { act_all<A, SLOPE, V>(v); });
}

struct ConvArgs {
    Seqs q;
    const void *x, *w;
    const float* bias;    // nullable
    const void* initial;  // nullable [batch][W-1][D]
    int D, act, tx_log;   // threads of a workgroup side by side along the channels
    int64_t pitch;        // of x and dx
    // forward
    void *y, *final;      // final nullable
    int main_blocks;      // workgroups of the rows; those behind them write the final states
    // backward
    const void *dy, *dfinal;  // dfinal nullable
    void *dx, *dinitial;      // dinitial nullable
    float* part;              // [workgroups along the rows][D * (W + 1)]: dw, then db
    int run, col_blocks;      // rows a thread walks; workgroups side by side
};

// A thread's V channels begin at col and all exist: the last threads of a row step back and compute
// some channels twice, to the same values.  Rows of fewer than V channels take TAIL kernels, whose
// accesses stop after n.
template <int V, bool TAIL> struct Cols {
    int col, n;
    bool live;
    __device__ __forceinline__ Cols(int at, int D) : col(at), n(D - at), live(at < D) {
        if (!TAIL) {
            col = D - at < V ? D - V : at;
            n = V;
        }
    }
};

// The weights of a thread's V channels, w[d][k] at [k][d].
template <typename T, int W, int V> __device__ __forceinline__ void load_taps(const T* w, int col, int n, float (&k)[W][V]) {
    const T* p = w + (int64_t)col * W;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        float f[V];
        load_wide<T, V>(p + i * V, n * W - i * V, f);
#pragma unroll
        for (int j = 0; j < V; ++j) k[(i * V + j) % W][(i * V + j) / W] = f[j];
    }
}
// Row t of the initial state before sequence `seq`, t rows before its end (t = -1: the last).
template <typename T, int W, int V>
__device__ __forceinline__ Vec<T, V> state_row(const ConvArgs& a, int seq, int t, int col, int n) {
    const int64_t at = ((int64_t)seq * (W - 1) + (t + W - 1)) * a.D + col;
    if (!a.initial) return Vec<T, V>{};
    return load_vec<T, V>((const T*)a.initial + at, n);
}
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> conv_row(const ConvArgs& a, int t, int col, int n) {
    return load_vec<T, V>((const T*)a.x + (int64_t)t * a.pitch + col, n);
}
template <int W, int V>
__device__ __forceinline__ void conv_z(const float (&k)[W][V], const float (&b)[V], const float (&r)[V], int tap,
                                       float (&z)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = tap == 0 ? __builtin_fmaf(k[0][j], r[j], b[j]) : __builtin_fmaf(k[tap][j], r[j], z[j]);
}

// Final state of a sequence, of one channel a thread.
template <typename T> __device__ __forceinline__ void final_state(const ConvArgs& a, int W, int seq, int c) {
    if (c >= a.D) return;
    const int begin = seq_begin(a.q, seq), end = seq_end(a.q, seq, begin);
    for (int j = 0; j < W - 1; ++j) {
        const int t = end - (W - 1) + j;
        T v = 0;
        if (t >= begin) v = ((const T*)a.x)[(int64_t)t * a.pitch + c];
        else if (a.initial) v = ((const T*)a.initial)[((int64_t)seq * (W - 1) + (t - begin + W - 1)) * a.D + c];
        ((T*)a.final)[((int64_t)seq * (W - 1) + j) * a.D + c] = v;
    }
}
// The final states alone, where they take the initial ones' place: those must have been read.
template <typename T> __global__ __launch_bounds__(kThreads) void conv_final(ConvArgs a, int W) {
    const int blocks = (a.D + kThreads - 1) / kThreads;
    final_state<T>(a, W, blockIdx.x / blocks, (int)(blockIdx.x % blocks) * kThreads + threadIdx.x);
}

// A thread computes V channels of U consecutive rows, whose loads are all in flight at once.
template <typename T, int W, int U, int V, bool SILU, bool TAIL>
__global__ __launch_bounds__(kThreads) void conv_fwd(ConvArgs a) {
    if ((int)blockIdx.x >= a.main_blocks) {
        const int blocks = (a.D + kThreads - 1) / kThreads, b = blockIdx.x - a.main_blocks;
        final_state<T>(a, W, b / blocks, b % blocks * kThreads + threadIdx.x);
        return;
    }
    const int tx = 1 << a.tx_log, ty = kThreads >> a.tx_log, act = SILU ? ACT_SILU : a.act;
    const int cb = blockIdx.x % a.col_blocks, rb = blockIdx.x / a.col_blocks;
    const Cols<V, TAIL> c((cb * tx + (threadIdx.x & (tx - 1))) * V, a.D);
    int seq = wave_seq_of_row(a.q, rb * ty * U);
    if (!c.live) return;
    const int col = c.col, n = c.n;
    int t = (rb * ty + (threadIdx.x >> a.tx_log)) * U;
    const int last = t + U < a.q.rows ? t + U : a.q.rows;
    float k[W][V], b[V];
    load_taps<T, W, V>((const T*)a.w, col, n, k);
    load_wide<float, V>(a.bias + col, a.bias ? n : 0, b);
    if (seq < 0) seq = 0;
    for (; seq < a.q.batch && t < last; ++seq) {
        const int begin = seq_begin(a.q, seq), end = seq_end(a.q, seq, begin);
        if (t < begin) t = begin;
        const int stop = end < last ? end : last;
        if (t >= stop) continue;
        // rows of this run that lie in the sequence; the loads behind them repeat its last row
        Vec<T, V> raw[U + W - 1];
#pragma unroll
        for (int i = 0; i < U + W - 1; ++i) {
            const int r = t - (W - 1) + i;
            raw[i] = conv_row<T, V>(a, seq_clamp(r, begin, stop - 1), col, n);
        }
        if (t - (W - 1) < begin) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i)
                if (t - (W - 1) + i < begin) raw[i] = state_row<T, W, V>(a, seq, t - (W - 1) + i - begin, col, n);
        }
        float r[U + W - 1][V];
#pragma unroll
        for (int i = 0; i < U + W - 1; ++i) widen<T, V>(raw[i], r[i]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float z[V];
#pragma unroll
            for (int i = 0; i < W; ++i) conv_z<W, V>(k, b, r[u + i], i, z);
            activate<false, V>(act, z);
            if (t + u < stop) store_vec<T, V>((T*)a.y + (int64_t)(t + u) * a.D + col, n, z);
        }
        t = stop;
    }
}

// A thread walks `run` rows of V channels and W-1 rows beyond them, whose dz its last rows need.
// Rows t of a sequence keep their x and their unfinished dx in slot (t - first) % W of rings.
template <typename T, int W, int V, bool SILU, bool TAIL> __global__ __launch_bounds__(kThreads, 2) void conv_bwd(ConvArgs a) {
    constexpr int U = W < 3 ? 4 : W;  // rows whose loads are in flight together, a multiple of W
    __shared__ float cs[W + 1][kThreads * V];
    const int tx = 1 << a.tx_log, ty = kThreads >> a.tx_log, act = SILU ? ACT_SILU : a.act;
    const int cb = blockIdx.x % a.col_blocks, rb = blockIdx.x / a.col_blocks;
    const Cols<V, TAIL> c((cb * tx + (threadIdx.x & (tx - 1))) * V, a.D);
    const int col = c.col, n = c.n;
    int seq = wave_seq_of_row(a.q, rb * ty * a.run);
    if (seq < 0) seq = 0;
    int t = (rb * ty + (threadIdx.x >> a.tx_log)) * a.run;
    const int last = !c.live ? t : a.q.rows - t > a.run ? t + a.run : a.q.rows;
    float k[W][V], b[V], dw[W][V], db[V];
    if (c.live) {
        load_taps<T, W, V>((const T*)a.w, col, n, k);
        load_wide<float, V>(a.bias + col, a.bias ? n : 0, b);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        db[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) dw[i][j] = 0.0f;
    }
    for (; seq < a.q.batch && t < last; ++seq) {
        const int begin = seq_begin(a.q, seq), end = seq_end(a.q, seq, begin);
        if (t < begin) t = begin;
        const int first = t, stop = end < last ? end : last;
        if (first >= stop) continue;
        const int beyond = stop + W - 1;  // dz of rows end .. beyond - 1 is zero
        float x[W][V], acc[W][V];
        Vec<T, V> rx[U], ry[U];
        auto fetch = [&](int at) {  // rows behind the sequence repeat its last one
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = at + u < end ? at + u : end - 1;
                rx[u] = conv_row<T, V>(a, r, col, n);
                ry[u] = load_vec<T, V>((const T*)a.dy + (int64_t)r * a.D + col, n);
            }
        };
        {
            Vec<T, V> raw[W];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                const int r = first - (W - 1) + i;
                raw[i] = conv_row<T, V>(a, r < begin ? begin : r, col, n);
            }
            fetch(first);
            if (first - (W - 1) < begin) {
#pragma unroll
                for (int i = 0; i < W - 1; ++i)
                    if (first - (W - 1) + i < begin)
                        raw[i] = state_row<T, W, V>(a, seq, first - (W - 1) + i - begin, col, n);
            }
#pragma unroll
            for (int i = 0; i < W - 1; ++i) widen<T, V>(raw[i], x[(i + 1) % W]);
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) acc[i][j] = 0.0f;
        for (; t < beyond; t += U) {
            Vec<T, V> cx[U], cy[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                cx[u] = rx[u];
                cy[u] = ry[u];
            }
            fetch(t + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int now = t + u, s = u % W;
                float z[V], d[V];
                widen<T, V>(cx[u], x[s]);
                widen<T, V>(cy[u], d);
#pragma unroll
                for (int i = 0; i < W; ++i) conv_z<W, V>(k, b, x[(s + 1 + i) % W], i, z);
                activate<true, V>(act, z);
#pragma unroll
                for (int j = 0; j < V; ++j) d[j] = now < end ? d[j] * z[j] : 0.0f;
#pragma unroll
                for (int i = 0; i < W; ++i)  // row now - (W-1) + i took tap i's product with x of that row
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float& o = acc[(s + 1 + i) % W][j];
                        o = i == W - 1 ? k[i][j] * d[j] : __builtin_fmaf(k[i][j], d[j], o);
                    }
                if (now < stop) {  // each row counts in one run, none behind the end: 0 times its x may be no 0
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        db[j] += d[j];
#pragma unroll
                        for (int i = 0; i < W; ++i) dw[i][j] = __builtin_fmaf(d[j], x[(s + 1 + i) % W][j], dw[i][j]);
                    }
                }
                const int done = now - (W - 1);  // has met all its taps
                float(&o)[V] = acc[(s + 1) % W];
                if (done >= first && done < stop) {
                    if (a.dfinal && done >= end - (W - 1)) {
                        float f[V];
                        load_wide<T, V>((const T*)a.dfinal + ((int64_t)seq * (W - 1) + done - (end - (W - 1))) * a.D + col, n, f);
#pragma unroll
                        for (int j = 0; j < V; ++j) o[j] += f[j];
                    }
                    store_vec<T, V>((T*)a.dx + (int64_t)done * a.pitch + col, n, o);
                }
            }
        }
        t = stop;
    }
    // the workgroup's row groups, in order
    if (!a.part) return;
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int i = 0; i < W; ++i) cs[i][threadIdx.x * V + j] = dw[i][j];
        cs[W][threadIdx.x * V + j] = db[j];
    }
    __syncthreads();
    const int64_t DW = (int64_t)a.D * W;
    float* part = a.part + (int64_t)rb * (DW + a.D);
    for (int e = threadIdx.x; e < tx * V; e += kThreads) {
        const Cols<V, TAIL> at((cb * tx + e / V) * V, a.D);
        const int d = at.col + e % V;
        if (!at.live || d >= a.D) continue;
#pragma unroll
        for (int i = 0; i <= W; ++i) {
            float s = 0.0f;
            for (int g = 0; g < ty; ++g) s += cs[i][g * tx * V + e];
            part[i < W ? (int64_t)d * W + i : DW + d] = s;
        }
    }
}

// Gradient of the initial states: row q of W-1 lies W-1-q rows before the sequence.
template <typename T, int W> __global__ __launch_bounds__(kThreads) void conv_dinitial(ConvArgs a) {
    const int seq = blockIdx.x / a.col_blocks, c = blockIdx.x % a.col_blocks * kThreads + threadIdx.x;
    if (c >= a.D) return;
    const int begin = seq_begin(a.q, seq), end = seq_end(a.q, seq, begin);
    float k[W], o[W], x[2 * W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        k[i] = to_f32(((const T*)a.w)[(int64_t)c * W + i]);
        o[i] = 0.0f;
    }
    const float bias = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * W - 2; ++i) {
        const int t = begin - (W - 1) + i;
        float v[1] = {0.0f};
        if (t < begin) v[0] = a.initial ? to_f32(((const T*)a.initial)[((int64_t)seq * (W - 1) + i) * a.D + c]) : 0.0f;
        else if (t < end) v[0] = to_f32(((const T*)a.x)[(int64_t)t * a.pitch + c]);
        x[i] = v[0];
    }
#pragma unroll
    for (int m = 0; m < W - 1; ++m) {
        if (begin + m >= end) break;
        float z[1] = {bias};
#pragma unroll
        for (int i = 0; i < W; ++i) z[0] = __builtin_fmaf(k[i], x[m + i], z[0]);
        activate<true, 1>(a.act, z);
        const float d = z[0] * to_f32(((const T*)a.dy)[(int64_t)(begin + m) * a.D + c]);
#pragma unroll
        for (int q = m; q < W - 1; ++q) o[q] = __builtin_fmaf(k[q - m], d, o[q]);  // its tap q - m
    }
#pragma unroll
    for (int q = 0; q < W - 1; ++q) {
        const int j = begin + q - end;  // its row of the final state, where the sequence is that short
        if (a.dfinal && j >= 0) o[q] += to_f32(((const T*)a.dfinal)[((int64_t)seq * (W - 1) + j) * a.D + c]);
        ((T*)a.dinitial)[((int64_t)seq * (W - 1) + q) * a.D + c] = from_f32<T>(o[q]);
    }
}

// dw, db (+)= sums over the partial rows, in fp64 and in order.
__global__ __launch_bounds__(kThreads) void conv_merge(const float* __restrict__ part, int slabs, int64_t DW, int D,
                                                       int accumulate, float* __restrict__ dw, float* __restrict__ db) {
    constexpr int G = 16, U = 8;
    __shared__ double cs[G][kThreads / G];
    const int x = threadIdx.x % (kThreads / G), y = threadIdx.x / (kThreads / G);
    const int64_t c = (int64_t)blockIdx.x * (kThreads / G) + x, width = DW + D;
    double s = 0.0;
    if (c < width) {
        int k = y;
        for (; k + G * (U - 1) < slabs; k += G * U) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = part[(k + G * u) * width + c];
#pragma unroll
            for (int u = 0; u < U; ++u) s += (double)v[u];
        }
        for (; k < slabs; k += G) s += (double)part[k * width + c];
    }
    cs[y][x] = s;
    __syncthreads();
    if (y != 0 || c >= width) return;
    for (int g = 1; g < G; ++g) s += cs[g][x];
    float* out = c < DW ? (dw ? dw + c : nullptr) : (db ? db + (c - DW) : nullptr);
    if (out) *out = accumulate ? (float)((double)*out + s) : (float)s;
}

// One token of each row's sequence: the state of its slot is used and moved by one row.  Everything
// is loaded before the slot is known to be the row's own.
template <typename T, int W, int V, bool TAIL> __global__ __launch_bounds__(kThreads) void conv_step(ConvArgs a, Slots sl) {
    const int row = blockIdx.x / a.col_blocks;
    const Cols<V, TAIL> c((blockIdx.x % a.col_blocks * kThreads + threadIdx.x) * V, a.D);
    const int col = c.col, n = c.live ? c.n : 0;
    const int slot = slot_of(sl, row);
    T* state = (T*)a.final + (int64_t)slot * (W - 1) * a.D + col;
    Vec<T, V> raw[W];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) raw[i] = load_vec<T, V>(state + (int64_t)i * a.D, slot >= 0 ? n : 0);
    raw[W - 1] = load_vec<T, V>((const T*)a.x + (int64_t)row * a.pitch + col, n);
    float k[W][V], b[V];
    load_taps<T, W, V>((const T*)a.w, col, n, k);
    load_wide<float, V>(a.bias + col, a.bias ? n : 0, b);
    const bool bad = slot_taken(sl, row, slot);
    if (slot == kSlotNone || !c.live) return;
    float z[V];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        float r[V];
        widen<T, V>(raw[i], r);
        conv_z<W, V>(k, b, r, i, z);
        if (i > 0 && !bad) store_vec<T, V>(state + (int64_t)(i - 1) * a.D, n, r);
    }
    activate<false, V>(a.act, z);
    if (bad) {
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] = __uint_as_float(0x7fc00000u);
    }
    store_vec<T, V>((T*)a.y + (int64_t)row * a.D + col, n, z);
}

#define CONVMI_TAPS_SWITCH(taps, W, ...)                          \
    switch (taps) {                                               \
    case 1: { constexpr int W = 1; __VA_ARGS__; } break;          \
    case 2: { constexpr int W = 2; __VA_ARGS__; } break;          \
    case 3: { constexpr int W = 3; __VA_ARGS__; } break;          \
    case 4: { constexpr int W = 4; __VA_ARGS__; } break;          \
    case 5: { constexpr int W = 5; __VA_ARGS__; } break;          \
    case 6: { constexpr int W = 6; __VA_ARGS__; } break;          \
    case 7: { constexpr int W = 7; __VA_ARGS__; } break;          \
    default: { constexpr int W = 8; __VA_ARGS__; } break;         \
    }

// Eight rows a thread keep eleven loads in flight and read 3 / 8 of the rows twice, from the cache.
// Channels a thread holds: 16 bytes of them in the forward; in the backward as many as leave room for
// three waves a SIMD beside the rings, weights and sums (8192 x 4096 bf16, four taps: four
// channels 50 us, eight, with one or two waves, 79 and 88).
template <typename T> constexpr int fwd_vec() { return 16 / sizeof(T); }
constexpr int bwd_vec(int W) { return W <= 6 ? 4 : 2; }
constexpr int kFwdRows = 8;

int tx_log_for(int D, int V) {
    int l = 0;
    while (l < 6 && (V << l) < D) ++l;
    return l;
}

struct FwdPlan {
    int tx_log, col_blocks;
    int64_t blocks;
};
template <typename T> FwdPlan fwd_plan(int64_t rows, int D) {
    FwdPlan p;
    p.tx_log = tx_log_for(D, fwd_vec<T>());
    p.col_blocks = (int)ceil_div(D, fwd_vec<T>() << p.tx_log);
    p.blocks = ceil_div(rows, (kThreads >> p.tx_log) * kFwdRows) * p.col_blocks;
    return p;
}
struct BwdPlan {
    int tx_log, col_blocks, run, row_blocks;
};
// Runs as long as leave some 512 workgroups: the rows beyond a run are read twice, and each
// workgroup along the rows leaves a row of partial sums (8192 x 4096 bf16: 54 us in 256, 50 in
// 512, 52 in 768, 56 in 1024, 68 in 4096).
BwdPlan bwd_plan(int64_t rows, int D, int taps) {
    const int V = bwd_vec(taps);
    BwdPlan p;
    p.tx_log = tx_log_for(D, V);
    p.col_blocks = (int)ceil_div(D, V << p.tx_log);
    const int ty = kThreads >> p.tx_log;
    int64_t run = ceil_div(rows, ceil_div(512, p.col_blocks) * ty);
    if (run < 4) run = 4;
    if (run > 256) run = 256;
    p.run = (int)run;
    p.row_blocks = (int)ceil_div(rows, run * ty);
    return p;
}

ConvArgs conv_args(const CausalConvDims& d) {
    ConvArgs a{};
    a.q = d.q;
    a.x = d.x;
    a.w = d.w;
    a.bias = d.bias;
    a.initial = d.initial;
    a.D = d.D;
    a.act = d.act;
    a.pitch = d.pitch;
    return a;
}

template <typename T> hipError_t fwd(const CausalConvDims& d, void* y, void* final, hipStream_t s) {
    ConvArgs a = conv_args(d);
    a.y = y;
    a.final = final;
    constexpr int V = fwd_vec<T>(), U = kFwdRows;
    const FwdPlan p = fwd_plan<T>(d.q.rows, d.D);
    a.tx_log = p.tx_log;
    a.col_blocks = p.col_blocks;
    const int64_t states = final && d.taps > 1 ? d.q.batch * ceil_div(d.D, kThreads) : 0;
    const bool apart = states > 0 && final == d.initial;
    a.main_blocks = (int)p.blocks;
    const unsigned blocks = (unsigned)(p.blocks + (apart ? 0 : states));
    if (blocks > 0) {
        CONVMI_TAPS_SWITCH(d.taps, W, {
            if (d.D < V) conv_fwd<T, W, U, V, false, true><<<blocks, kThreads, 0, s>>>(a);
            else if (d.act == ACT_SILU) conv_fwd<T, W, U, V, true, false><<<blocks, kThreads, 0, s>>>(a);
            else conv_fwd<T, W, U, V, false, false><<<blocks, kThreads, 0, s>>>(a);
        });
    }
    if (apart) conv_final<T><<<(unsigned)states, kThreads, 0, s>>>(a, d.taps);
    return hipGetLastError();
}

template <typename T>
hipError_t bwd(const CausalConvDims& d, const void* dy, const void* dfinal, void* dx, void* dinitial, float* dw,
               float* db, int accumulate, void* ws, hipStream_t s) {
    ConvArgs a = conv_args(d);
    a.dy = dy;
    a.dfinal = dfinal;
    a.dx = dx;
    a.dinitial = dinitial;
    const bool sums = dw || db;
    if (dinitial && d.taps > 1 && d.q.batch > 0) {
        a.col_blocks = (int)ceil_div(d.D, kThreads);
        CONVMI_TAPS_SWITCH(d.taps, W, {
            conv_dinitial<T, W><<<(unsigned)((int64_t)d.q.batch * a.col_blocks), kThreads, 0, s>>>(a);
        });
    }
    int slabs = 0;
    if (d.q.rows > 0) {
        const BwdPlan p = bwd_plan(d.q.rows, d.D, d.taps);
        a.part = sums ? (float*)ws : nullptr;
        a.tx_log = p.tx_log;
        a.run = p.run;
        a.col_blocks = p.col_blocks;
        slabs = p.row_blocks;
        CONVMI_TAPS_SWITCH(d.taps, W, {
            constexpr int V = bwd_vec(W);
            const unsigned blocks = (unsigned)((int64_t)p.row_blocks * p.col_blocks);
            if (d.D < V) conv_bwd<T, W, V, false, true><<<blocks, kThreads, 0, s>>>(a);
            else if (d.act == ACT_SILU) conv_bwd<T, W, V, true, false><<<blocks, kThreads, 0, s>>>(a);
            else conv_bwd<T, W, V, false, false><<<blocks, kThreads, 0, s>>>(a);
        });
    }
    if (sums) {
        const int64_t DW = (int64_t)d.D * d.taps;
        conv_merge<<<(unsigned)ceil_div(DW + d.D, 16), kThreads, 0, s>>>((const float*)ws, slabs, DW, d.D, accumulate,
                                                                         dw, db);
    }
    return hipGetLastError();
}

template <typename T> hipError_t step(const CausalConvDims& d, const Slots& sl, void* state, void* y, hipStream_t s) {
    if (d.q.rows == 0) return hipSuccess;
    ConvArgs a = conv_args(d);
    a.y = y;
    a.final = state;
    constexpr int V = 16 / sizeof(T);
    a.col_blocks = (int)ceil_div(d.D, kThreads * V);
    CONVMI_TAPS_SWITCH(d.taps, W, {
        const unsigned blocks = (unsigned)((int64_t)d.q.rows * a.col_blocks);
        // no channel twice: its state is moved in place
        if (d.D % V) conv_step<T, W, V, true><<<blocks, kThreads, 0, s>>>(a, sl);
        else conv_step<T, W, V, false><<<blocks, kThreads, 0, s>>>(a, sl);
    });
    return hipGetLastError();
}

}  // namespace

bool causal_conv_fits(int64_t rows, int64_t batch, int D, int taps, int dtype) {
    const FwdPlan f = dtype == DT_BF16 ? fwd_plan<bf16>(rows, D) : fwd_plan<float>(rows, D);
    const BwdPlan b = bwd_plan(rows, D, taps);
    return grid_fits(f.blocks + batch * ceil_div(D, kThreads), kThreads) &&
           grid_fits((int64_t)b.row_blocks * b.col_blocks, kThreads);
}
bool causal_conv_step_fits(int64_t rows, int D, int dtype) {
    return grid_fits(rows * ceil_div(D, kThreads * (16 / (int)dtype_size(dtype))), kThreads);
}
size_t causal_conv_ws_bytes(int64_t rows, int D, int taps) {
    if (rows == 0) return 0;
    return align_up((size_t)bwd_plan(rows, D, taps).row_blocks * D * (taps + 1) * sizeof(float), 256);
}

hipError_t launch_causal_conv_fwd(const CausalConvDims& d, void* y, void* final, hipStream_t s) {
    return d.dtype == DT_BF16 ? fwd<bf16>(d, y, final, s) : fwd<float>(d, y, final, s);
}

hipError_t launch_causal_conv_bwd(const CausalConvDims& d, const void* dy, const void* dfinal, void* dx, void* dinitial,
                                  float* dw, float* db, int accumulate, void* ws, hipStream_t s) {
    return d.dtype == DT_BF16 ? bwd<bf16>(d, dy, dfinal, dx, dinitial, dw, db, accumulate, ws, s)
                              : bwd<float>(d, dy, dfinal, dx, dinitial, dw, db, accumulate, ws, s);
}

hipError_t launch_causal_conv_step(const CausalConvDims& d, const Slots& sl, void* state, void* y, hipStream_t s) {
    return d.dtype == DT_BF16 ? step<bf16>(d, sl, state, y, s) : step<float>(d, sl, state, y, s);
}

}  // namespace convmi
