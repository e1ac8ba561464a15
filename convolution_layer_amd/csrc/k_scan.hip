// k_scan.hip -- selective state space scan along sequences: forward, backward, single tokens.
//
//   v = dt + dt_bias;  delta = softplus(v) (or v)
//   h_t[d,n] = a h_(t-1)[d,n] + delta x B_t[n],  a = exp(delta A[d,n])
//   y_t[d] = (sum_n C_t[n] h_t[d,n] + D x) silu(z)
// and back, with dy' = dy silu(z) and G the gradient that comes from later rows:
//   g = C_t dy' + G;  G <- a g
//   dC_t[n] = sum_d dy' h_t;  dB_t[n] = sum_d delta x g;  s = sum_n B_t g;  w = sum_n A G h_(t-1)
//   dA[d,n] = sum_t delta G h_(t-1);  dx = delta s + D dy';  ddelta = x s + w
//
// A channel belongs to eight lanes, each holding S states in registers; a workgroup of eight waves
// takes 64 channels of a chunk of one sequence, tile by tile: all threads bring a tile of rows
// into LDS (delta, delta x, B, C in fp32), each wave runs its 8 channels through the rows, all
// threads finish and write the outputs.  Rows behind a sequence's end count as delta = 0 and
// B = C = 0, which leaves the state as it is.
//
// Bound by the vector ALU: every h takes an exponential and four operations forward (and two and a half
// times that backward), against 8 bytes a channel and row of bf16.  A wave-wide operation takes a
// SIMD 1.9 ns, an exponential 4.0, a swap of halves 4.5 with four waves on it, 2.1, 4.6 and 5.5 with
// two, 2.6, 6.9 and 10.6 with one: hence eight lanes a channel, which give each of 1024 SIMDs two
// waves from 4 x 4096 channels (four lanes, one wave: forward 243 us, backward 839, eight: 203 and
// 642 at that stage).  Now 8192 x 4096 bf16, 16 states, four sequences:
// forward 194 us, backward 555 (vector ALU busy some 80 and 87 %), sums 13.  Sums over lanes go through
// folds that halve the number of values at each step instead of repeating every sum in every lane.
#include <cfloat>

#include "internal.hpp"
#include "seq.hpp"
#include "vec.hpp"

namespace convmi {
namespace {

constexpr int kCh = 64, kQ = 8, kThreads = kCh * kQ;  // channels of a workgroup, lanes of a channel
constexpr int kTile = 32;                             // rows of a tile
constexpr int kV = kTile * kCh / kThreads;            // channels of a thread while a tile is loaded or finished
constexpr int kSmall = 256;                           // threads of the other kernels' workgroups
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The backward's tile; rows between two kept states; rows of which a lane holds h and a.
constexpr int seg_rows(int S) { return S <= 4 ? kTile : kTile / 2; }
constexpr int keep_rows(int S) { return S == 4 ? 32 : 16; }
constexpr int sub_rows(int S) { return S <= 2 ? 16 : S == 4 ? 8 : 4; }

template <int CTRL> __device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// Sums of four values over four lanes: lane q gets the sum of y[q].  The first step adds lanes 1,0,3,2, the
// second lanes 2,3,0,1.
__device__ __forceinline__ float quad_sums(const float (&y)[4], int q) {
    const bool odd = q & 1, high = q & 2;
    const float a = (odd ? y[1] : y[0]) + dpp<0xB1>(odd ? y[0] : y[1]);
    const float c = (odd ? y[3] : y[2]) + dpp<0xB1>(odd ? y[2] : y[3]);
    return (high ? c : a) + dpp<0x4E>(high ? a : c);
}
// Sums of eight values over the eight lanes of a channel: lane q gets the sum of y[q].  Lanes q
// and 7 - q meet first, each keeping four of the values, then the lanes of a quad.
__device__ __forceinline__ float oct_sums(const float (&y)[8], int q) {
    const bool high = q & 4;
    float a[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) a[m] = (high ? y[m + 4] : y[m]) + dpp<0x141>(high ? y[m] : y[m + 4]);
    return quad_sums(a, q & 3);
}
__device__ __forceinline__ const float (&first4(const float (&y)[8]))[4] { return *(const float(*)[4])y; }
// Halves of the wave: lanes 0-31 get the sum over lanes l, l+32 of a, the others that of b.
__device__ __forceinline__ float fold32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// The same within each half: 16-lane rows 0 and 2 get a's sums, rows 1 and 3 b's.
__device__ __forceinline__ float fold16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// exp2 is the hardware's (off by one step at most), of a product with log2 e rounded into A.
// log(1 + e) for e in [0, 1]: e times a polynomial of degree 8 fitted to log1p(e) / e at
// Chebyshev nodes (relative error 3.1e-8, with its roundings 3 * 2^-24).
__device__ __forceinline__ float log1p_unit(float e) {
    float p = 0.005253457929939032f;
    p = __builtin_fmaf(p, e, -0.02958850748836994f);
    p = __builtin_fmaf(p, e, 0.07836166769266129f);
    p = __builtin_fmaf(p, e, -0.13674770295619965f);
    p = __builtin_fmaf(p, e, 0.19111430644989014f);
    p = __builtin_fmaf(p, e, -0.24844369292259216f);
    p = __builtin_fmaf(p, e, 0.33319270610809326f);
    p = __builtin_fmaf(p, e, -0.49999502301216125f);
    p = __builtin_fmaf(p, e, 1.0f);
    return p * e;
}
// log(1 + exp(v)), and its derivative 1 / (1 + exp(-v)).
__device__ __forceinline__ float softplus(float v) {
    return __builtin_fmaxf(v, 0.0f) + log1p_unit(__builtin_amdgcn_exp2f(__builtin_fabsf(v) * -kLog2e));
}

// v <- delta of v + bias, 0 behind the end.
__device__ __forceinline__ void steps(float (&v)[kV], const float (&bias)[kV], int plus, bool in) {
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] += bias[j];
    if (plus) {
#pragma unroll
        for (int j = 0; j < kV; ++j) v[j] = softplus(v[j]);
    }
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] = in ? v[j] : 0.0f;
}

struct ScanArgs {
    Seqs q;
    const void *x, *dt, *B, *C, *z;     // z nullable
    const float *dt_bias, *A, *D;       // dt_bias, D nullable
    const float* initial;               // nullable
    int ch, N, cpg, col_blocks;         // channels, states, channels of a group, workgroups of a group's channels
    int softplus;
    int64_t xp, dtp, zp, bcp;           // pitches
    int chunk, slots;                   // rows of a chunk, chunk slots
    int paired;                         // how local and decay are numbered, see Place::home
    float *local, *decay;               // per chunk: state from zero [ch][N], sum of delta [ch]
    // forward
    void* y;
    float *final, *saved;               // nullable
    // backward
    const float* kept;                  // the forward's saved
    const void* dy;
    const float* dfinal;                // nullable
    void *dx, *ddt, *dz;                // dz with z
    float* dinitial;                    // nullable
    int per;                            // chunk slots of a workgroup
    float *part_p, *part_bc;            // partial sums of dA, dD, ddt_bias per `per` slots; of dB, dC per workgroup column
};

// What a workgroup works on: 64 channels from c0 on (live of them), rows [row, stop) of sequence seq.
struct Place {
    int seq, begin, end, k, row, stop, slot, home, group, c0, live;
    bool some, last;  // there is such a chunk; it is its sequence's last
};
// Chunk k of sequence i has slot begin_i / chunk + i + k: the sequences' slots do not meet, and
// a slot tells its sequence without a list.  Its place in local and decay is home + k: home is the slot
// of the sequence's chunk 0 or, where that leaves most places to sequences of one chunk (which need
// none), 2 floor(begin_i / chunk) (`paired`).  Then sequences of several chunks do not meet either: one of
// length l > chunk has ceil(l / chunk) <= 2 floor(l / chunk) of them, and floor(begin / chunk) + floor(l /
// chunk) is at most the floor of where it ends, so that 2 floor(rows / chunk) places hold all.
__device__ __forceinline__ Place place_of(const ScanArgs& a, int cb, int slot) {
    Place p;
    p.slot = slot;
    p.group = cb / a.col_blocks;
    const int in = cb % a.col_blocks * kCh;
    p.c0 = p.group * a.cpg + in;
    p.live = a.cpg - in < kCh ? a.cpg - in : kCh;
    p.seq = wave_last(a.q.batch, [&](int i) { return seq_begin(a.q, i) / a.chunk + i <= p.slot; });
    p.some = p.seq >= 0;
    if (!p.some) return p;
    p.begin = seq_begin(a.q, p.seq);
    p.end = seq_end(a.q, p.seq, p.begin);
    const int before = p.begin / a.chunk;
    p.home = a.paired ? 2 * before : before + p.seq;
    p.k = p.slot - before - p.seq;
    const int64_t off = (int64_t)p.k * a.chunk;
    p.some = p.k >= 0 && (p.k == 0 || off < p.end - p.begin);
    if (!p.some) return p;
    p.row = p.begin + (int)off;
    p.stop = p.end - p.row > a.chunk ? p.row + a.chunk : p.end;
    p.last = p.stop == p.end;
    return p;
}

// S states of a lane, n0 on, of [N] values at p; 0 behind the last, and in all where not live.
template <int S> __device__ __forceinline__ void load_states(const float* p, int n0, int N, bool live, float (&v)[S]) {
    if constexpr (S > 1) {
        load_wide<float, S>(p + n0, live ? N - n0 : 0, v);
    } else {
        v[0] = live && n0 < N ? p[n0] : 0.0f;
    }
}
template <int S> __device__ __forceinline__ void store_states(float* p, int n0, int N, const float (&v)[S]) {
    if constexpr (S > 1) {
        if (n0 < N) store_vec<float, S>(p + n0, N - n0, v);
    } else {
        if (n0 < N) p[n0] = v[0];
    }
}

// The same of B or C, in the data type.
template <typename T, int S> __device__ __forceinline__ void load_bc(const T* p, int n0, int N, float (&v)[S]) {
    if constexpr (S > 1) load_wide<T, S>(p + n0, N - n0, v);
    else v[0] = n0 < N ? to_f32(p[n0]) : 0.0f;
}

// B and C of a tile of TT rows, W = kQ S values each, read into registers and put into LDS in fp32, the S
// values of B and of C that a lane needs side by side.
template <typename T, int TT, int S> struct TileBC {
    static constexpr int W = kQ * S, PER = (TT * W + kThreads - 1) / kThreads;
    T b[PER], c[PER];
    __device__ __forceinline__ void load(const ScanArgs& a, const Place& p, int row, int stop) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * kThreads + threadIdx.x, t = row + e / W, n = e % W;
            const bool in = e < TT * W && t < stop && n < a.N;
            const int64_t at = (int64_t)t * a.bcp + (int64_t)p.group * a.N + n;
            b[i] = in ? ((const T*)a.B)[at] : (T)0;
            c[i] = in ? ((const T*)a.C)[at] : (T)0;
        }
    }
    __device__ __forceinline__ void put(float (*bc)[kQ][2][S]) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * kThreads + threadIdx.x, n = e % W;
            if (e < TT * W) {
                bc[e / W][n / S][0][n % S] = to_f32(b[i]);
                bc[e / W][n / S][1][n % S] = to_f32(c[i]);
            }
        }
    }
};

template <int S> __device__ __forceinline__ void load_A2(const ScanArgs& a, int c, int n0, bool live, float (&A2)[S]) {
    load_states<S>(a.A + (int64_t)c * a.N, n0, a.N, live, A2);
#pragma unroll
    for (int j = 0; j < S; ++j) {
        A2[j] *= kLog2e;
        A2[j] = A2[j] < -FLT_MAX ? -FLT_MAX : A2[j] > FLT_MAX ? FLT_MAX : A2[j];  // 0 times it is 0 where no row is
    }
}

// 2^x v + l.  The whole part of x goes into v's exponent, so that a factor beyond fp32 neither makes a
// NaN of v = 0 nor loses a product that lies inside; beyond 2^+-400 every product is infinite or 0.
__device__ __forceinline__ float scaled_add(float x, float v, float l) {
    x = __builtin_amdgcn_fmed3f(x, -400.0f, 400.0f);  // finite where x is NaN: then l is NaN too
    const float n = __builtin_floorf(x);
    return __builtin_fmaf(__builtin_amdgcn_exp2f(x - n), __builtin_ldexpf(v, (int)n), l);
}

// v brought through the chunks at from, from + step .. before to: v <- decay v + what the chunk adds,
// the loads of eight chunks in flight.
template <int S>
__device__ __forceinline__ void through(const ScanArgs& a, int from, int to, int step, int c, int n0, bool live,
                                        const float (&A2)[S], float (&v)[S]) {
    constexpr int B = 8;
    for (int k = from; k != to;) {
        float l[B][S], sum[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const bool in = live && (step > 0 ? k + i < to : k - i > to);
            const int64_t at = (int64_t)(k + i * step) * a.ch + c;
            load_states<S>(a.local + at * a.N, n0, a.N, in, l[i]);
            sum[i] = in ? a.decay[at] : 0.0f;  // behind the last: exp(0) v + 0
        }
#pragma unroll
        for (int i = 0; i < B; ++i)
#pragma unroll
            for (int j = 0; j < S; ++j) v[j] = scaled_add(A2[j] * sum[i], v[j], l[i][j]);
        const int left = step > 0 ? to - k : k - to;
        k = left > B ? k + B * step : to;
    }
}

// ---------------------------------------------------------------- forward
// LOCAL: only the state that the chunk leaves behind from zero and its sum of delta.
template <typename T, int S, bool LOCAL>
__device__ __forceinline__ void scan_chunk(const ScanArgs& a, const Place& p, float2 (&dd)[kTile][kCh],
                                           float (&lbc)[kTile][kQ][2][S], float (&ly)[kTile][kCh + 4]) {
    constexpr int TT = kTile, KEEP = keep_rows(S);
    const int q = threadIdx.x % kQ, lch = threadIdx.x / kQ;
    const int c = p.c0 + lch, n0 = q * S;
    const bool live = lch < p.live;
    const int tr = threadIdx.x / (kCh / kV), tc = threadIdx.x % (kCh / kV) * kV, tn = p.live - tc;
    float A2[S], h[S], sum = 0.0f;
    load_A2<S>(a, c, n0, live, A2);
    if constexpr (LOCAL) {
#pragma unroll
        for (int j = 0; j < S; ++j) h[j] = 0.0f;
    } else if (p.k == 0) {
        load_states<S>(a.initial + ((int64_t)p.seq * a.ch + c) * a.N, n0, a.N, live && a.initial, h);
    } else {  // the first chunk left its state whole
        load_states<S>(a.local + ((int64_t)p.home * a.ch + c) * a.N, n0, a.N, live, h);
        through<S>(a, p.home + 1, p.home + p.k, 1, c, n0, live, A2, h);
    }
    float bias[kV], skip[kV];
    load_wide<float, kV>(a.dt_bias + p.c0 + tc, a.dt_bias ? tn : 0, bias);
    load_wide<float, kV>(a.D + p.c0 + tc, a.D && !LOCAL ? tn : 0, skip);
    Vec<T, kV> rx, rd, rz;
    TileBC<T, TT, S> bc;
    auto fetch = [&](int row) {
        const int t = row + tr, n = t < p.stop ? tn : 0;
        rx = load_vec<T, kV>((const T*)a.x + (int64_t)t * a.xp + p.c0 + tc, n);
        rd = load_vec<T, kV>((const T*)a.dt + (int64_t)t * a.dtp + p.c0 + tc, n);
        if (!LOCAL) rz = load_vec<T, kV>((const T*)a.z + (int64_t)t * a.zp + p.c0 + tc, a.z ? n : 0);
        bc.load(a, p, row, p.stop);
    };
    fetch(p.row);
    for (int row = p.row; row < p.stop; row += TT) {
        float x[kV], z[kV];
        widen<T, kV>(rx, x);
        {
            float d[kV];
            widen<T, kV>(rd, d);
            steps(d, bias, a.softplus, row + tr < p.stop);
#pragma unroll
            for (int j = 0; j < kV; ++j) dd[tr][tc + j] = make_float2(d[j], d[j] * x[j]);
        }
        if (!LOCAL) widen<T, kV>(rz, z);
        bc.put(lbc);
        __syncthreads();
        if (row + TT < p.stop) fetch(row + TT);
#pragma unroll
        for (int t0 = 0; t0 < TT; t0 += 8) {
            if (!LOCAL && t0 % KEEP == 0 && a.saved && live && row + t0 < p.stop) {
                const int64_t at = (int64_t)(p.begin / KEEP + p.seq + (row + t0 - p.begin) / KEEP) * a.ch + c;
                store_states<S>(a.saved + at * a.N, n0, a.N, h);
            }
            float y[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float2 v = dd[t0 + u][lch];
                y[u] = 0.0f;
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    const float e = __builtin_amdgcn_exp2f(v.x * A2[j]);
                    h[j] = __builtin_fmaf(e, h[j], v.y * lbc[t0 + u][q][0][j]);
                    if (!LOCAL) y[u] = __builtin_fmaf(lbc[t0 + u][q][1][j], h[j], y[u]);
                }
                if (LOCAL) sum += v.x;
            }
            if (!LOCAL) ly[t0 + q][lch] = oct_sums(y, q);
        }
        __syncthreads();
        if (!LOCAL && row + tr < p.stop && tn > 0) {
            float o[kV];
#pragma unroll
            for (int j = 0; j < kV; ++j) o[j] = __builtin_fmaf(skip[j], x[j], ly[tr][tc + j]);
            if (a.z) {
#pragma unroll
                for (int j = 0; j < kV; ++j) o[j] *= silu(z[j]);
            }
            store_vec<T, kV>((T*)a.y + (int64_t)(row + tr) * a.ch + p.c0 + tc, tn, o);
        }
    }
    if (!live) return;
    const int64_t at = (int64_t)(p.home + p.k) * a.ch + c;
    if (LOCAL || (p.k == 0 && !p.last)) store_states<S>(a.local + at * a.N, n0, a.N, h);
    else if (a.final && p.last) store_states<S>(a.final + ((int64_t)p.seq * a.ch + c) * a.N, n0, a.N, h);
    if (LOCAL && q == 0) a.decay[at] = sum;
}
// Sequences in one chunk each, or the two passes over several: the first takes the chunks that sequences
// begin with whole, from the initial state, and leaves the others' LOCAL ones; the second takes the
// others whole.  Only first chunks read the initial state, so the final one may take its place.
constexpr int kWhole = 0, kFirst = 1, kSecond = 2;
template <typename T, int S, int PASS> __global__ __launch_bounds__(kThreads) void scan_fwd(ScanArgs a) {
    __shared__ float2 dd[kTile][kCh];  // delta, delta x
    __shared__ __align__(16) float lbc[kTile][kQ][2][S];
    __shared__ float ly[kTile][kCh + 4];  // sum_n C h; the pad spreads a channel's rows over the banks
    const int cols = a.ch / a.cpg * a.col_blocks;
    const Place p = place_of(a, blockIdx.x % cols, blockIdx.x / cols);
    if (!p.some || (PASS == kSecond && p.k == 0)) return;
    if (PASS != kFirst || p.k == 0) scan_chunk<T, S, false>(a, p, dd, lbc, ly);
    else if (!p.last) scan_chunk<T, S, true>(a, p, dd, lbc, ly);
}

// ---------------------------------------------------------------- backward
// The gradient that a chunk hands to the one before it, from zero, and its sum of delta.
template <typename T, int S> __global__ __launch_bounds__(kThreads) void scan_bwd_local(ScanArgs a) {
    constexpr int TT = kTile;
    __shared__ float2 dd[TT][kCh];  // delta, dy'
    __shared__ __align__(16) float lbc[TT][kQ][2][S];
    const int cols = a.ch / a.cpg * a.col_blocks;
    const Place p = place_of(a, blockIdx.x % cols, blockIdx.x / cols);
    if (!p.some || p.k == 0) return;
    const int q = threadIdx.x % kQ, lch = threadIdx.x / kQ;
    const int c = p.c0 + lch, n0 = q * S;
    const bool live = lch < p.live;
    const int tr = threadIdx.x / (kCh / kV), tc = threadIdx.x % (kCh / kV) * kV, tn = p.live - tc;
    float A2[S], G[S], sum = 0.0f;
    load_A2<S>(a, c, n0, live, A2);
#pragma unroll
    for (int j = 0; j < S; ++j) G[j] = 0.0f;
    float bias[kV];
    load_wide<float, kV>(a.dt_bias + p.c0 + tc, a.dt_bias ? tn : 0, bias);
    Vec<T, kV> ry, rd, rz;
    TileBC<T, TT, S> bc;
    auto fetch = [&](int row) {
        const int t = row + tr, n = t < p.stop ? tn : 0;
        rd = load_vec<T, kV>((const T*)a.dt + (int64_t)t * a.dtp + p.c0 + tc, n);
        ry = load_vec<T, kV>((const T*)a.dy + (int64_t)t * a.ch + p.c0 + tc, n);
        rz = load_vec<T, kV>((const T*)a.z + (int64_t)t * a.zp + p.c0 + tc, a.z ? n : 0);
        bc.load(a, p, row, p.stop);
    };
    int row = p.row + (p.stop - p.row - 1) / TT * TT;
    fetch(row);
    for (; row >= p.row; row -= TT) {
        float d[kV], y[kV], z[kV];
        widen<T, kV>(rd, d);
        widen<T, kV>(ry, y);
        widen<T, kV>(rz, z);
        steps(d, bias, a.softplus, row + tr < p.stop);
        if (a.z) {
#pragma unroll
            for (int j = 0; j < kV; ++j) y[j] *= silu(z[j]);
        }
#pragma unroll
        for (int j = 0; j < kV; ++j) dd[tr][tc + j] = make_float2(d[j], y[j]);
        bc.put(lbc);
        __syncthreads();
        if (row > p.row) fetch(row - TT);
#pragma unroll 8
        for (int t = TT - 1; t >= 0; --t) {
            const float2 v = dd[t][lch];
#pragma unroll
            for (int j = 0; j < S; ++j)
                G[j] = __builtin_amdgcn_exp2f(v.x * A2[j]) * __builtin_fmaf(lbc[t][q][1][j], v.y, G[j]);
            sum += v.x;
        }
        __syncthreads();
    }
    if (!live) return;
    const int64_t at = (int64_t)(p.home + p.k) * a.ch + c;
    store_states<S>(a.local + at * a.N, n0, a.N, G);
    if (q == 0) a.decay[at] = sum;
}

__device__ __forceinline__ void put3(float4& o, float x, float y, float z) {
    o.x = x;
    o.y = y;
    o.z = z;
}
// The whole backward of `per` chunk slots, of each chunk from its last tile to its first.  Each sub of a tile, from the last
// on, runs forward from its first state with h and a in registers, then back.  With 16 states and
// fewer that state was kept by the forward (8192 x 4096, 16 states, forward and backward: 753 us;
// one kept every 32 rows, half of each tile run through twice, 793); beyond, the subs between two
// kept states are run through once before.
template <typename T, int S> __global__ __launch_bounds__(kThreads, 1) void scan_bwd(ScanArgs a) {
    constexpr int SEG = seg_rows(S), SUB = sub_rows(S), K = SEG / SUB, W = kQ * S, NW = kThreads / 64;
    constexpr int KEEP = keep_rows(S), KT = SEG / KEEP, KS = KEEP / SUB;  // kept states of a tile, subs of one
    constexpr int R = SUB < 8 ? SUB : 8;  // rows whose sums over lanes are taken together
    __shared__ float4 dd[SEG][kCh + 1];    // delta, delta x, dy', delta; then s, w, sum_n C h in the first; padded as ly
    __shared__ __align__(16) float lbc[SEG][kQ][2][S];
    __shared__ float bcs[NW][SEG][2 * W];  // each wave's sums for dB and dC
    const int cols = a.ch / a.cpg * a.col_blocks, part_row = blockIdx.x / cols;
    Place p = place_of(a, blockIdx.x % cols, part_row * a.per);
    const int64_t wide = (int64_t)a.ch * (a.N + 2);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = threadIdx.x % kQ, lch = threadIdx.x / kQ;
    const int c = p.c0 + lch, n0 = q * S;
    const bool live = lch < p.live;
    const int tr = threadIdx.x / (kCh / kV), tc = threadIdx.x % (kCh / kV) * kV, tn = tr < SEG ? p.live - tc : 0;
    float* part = a.part_p + part_row * wide;
    float dA[S], dD[kV], db[kV];
#pragma unroll
    for (int j = 0; j < S; ++j) dA[j] = 0.0f;
#pragma unroll
    for (int j = 0; j < kV; ++j) dD[j] = db[j] = 0.0f;
    const int behind_slot = (part_row + 1) * a.per < a.slots ? (part_row + 1) * a.per : a.slots;
    for (int slot = part_row * a.per; slot < behind_slot; ++slot) {
        if (slot != part_row * a.per) p = place_of(a, blockIdx.x % cols, slot);
        if (!p.some) continue;
        float A2[S], G[S];
        load_A2<S>(a, c, n0, live, A2);
        // what comes from behind the sequence, brought back through the chunks behind this one
        load_states<S>(a.dfinal + ((int64_t)p.seq * a.ch + c) * a.N, n0, a.N, live && a.dfinal, G);
        const int behind = p.end > p.begin ? (p.end - p.begin - 1) / a.chunk : 0;
        through<S>(a, p.home + behind, p.home + p.k, -1, c, n0, live, A2, G);
        float bias[kV], skip[kV];
        load_wide<float, kV>(a.dt_bias + p.c0 + tc, a.dt_bias ? tn : 0, bias);
        load_wide<float, kV>(a.D + p.c0 + tc, a.D ? tn : 0, skip);
        Vec<T, kV> rx, rd, rz, ry;
        TileBC<T, SEG, S> bc;
        float h0[KT][S];
        auto fetch = [&](int row) {
            const int t = row + tr, n = t < p.stop ? tn : 0;
            rx = load_vec<T, kV>((const T*)a.x + (int64_t)t * a.xp + p.c0 + tc, n);
            rd = load_vec<T, kV>((const T*)a.dt + (int64_t)t * a.dtp + p.c0 + tc, n);
            rz = load_vec<T, kV>((const T*)a.z + (int64_t)t * a.zp + p.c0 + tc, a.z ? n : 0);
            ry = load_vec<T, kV>((const T*)a.dy + (int64_t)t * a.ch + p.c0 + tc, n);
            bc.load(a, p, row, p.stop);
            const int64_t at = (int64_t)(p.begin / KEEP + p.seq + (row - p.begin) / KEEP) * a.ch + c;
#pragma unroll
            for (int i = 0; i < KT; ++i)
                load_states<S>(a.kept + (at + (int64_t)i * a.ch) * a.N, n0, a.N, live && row + i * KEEP < p.stop, h0[i]);
        };
        int row = p.row + (p.stop - p.row - 1) / SEG * SEG;
        if (p.stop > p.row) fetch(row);
        for (; p.stop > p.row && row >= p.row; row -= SEG) {
            const bool in = row + tr < p.stop;
            const Vec<T, kV> cx = rx, cd = rd, cz = rz, cy = ry;
            float hk[K][S];  // states at the subs' starts
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int j = 0; j < S; ++j) hk[i * KS][j] = h0[i][j];
            if (tr < SEG) {
                float x[kV], d[kV], z[kV], y[kV];
                widen<T, kV>(cx, x);
                widen<T, kV>(cd, d);
                widen<T, kV>(cz, z);
                widen<T, kV>(cy, y);
                steps(d, bias, a.softplus, in);
                if (a.z) {
#pragma unroll
                    for (int j = 0; j < kV; ++j) y[j] *= silu(z[j]);
                }
#pragma unroll
                for (int j = 0; j < kV; ++j) dd[tr][tc + j] = make_float4(d[j], d[j] * x[j], y[j], d[j]);
            }
            bc.put(lbc);
            __syncthreads();
            if (row > p.row) fetch(row - SEG);
#pragma unroll
            for (int k = 0; k < K - 1; ++k) {
                if ((k + 1) % KS == 0) continue;  // the next one's state was kept
                float h[S];
#pragma unroll
                for (int j = 0; j < S; ++j) h[j] = hk[k][j];
#pragma unroll
                for (int t = k * SUB; t < (k + 1) * SUB; ++t) {
                    const float4 v = dd[t][lch];
#pragma unroll
                    for (int j = 0; j < S; ++j)
                        h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(v.x * A2[j]), h[j], v.y * lbc[t][q][0][j]);
                }
#pragma unroll
                for (int j = 0; j < S; ++j) hk[k + 1][j] = h[j];
            }
            float dAs[S];
#pragma unroll
            for (int j = 0; j < S; ++j) dAs[j] = 0.0f;
#pragma unroll 1
            for (int k = K - 1; k >= 0; --k) {
                float ha[SUB + 1][S], ea[SUB][S];  // ha[i + 1]: h of the sub's row i
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    ha[0][j] = hk[0][j];
#pragma unroll
                    for (int m = 1; m < K; ++m) ha[0][j] = k == m ? hk[m][j] : ha[0][j];
                }
#pragma unroll
                for (int i = 0; i < SUB; ++i) {
                    const float4 v = dd[k * SUB + i][lch];
#pragma unroll
                    for (int j = 0; j < S; ++j) {
                        ea[i][j] = __builtin_amdgcn_exp2f(v.x * A2[j]);
                        ha[i + 1][j] = __builtin_fmaf(ea[i][j], ha[i][j], v.y * lbc[k * SUB + i][q][0][j]);
                    }
                }
#pragma unroll
                for (int i0 = SUB - R; i0 >= 0; i0 -= R) {
                    const int t0 = k * SUB + i0;
                    float s[8], w[8], yn[8], r[R][S];
#pragma unroll
                    for (int i = R - 1; i >= 0; --i) {
                        const float4 v = dd[t0 + i][lch];
                        s[i] = w[i] = yn[i] = 0.0f;
#pragma unroll
                        for (int j = 0; j < S; ++j) {
                            const float b = lbc[t0 + i][q][0][j], cc = lbc[t0 + i][q][1][j], hj = ha[i0 + i + 1][j];
                            const float g = __builtin_fmaf(cc, v.z, G[j]);
                            r[i][j] = fold32(v.y * g, v.z * hj);  // dB's terms in lanes 0-31, dC's in the others
                            s[i] = __builtin_fmaf(b, g, s[i]);
                            yn[i] = __builtin_fmaf(cc, hj, yn[i]);
                            G[j] = ea[i0 + i][j] * g;
                            const float f = G[j] * ha[i0 + i][j];
                            dAs[j] = __builtin_fmaf(v.x, f, dAs[j]);
                            w[i] = __builtin_fmaf(A2[j], f, w[i]);
                        }
                    }
                    if constexpr (R == 8) {
                        put3(dd[t0 + q][lch], oct_sums(s, q), oct_sums(w, q), oct_sums(yn, q));
                    } else {  // lanes q and 7 - q together, then the quad; both quads write the same
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            s[i] += dpp<0x141>(s[i]);
                            w[i] += dpp<0x141>(w[i]);
                            yn[i] += dpp<0x141>(yn[i]);
                        }
                        const int e = q & 3;
                        put3(dd[t0 + e][lch], quad_sums(first4(s), e), quad_sums(first4(w), e), quad_sums(first4(yn), e));
                    }
                    // over the wave's 8 channels: 16-lane rows hold two states (or rows t), eight lanes of a
                    // row and the other eight end with the same sums and write one of two each
                    constexpr int M = R * S / 2;
                    auto over_channels = [&](int m) {
                        float f;
                        if constexpr (S > 1) f = fold16(r[2 * m / S][2 * m % S], r[2 * m / S][2 * m % S + 1]);
                        else f = fold16(r[2 * m][0], r[2 * m + 1][0]);
                        return f + dpp<0x128>(f);
                    };
                    const int odd = lane >> 4 & 1, eight = lane >> 3 & 1;
#pragma unroll
                    for (int e = 0; e < M / 2; ++e) {
                        const float lo = over_channels(2 * e), hi = over_channels(2 * e + 1);
                        const int m = 2 * e + eight;
                        const int tt = S > 1 ? 2 * m / S : 2 * m + odd, n = S > 1 ? n0 + 2 * m % S + odd : n0;
                        bcs[wave][t0 + tt][(lane >> 5) * W + n] = eight ? hi : lo;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < S; ++j) dA[j] += dAs[j];
            __syncthreads();
            if (in && tn > 0) {
                float x[kV], d[kV], z[kV], y[kV], ox[kV], od[kV], oz[kV];
                widen<T, kV>(cx, x);
                widen<T, kV>(cd, d);
                widen<T, kV>(cz, z);
                widen<T, kV>(cy, y);
#pragma unroll
                for (int j = 0; j < kV; ++j) oz[j] = __builtin_fmaf(skip[j], x[j], dd[tr][tc + j].z);
                if (a.z) {
#pragma unroll
                    for (int j = 0; j < kV; ++j) {
                        float m;
                        const float g = both_sigmoids(z[j], m);
                        oz[j] *= y[j] * __builtin_fmaf(z[j] * m, g, g);
                        y[j] *= z[j] * g;
                    }
                }
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const float4 v = dd[tr][tc + j];
                    od[j] = __builtin_fmaf(x[j], v.x, v.y * kLn2);
                    ox[j] = v.w * v.x;
                }
                if (a.softplus) {
#pragma unroll
                    for (int j = 0; j < kV; ++j) {
                        float m;
                        od[j] *= both_sigmoids(d[j] + bias[j], m);
                    }
                }
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    ox[j] = __builtin_fmaf(skip[j], y[j], ox[j]);
                    dD[j] = __builtin_fmaf(y[j], x[j], dD[j]);
                    db[j] += od[j];
                }
                const int64_t t = row + tr;
                store_vec<T, kV>((T*)a.dx + t * a.xp + p.c0 + tc, tn, ox);
                store_vec<T, kV>((T*)a.ddt + t * a.dtp + p.c0 + tc, tn, od);
                if (a.z) store_vec<T, kV>((T*)a.dz + t * a.zp + p.c0 + tc, tn, oz);
            }
            // [workgroup column][row][group][dB, dC][N]
            const int groups = a.ch / a.cpg;
            const int64_t col = (p.c0 - p.group * a.cpg) / kCh;
            for (int e = threadIdx.x; e < SEG * 2 * W; e += kThreads) {
                const int t = e / (2 * W), m = e % (2 * W), n = m % W;
                if (row + t >= p.stop || n >= a.N) continue;
                float s = 0.0f;
#pragma unroll
                for (int v = 0; v < NW; ++v) s += bcs[v][t][m];
                a.part_bc[((col * a.q.rows + row + t) * groups + p.group) * 2 * a.N + m / W * a.N + n] = s;
            }
            __syncthreads();
        }
        if (a.dinitial && p.k == 0 && live) store_states<S>(a.dinitial + ((int64_t)p.seq * a.ch + c) * a.N, n0, a.N, G);
    }
    // these slots' shares of dA, dD and ddt_bias (zeros from slots without a chunk)
    if (live) store_states<S>(part + (int64_t)c * a.N, n0, a.N, dA);
    float* sums = (float*)dd;  // [2][rows of threads][64]
    constexpr int TR = kThreads / (kCh / kV);
    static_assert(sizeof(dd) >= 2 * TR * kCh * sizeof(float), "the sums of the rows of threads fit");
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        sums[tr * kCh + tc + j] = dD[j];
        sums[(TR + tr) * kCh + tc + j] = db[j];
    }
    __syncthreads();
    if (threadIdx.x < 2 * kCh) {
        const int which = threadIdx.x / kCh, ch = threadIdx.x % kCh;
        float s = 0.0f;
        for (int r = 0; r < TR; ++r) s += sums[(which * TR + r) * kCh + ch];
        if (ch < p.live) part[(int64_t)a.ch * a.N + (int64_t)which * a.ch + p.c0 + ch] = s;
    }
}

// The first workgroups: dB, dC of a row each wave at a time, the sums over the workgroup columns.  The others:
// dA, dD, ddt_bias (+)= sums over the rows of partial sums, in fp64 and in order; each output may be null.
struct MergeArgs {
    Seqs q;
    const float *part_bc, *part_p;
    int row_blocks, cols, G, N, ch, parts, accumulate;
    int64_t bcp;
    void *dB, *dC;
    float *dA, *dD, *db;
};
template <typename T> __global__ __launch_bounds__(kSmall) void scan_merge(MergeArgs a) {
    if ((int)blockIdx.x < a.row_blocks) {
        for (int row = blockIdx.x * (kSmall / 64) + (threadIdx.x >> 6); row < a.q.rows; row += a.row_blocks * (kSmall / 64)) {
            const int seq = wave_seq_of_row(a.q, row);
            if (seq < 0 || row < seq_begin(a.q, seq) || row >= seq_end(a.q, seq, seq_begin(a.q, seq))) continue;
            const int wide = 2 * a.G * a.N;
            for (int e = threadIdx.x & 63; e < wide; e += 64) {
                float s = 0.0f;
#pragma unroll 8
                for (int k = 0; k < a.cols; ++k) s += a.part_bc[((int64_t)k * a.q.rows + row) * wide + e];
                const int n = e % a.N, which = e / a.N % 2, g = e / (2 * a.N);
                ((T*)(which ? a.dC : a.dB))[row * a.bcp + g * a.N + n] = from_f32<T>(s);
            }
        }
        return;
    }
    const int64_t wide = (int64_t)a.ch * (a.N + 2), i = (int64_t)(blockIdx.x - a.row_blocks) * kSmall + threadIdx.x;
    if (i >= wide) return;
    const int64_t nA = (int64_t)a.ch * a.N, in = i - nA;
    float* out = i < nA ? a.dA + i : in < a.ch ? a.dD + in : a.db + (in - a.ch);
    if (!(i < nA ? a.dA : in < a.ch ? a.dD : a.db)) return;
    double s = 0.0;
#pragma unroll 8
    for (int k = 0; k < a.parts; ++k) s += (double)a.part_p[k * wide + i];
    *out = a.accumulate ? (float)((double)*out + s) : (float)s;
}

// ---------------------------------------------------------------- single tokens
// Four lanes a channel, 16 bytes of 16 states each, and four rows: lane q brings in and finishes row q's
// delta, gate and y of its channel, all four lanes run all rows' states.  Everything is loaded
// before a slot is known to be its row's own.  4096 channels, 16 states, bf16: 64, 128 and 256 rows
// take 12.3, 18.6 and 32 us, some 6 us of launch and latency and then 4.5-5.4 TB/s; one row a
// workgroup, every lane with its own delta and gate, takes as long for 64.
template <typename T, int S> __global__ __launch_bounds__(kSmall) void scan_step(ScanArgs a, Slots sl) {
    constexpr int R = 4;
    __shared__ int flags;
    const int groups = a.ch / a.cpg, cols = groups * a.col_blocks;
    const int row0 = blockIdx.x / cols * R, cb = blockIdx.x % cols, group = cb / a.col_blocks;
    const int in = cb % a.col_blocks * kCh + (threadIdx.x >> 2), c = group * a.cpg + in;
    const int q = threadIdx.x & 3, n0 = q * S, row = row0 + q;
    const bool mine = in < a.cpg, here = mine && row < a.q.rows;
    int slot[R];
    float h[R][S], A2[S];
#pragma unroll
    for (int r = 0; r < R; ++r) slot[r] = row0 + r < a.q.rows ? slot_of(sl, row0 + r) : kSlotNone;
#pragma unroll
    for (int r = 0; r < R; ++r)
        load_states<S>(a.final + ((int64_t)slot[r] * a.ch + c) * a.N, n0, a.N, mine && slot[r] >= 0, h[r]);
    float x = 0.0f, d = 0.0f, z = 0.0f, skip = 0.0f;
    if (here) {
        x = to_f32(((const T*)a.x)[row * a.xp + c]);
        d = to_f32(((const T*)a.dt)[row * a.dtp + c]);
        if (a.z) z = to_f32(((const T*)a.z)[row * a.zp + c]);
        if (a.dt_bias) d += a.dt_bias[c];
        if (a.D) skip = a.D[c];
    }
    load_A2<S>(a, c, n0, mine, A2);
    float b[R][S], cc[R][S];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t at = (int64_t)(row0 + r) * a.bcp + (int64_t)group * a.N;
        const int n = row0 + r < a.q.rows ? a.N : 0;
        load_bc<T, S>((const T*)a.B + at, n0, n, b[r]);
        load_bc<T, S>((const T*)a.C + at, n0, n, cc[r]);
    }
    const int bad = slots_taken<R>(sl, row0, slot, &flags);
    if (a.softplus) d = softplus(d);
    const float dx = d * x;
    float y[R];
    auto one = [&](int r, float dr, float dxr) {
        y[r] = 0.0f;
#pragma unroll
        for (int j = 0; j < S; ++j) {
            h[r][j] = __builtin_fmaf(__builtin_amdgcn_exp2f(dr * A2[j]), h[r][j], dxr * b[r][j]);
            y[r] = __builtin_fmaf(cc[r][j], h[r][j], y[r]);
        }
        if (mine && slot[r] >= 0 && !(bad >> r & 1))
            store_states<S>(a.final + ((int64_t)slot[r] * a.ch + c) * a.N, n0, a.N, h[r]);
    };
    one(0, dpp<0x00>(d), dpp<0x00>(dx));  // the values of a quad's lane 0, 1, 2, 3
    one(1, dpp<0x55>(d), dpp<0x55>(dx));
    one(2, dpp<0xAA>(d), dpp<0xAA>(dx));
    one(3, dpp<0xFF>(d), dpp<0xFF>(dx));
    float o = __builtin_fmaf(skip, x, quad_sums(y, q));
    if (a.z) o *= silu(z);
    const int my = q & 2 ? (q & 1 ? slot[3] : slot[2]) : (q & 1 ? slot[1] : slot[0]);
    if (!here || my == kSlotNone) return;
    ((T*)a.y)[(int64_t)row * a.ch + c] = from_f32<T>(bad >> q & 1 ? __uint_as_float(0x7fc00000u) : o);
}

// ---------------------------------------------------------------- host side
#define CONVMI_STATES_SWITCH(N, S, ...)                           \
    do {                                                          \
        if ((N) <= kQ) { constexpr int S = 1; __VA_ARGS__; }          \
        else if ((N) <= 2 * kQ) { constexpr int S = 2; __VA_ARGS__; } \
        else if ((N) <= 4 * kQ) { constexpr int S = 4; __VA_ARGS__; } \
        else { constexpr int S = 8; __VA_ARGS__; }                    \
    } while (0)

int keep_of(int N) {
    int r = 0;
    CONVMI_STATES_SWITCH(N, S, { r = keep_rows(S); });
    return r;
}

// Rows of a chunk.  One pass over whole sequences where they and the channels give five of eight CUs a
// workgroup; else chunks, which cost a pass more for the states between them (8192 x 4096 bf16, 64
// workgroups a sequence, forward and backward: two sequences 361 + 1099 us whole, 257 + 736 in chunks;
// three 252 + 748 and 260 + 725; four 200 + 570 and 239 + 717).  Sequences whose lengths only the
// device knows may be one long one and run in chunks wherever one would: equal ones that fill the chip pay
// for it when they are given by starts (those four by whole calls: 220 + 721 us against 189 + 561).
// Some 1536 workgroups, twice as many as fit at once in the forward (three a CU by 74-78 registers), six
// times in the backward (one a CU by 253), even out chunks of unequal length (6151 x 4096 in five sequences: 203 + 586 us
// in 512, 200 + 567 in 1024, 190 + 570 in 1536, 196 + 566 in 2048, 204 + 601 in 4096; one of 2048 x 2048 backward
// 114, 127, 126, 158, 159), down to one tile a chunk (701 x 134 fp32: backward 18 us in chunks of 64
// rows, 12 in 32).  Up to two tiles run whole: two launches fewer (64 x 512, forward and backward,
// eager: 46.7 -> 39 us; 100 rows whole 57).
struct ChunkPlan {
    int chunk, slots, cols;  // rows of a chunk; chunk slots; workgroups of all channels
    bool split;              // a sequence may have several chunks
    bool paired;             // places of the chunks' states, Place::home; `places` of them
    int places;
};
ChunkPlan chunk_plan(int64_t rows, int64_t batch, int ch, int G, bool ragged) {
    ChunkPlan p;
    p.cols = (int)(G * ceil_div(ch / G, kCh));
    const int64_t known = ragged ? 1 : batch, one = rows > 0 ? rows : 1;
    int64_t chunk = one;
    if (known * p.cols < 160 && ceil_div(one, known > 0 ? known : 1) > 2 * kTile) {
        const int64_t parts = ceil_div(1536, known * p.cols);
        chunk = ceil_div(ceil_div(rows, known), parts);
        if (chunk > one) chunk = one;
    }
    p.chunk = (int)align_up(chunk, kTile);
    p.slots = (int)(rows / p.chunk + batch);
    p.split = p.chunk < (ragged || batch == 0 ? rows : rows / batch);
    p.paired = p.slots > 2 * (rows / p.chunk);
    p.places = !p.split ? 0 : p.paired ? (int)(2 * (rows / p.chunk)) : p.slots;
    return p;
}
struct ScanWs {
    size_t local, decay, part_p, part_bc, total;
    int per, parts;  // chunk slots of a workgroup of the backward, rows of part_p
};
ScanWs scan_ws(const ScanDims& d, bool ragged, bool backward) {
    ScanWs w{};
    const ChunkPlan p = chunk_plan(d.q.rows, d.q.batch, d.ch, d.G, ragged);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t r = at;
        at += align_up(bytes, 256);
        return r;
    };
    w.local = take((size_t)p.places * d.ch * d.N * 4);
    w.decay = take((size_t)p.places * d.ch * 4);
    if (backward) {
        // some 2048 workgroups or 64 rows of partial sums are enough, however many sequences there are
        const int64_t most = ceil_div(2048, p.cols) > 64 ? ceil_div(2048, p.cols) : 64;
        w.per = (int)(p.slots > most ? ceil_div(p.slots, most) : 1);
        w.parts = (int)ceil_div(p.slots, w.per);
        w.part_p = take((size_t)w.parts * d.ch * (d.N + 2) * 4);
        w.part_bc = take((size_t)ceil_div(d.ch / d.G, kCh) * d.q.rows * 2 * d.G * d.N * 4);
    }
    w.total = at;
    return w;
}

ScanArgs scan_args(const ScanDims& d, const ChunkPlan& p, const ScanWs& w, void* ws) {
    ScanArgs a{};
    a.q = d.q;
    a.x = d.x; a.dt = d.dt; a.B = d.B; a.C = d.C; a.z = d.z;
    a.dt_bias = d.dt_bias; a.A = d.A; a.D = d.D;
    a.initial = d.initial;
    a.ch = d.ch;
    a.N = d.N;
    a.cpg = d.ch / d.G;
    a.col_blocks = (int)ceil_div(a.cpg, kCh);
    a.softplus = d.softplus;
    a.xp = d.xp; a.dtp = d.dtp; a.zp = d.zp; a.bcp = d.bcp;
    a.chunk = p.chunk;
    a.slots = p.slots;
    a.paired = p.paired;
    a.per = w.per;
    a.local = (float*)((char*)ws + w.local);
    a.decay = (float*)((char*)ws + w.decay);
    a.part_p = (float*)((char*)ws + w.part_p);
    a.part_bc = (float*)((char*)ws + w.part_bc);
    return a;
}

template <typename T> hipError_t fwd(const ScanDims& d, void* y, float* final, float* saved, void* ws, hipStream_t s) {
    const ChunkPlan p = chunk_plan(d.q.rows, d.q.batch, d.ch, d.G, d.q.starts != nullptr);
    ScanArgs a = scan_args(d, p, scan_ws(d, d.q.starts != nullptr, false), ws);
    a.y = y;
    a.final = final;
    a.saved = saved;
    const unsigned blocks = (unsigned)((int64_t)p.slots * p.cols);
    if (blocks == 0) return hipSuccess;
    CONVMI_STATES_SWITCH(d.N, S, {
        if (p.split) {
            scan_fwd<T, S, kFirst><<<blocks, kThreads, 0, s>>>(a);
            scan_fwd<T, S, kSecond><<<blocks, kThreads, 0, s>>>(a);
        } else {
            scan_fwd<T, S, kWhole><<<blocks, kThreads, 0, s>>>(a);
        }
    });
    return hipGetLastError();
}

// A wave takes one row up to 2^22 rows, several beyond, so that the launch fits whatever the rows.
int merge_row_blocks(int64_t rows) {
    const int64_t most = 1 << 20, need = ceil_div(rows, kSmall / 64);
    return (int)(need < most ? need : most);
}
template <typename T> hipError_t bwd(const ScanDims& d, const ScanGrads& g, void* ws, hipStream_t s) {
    const ChunkPlan p = chunk_plan(d.q.rows, d.q.batch, d.ch, d.G, d.q.starts != nullptr);
    const ScanWs w = scan_ws(d, d.q.starts != nullptr, true);
    ScanArgs a = scan_args(d, p, w, ws);
    a.kept = g.saved;
    a.dy = g.dy;
    a.dfinal = g.dfinal;
    a.dx = g.dx; a.ddt = g.ddt; a.dz = g.dz;
    a.dinitial = g.dinitial;
    const unsigned blocks = (unsigned)((int64_t)p.slots * p.cols);
    if (blocks > 0) {
        CONVMI_STATES_SWITCH(d.N, S, {
            if (p.split) scan_bwd_local<T, S><<<blocks, kThreads, 0, s>>>(a);
            scan_bwd<T, S><<<(unsigned)((int64_t)w.parts * p.cols), kThreads, 0, s>>>(a);
        });
    }
    const int row_blocks = merge_row_blocks(d.q.rows);
    const int64_t sums = g.dA || g.dD || g.ddt_bias ? ceil_div((int64_t)d.ch * (d.N + 2), kSmall) : 0;
    if (row_blocks + sums > 0) {
        const MergeArgs m{d.q, a.part_bc, a.part_p, row_blocks, a.col_blocks, d.G, d.N, d.ch, w.parts, g.accumulate,
                          d.bcp, g.dB, g.dC, g.dA, g.dD, g.ddt_bias};
        scan_merge<T><<<(unsigned)(row_blocks + sums), kSmall, 0, s>>>(m);
    }
    return hipGetLastError();
}

template <typename T> hipError_t step(const ScanDims& d, const Slots& sl, float* state, void* y, hipStream_t s) {
    if (d.q.rows == 0) return hipSuccess;
    ScanArgs a = scan_args(d, ChunkPlan{1, 0, 0, false, false, 0}, ScanWs{}, nullptr);
    a.final = state;
    a.y = y;
    const unsigned blocks = (unsigned)(ceil_div(d.q.rows, 4) * d.G * a.col_blocks);
    if (d.N <= 4) scan_step<T, 1><<<blocks, kSmall, 0, s>>>(a, sl);
    else if (d.N <= 8) scan_step<T, 2><<<blocks, kSmall, 0, s>>>(a, sl);
    else if (d.N <= 16) scan_step<T, 4><<<blocks, kSmall, 0, s>>>(a, sl);
    else if (d.N <= 32) scan_step<T, 8><<<blocks, kSmall, 0, s>>>(a, sl);
    else scan_step<T, 16><<<blocks, kSmall, 0, s>>>(a, sl);
    return hipGetLastError();
}

}  // namespace

bool scan_step_fits(const ScanDims& d) {
    return grid_fits(ceil_div(d.q.rows, 4) * d.G * ceil_div(d.ch / d.G, kCh), kSmall);
}
bool scan_fits(const ScanDims& d) {
    for (const bool ragged : {false, true}) {
        const ChunkPlan p = chunk_plan(d.q.rows, d.q.batch, d.ch, d.G, ragged);
        if (!grid_fits((int64_t)p.slots * p.cols, kThreads)) return false;
    }
    return grid_fits(merge_row_blocks(d.q.rows) + ceil_div((int64_t)d.ch * (d.N + 2), kSmall), kSmall);
}
size_t scan_saved_bytes(const ScanDims& d) {
    return ((size_t)(d.q.rows / keep_of(d.N)) + d.q.batch) * d.ch * d.N * sizeof(float);
}
size_t scan_ws_bytes(const ScanDims& d, bool backward) {
    const size_t even = scan_ws(d, false, backward).total, ragged = scan_ws(d, true, backward).total;
    return even > ragged ? even : ragged;
}
hipError_t launch_scan_fwd(const ScanDims& d, void* y, float* final, float* saved, void* ws, hipStream_t s) {
    return d.dtype == DT_BF16 ? fwd<bf16>(d, y, final, saved, ws, s) : fwd<float>(d, y, final, saved, ws, s);
}
hipError_t launch_scan_bwd(const ScanDims& d, const ScanGrads& g, void* ws, hipStream_t s) {
    return d.dtype == DT_BF16 ? bwd<bf16>(d, g, ws, s) : bwd<float>(d, g, ws, s);
}
hipError_t launch_scan_step(const ScanDims& d, const Slots& sl, float* state, void* y, hipStream_t s) {
    return d.dtype == DT_BF16 ? step<bf16>(d, sl, state, y, s) : step<float>(d, sl, state, y, s);
}

}  // namespace convmi
