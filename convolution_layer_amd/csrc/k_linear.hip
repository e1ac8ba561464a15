// k_linear.hip -- matrix products of the linear layer on gfx950 MFMA.
//
//   forward   z[m][n]  = sum_k x[m][k] w[n][k] + bias[n];  y = act(z) + residual
//   dX        dx[m][k] = sum_n dz[m][n] w[n][k]
//   dW        dw[n][k] = sum_m dz[m][n] x[m][k]
//
// All three are C[i][j] = sum_r A(i, r) B(j, r) with each operand stored either with r
// fastest (x and w in the forward, dz in dX) or with r slowest (w in dX, both in dW).
// One kernel takes both layouts: tiles come into LDS by LDS-DMA as they lie in memory and
// r-slowest tiles are read back transposed (ds_read_b64_tr_b16), so no operand is ever
// rearranged in memory.
//
// Operand types: bf16 (v_mfma_f32_32x32x16_bf16), fp32 (v_mfma_f32_32x32x2_f32) and MX8
// (e4m3 codes with a power-of-two scale per 32 values of r, v_mfma_scale_f32_32x32x64:
// the instruction takes the scale bytes as they are stored).  Sums are fp32 throughout, but
// for what an MX8 instruction does inside: of each eight consecutive values of r it cuts the
// products toward zero to multiples of 2^-13 of the largest product's power of two (exponents
// of the codes as stored, a subnormal code's being -6), adds them, and adds the groups in
// fp32.  491520 random groups, both instruction shapes, follow that rule bit for bit.  A group
// is off by less than 7 * 2^-13 of its magnitudes' sum (8.5e-4), less than the 2^-4 that each
// value may already have lost in packing; it is why products of MX8 operands have bf16
// outputs only.  Taking the rest in as well would need bf16 products of the unpacked values,
// at little more than half the rate (8192 x 4096 x 4096: 234 us instead of 134).
//
// Tiles are BM x BN with a step of 128 bytes of r, copies one or three steps ahead.
// M = 8192, K = N = 4096, bf16: forward 234 us (1.18 PFLOP/s), dX 233, dW with db 231; MX8 134
// us (2.06 PFLOP/s); the vendor library's bf16 product of that shape 178-185 on the same box,
// warmed up.  Power holds both back: on zeros, which toggle no operand bits, the same kernels
// take 180, 176, 182 and 115 us, the library's 130.  The distance to the library stays there,
// so that part of it is waiting: the matrix pipe is busy 57-60 % of the time (MX8 43 %) at
// 1.8-1.9 GHz (2.0).
// The MFMA operands are swapped (B first), so a lane's accumulators hold 4 consecutive
// columns of one row; each wave passes them through its own piece of LDS to write 8
// consecutive columns per lane.  Everything that follows the product -- bias, the kept z,
// activation, residual -- happens there, on fp32 sums.
//
// Few rows: up to 16 rows go to a kernel that streams the weights straight into registers,
// one 16- or 32-column strip per workgroup, its waves splitting r.  Otherwise, where
// the tiles alone would leave most CUs idle, r is split over workgroups whose
// partial sums a second kernel adds in order (no atomics: bitwise reproducible).
#include <type_traits>

#include "internal.hpp"
#include "lane_sums.hpp"
#include "lds_dma.hpp"
#include "mx8.hpp"

namespace convmi {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) shortx4* lds_short4_t;

constexpr uint32_t kOob = 0x80000000u;      // beyond every buffer: such pieces are zeros
constexpr uint32_t kRecords = 0x7fffffffu;  // pieces below it are checked one by one

// ---------------------------------------------------------------- operand types
// ES bytes per element; a step is 128 bytes of r, consumed in NSUB sub-steps of FV
// 16-byte chunks per lane and operand.
struct Bf16Op {
    using T = bf16;
    static constexpr int ES = 2, NSUB = 4, FV = 1;
    static constexpr bool MX = false;
    static __device__ __forceinline__ void run(floatx16& c, const uint4* a, const uint4* b, uint32_t, uint32_t) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a[0]),
                                                    __builtin_bit_cast(bf16x8, b[0]), c, 0, 0, 0);
    }
    static __device__ __forceinline__ float add_all(const uint4& a, float s) {  // s + eight values of r
        const bf16x2 ones = {(__bf16)1.0f, (__bf16)1.0f};
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)  // pairs times one, added in fp32
            s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, u[j]), ones, s, false);
        return s;
    }
    static __device__ __forceinline__ void run16(floatx4& c, const uint4* a, const uint4* b, uint32_t, uint32_t) {
#pragma unroll
        for (int v = 0; v < 2; ++v)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[v]),
                                                        __builtin_bit_cast(bf16x8, b[v]), c, 0, 0, 0);
    }
};
struct F32Op {
    using T = float;
    static constexpr int ES = 4, NSUB = 4, FV = 1;
    static constexpr bool MX = false;
    static __device__ __forceinline__ void run(floatx16& c, const uint4* a, const uint4* b, uint32_t, uint32_t) {
        const uint32_t x[4] = {a[0].x, a[0].y, a[0].z, a[0].w}, y[4] = {b[0].x, b[0].y, b[0].z, b[0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(x[j]), __uint_as_float(y[j]), c, 0, 0, 0);
    }
    static __device__ __forceinline__ float add_all(const uint4& a, float s) {
        return s + ((__uint_as_float(a.x) + __uint_as_float(a.y)) + (__uint_as_float(a.z) + __uint_as_float(a.w)));
    }
    static __device__ __forceinline__ void run16(floatx4& c, const uint4* a, const uint4* b, uint32_t, uint32_t) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const uint32_t x[4] = {a[v].x, a[v].y, a[v].z, a[v].w}, y[4] = {b[v].x, b[v].y, b[v].z, b[v].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[j]), __uint_as_float(y[j]), c, 0, 0, 0);
        }
    }
};
struct Mx8Op {
    using T = uint8_t;
    static constexpr int ES = 1, NSUB = 2, FV = 2;
    static constexpr bool MX = true;
    static __device__ __forceinline__ intx8 join(const uint4* v) {
        return intx8{(int)v[0].x, (int)v[0].y, (int)v[0].z, (int)v[0].w,
                     (int)v[1].x, (int)v[1].y, (int)v[1].z, (int)v[1].w};
    }
    // format 0 = e4m3; sa, sb: the lane's scale byte in bits 0-7
    static __device__ __forceinline__ void run(floatx16& c, const uint4* a, const uint4* b, uint32_t sa, uint32_t sb) {
        c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(a), join(b), c, 0, 0, 0, (int)sa, 0, (int)sb);
    }
    static __device__ __forceinline__ void run16(floatx4& c, const uint4* a, const uint4* b, uint32_t sa, uint32_t sb) {
        c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(a), join(b), c, 0, 0, 0, (int)sa, 0, (int)sb);
    }
};

// ---------------------------------------------------------------- epilogue
struct Epi {
    const float* bias;        // nullable, [cols]
    const void* residual;     // nullable, [rows][cols] of the output's type; may be out
    void* z;                  // nullable, [rows][cols] of the output's type
    uint8_t *z8, *z8_scales;  // nullable
    void* out;
    int64_t rows;
    int cols, nb, act;
    const float* db_part;     // linear_join only: [splits][rows] -> db, or null
    float* db;
    int db_add;
};
// GELU, tanh form, as a * sigmoid(2u) (the same function: (1 + tanh u)/2 = sigmoid(2u)), u =
// sqrt(2/pi) (a + 0.044715 a^3): 7 instructions a value instead of 12, and no cancellation
// for negative a.  a = -inf gives NaN, as the tanh form does.
__device__ __forceinline__ float gelu_sigmoid(float a) {
    constexpr float k = -2.0f * 1.4426950408889634f;  // exp(-2u) = 2^(k u)
    const float w = a * __builtin_fmaf(k * kGeluK0 * kGeluK1, a * a, k * kGeluK0);
    return a * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(w));
}
__device__ __forceinline__ void act_piece(float (&v)[kPiece], int act) {
    switch (act) {
    case ACT_RELU:
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[j] = act_fwd<ACT_RELU>(v[j]);
        break;
    case ACT_TANH:
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[j] = act_fwd<ACT_TANH>(v[j]);
        break;
    case ACT_SIGMOID:
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[j] = act_fwd<ACT_SIGMOID>(v[j]);
        break;
    case ACT_GELU:
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[j] = gelu_sigmoid(v[j]);
        break;
    default: break;
    }
}
// Eight columns from col of one row, of which n (possibly none) exist; res: the residual
// there, if any.  Called by whole groups of four lanes that hold the four pieces of a
// 32-column block.  y is formed from the fp32 z, not from z as stored, and rounded once.
template <typename T>
__device__ __forceinline__ void emit(const Epi& e, int64_t row, int col, int n, float (&v)[kPiece],
                                     const float (&bias)[kPiece], const float (&res)[kPiece], bool first) {
    const int64_t at = row * e.cols + col;
#pragma unroll
    for (int j = 0; j < kPiece; ++j) v[j] += bias[j];
    if (e.z && n > 0) store_piece((T*)e.z + at, n, v);
    if (e.z8) {
        float u[kPiece];
#pragma unroll
        for (int j = 0; j < kPiece; ++j) u[j] = v[j];
        if (n < kPiece) {  // columns that do not exist have no say in the scale
#pragma unroll
            for (int j = 0; j < kPiece; ++j) u[j] = j < n ? v[j] : 0.0f;
        }
        uint32_t s;
        const uint2 c = mx_pack(u, s);
        if (n > 0) {
            store_codes(e.z8 + at, n, c);
            if (first) e.z8_scales[row * e.nb + col / kMxBlock] = (uint8_t)s;
        }
    }
    if (n <= 0) return;
    act_piece(v, e.act);
#pragma unroll
    for (int j = 0; j < kPiece; ++j) v[j] += res[j];
    store_piece((T*)e.out + at, n, v);
}
template <typename T>
__device__ __forceinline__ void load_residual(const Epi& e, int64_t row, int col, int n, float (&r)[kPiece]) {
    load_piece((const T*)e.residual + row * e.cols + col, e.residual ? n : 0, r);
}

// ---------------------------------------------------------------- tile kernel
struct Prod {
    const void *a, *b;              // [rows][R] rows of lda bytes, or [R][rows] (r slowest)
    const uint8_t *a_sc, *b_sc;     // MX8 scale rows, ld_sc bytes apart (a multiple of 16)
    int64_t lda, ldb;               // bytes, multiples of 16
    int64_t rows;                   // of A
    int cols;                       // rows of B
    int64_t R;                      // reduction length
    int ld_sc;
    int tiles_m, tiles_n;
    int64_t steps, steps_per_split;
    float* part;                    // [splits][rows][cols], or null
    float* db;                      // r slowest: sums of A over r, [rows], or [splits][rows] with part; or null
    int db_add;                     // add to db (no part)
    Epi epi;
};

// 16-byte chunk swizzles of the LDS tiles (chunk c of row r lies at c ^ swizzle(r)).
// r fastest, 128-byte rows: 16 lanes of a ds_read_b128 pass read one or two chunks of 8
// or 16 rows and hit distinct slots of the 256 bytes that the banks span.  r slowest,
// bf16: the four rows of a transposing read fall in distinct 64-byte pieces; fp32: the
// two lane halves read rows four apart, kept in different halves of the bank span.
__device__ __forceinline__ int swz_row(int r) { return (r >> 1) & 7; }
template <int ES, int RB> __device__ __forceinline__ int swz_tr(int r) {
    if constexpr (ES == 4) return ((r >> 2) & 1) << 3;
    else return RB >= 256 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
}
// Chunk v of sub-step s that lane half h multiplies (r fastest).  MX8: the instruction's
// 64 values of r come as 16 from each lane half, twice, while its scales are those of 32
// consecutive values: half h brings the scale of values 32h..32h+31.
template <class Op> __device__ __forceinline__ int chunk_of(int s, int v, int h) {
    return Op::MX ? 4 * s + 2 * v + h : 2 * s + h;
}

// Copies of one operand tile: DIM rows (r fastest) or columns (r slowest).
template <class Op, int DIM, bool TR, int NWAVE> struct Copies {
    static constexpr int RB = TR ? DIM * Op::ES : 128;  // bytes of an LDS row
    static constexpr int CPR = RB / 16, RPI = 64 / CPR;  // chunks per row, rows per copy
    static constexpr int COUNT = DIM / 8;               // copies of 1 KB
    static constexpr int PER = (COUNT + NWAVE - 1) / NWAVE;
    static_assert(COUNT % NWAVE == 0, "every wave issues the same number of copies");
    static_assert(NWAVE % 2 == 0, "the rows of a wave's copies have one chunk pattern");
    const char* base;
    int64_t ld;
    uint32_t off[PER];  // byte offset of the lane's chunk from base, or kOob
    int lane_k[2];      // r fastest: byte offset of the lane's chunk within a step, by copy parity
    int row0;           // r slowest: the lane's row in copy 0 of the wave

    __device__ __forceinline__ void init(const void* p, int64_t ld_, int64_t d0, int64_t dim, int wid, int lane) {
        ld = ld_;
        if constexpr (!TR) {
            base = (const char*)p + d0 * ld;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = (wid + NWAVE * j) * RPI + lane / CPR;
                lane_k[j] = ((lane % CPR) ^ swz_row(row)) * 16;
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int row = (wid + NWAVE * j) * RPI + lane / CPR;
                off[j] = d0 + row < dim ? (uint32_t)(row * ld) : kOob;
            }
        } else {
            base = (const char*)p + d0 * Op::ES;
            row0 = wid * RPI + lane / CPR;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int row = row0 + NWAVE * RPI * j;
                const int c = ((lane % CPR) ^ swz_tr<Op::ES, RB>(row)) * 16;
                off[j] = d0 * Op::ES + c < dim * Op::ES ? (uint32_t)(row * ld + c) : kOob;
            }
        }
    }
    // Step st (of 128 bytes of r; R elements in all): its buffer and what is left of r.
    dma_rsrc rs;
    int left;
    __device__ __forceinline__ void step(int64_t st, int64_t R) {
        constexpr int KE = 128 / Op::ES;
        rs = make_rsrc(base + (TR ? st * KE * ld : st * 128), kRecords);
        const int64_t l = TR ? R - st * KE : R * Op::ES - st * 128;  // rows, or bytes of a row
        left = l < (1 << 20) ? (int)l : 1 << 20;
    }
    // Copy j of the wave's PER for that step into the LDS tile at dst.
    __device__ __forceinline__ void copy(int j, uint32_t dst, int wid) const {
        uint32_t o;
        if constexpr (!TR) o = lane_k[j & 1] < left ? off[j] + (uint32_t)lane_k[j & 1] : kOob;
        else o = row0 + NWAVE * RPI * j < left ? off[j] : kOob;
        dma16_buf(o, rs, __builtin_amdgcn_readfirstlane(dst + (uint32_t)(wid + NWAVE * j) * 1024));
    }
};

// The lane's chunks of sub-step s for 32 rows (or columns, r slowest) from d of a tile.
template <class Op, int DIM, bool TR>
__device__ __forceinline__ void read_frag(const unsigned char* tile, int d, int s, int lane, uint4* f) {
    const int h = lane >> 5;
    if constexpr (!TR) {
        const int row = d + (lane & 31);
#pragma unroll
        for (int v = 0; v < Op::FV; ++v)
            f[v] = *(const uint4*)(tile + row * 128 + ((chunk_of<Op>(s, v, h) ^ swz_row(row)) << 4));
    } else if constexpr (Op::ES == 2) {
        constexpr int RB = DIM * 2;
        const int l16 = lane & 15, hi = (lane >> 4) & 1;
        uint2 q[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = s * 16 + 8 * h + 4 * half + (l16 >> 2);
            const int cb = 2 * (d + 16 * hi + 4 * (l16 & 3));
            const int off = row * RB + ((((cb >> 4) ^ swz_tr<2, RB>(row)) << 4) | (cb & 15));
            q[half] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t)(tile + off)));
        }
        f[0] = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
    } else {
        constexpr int RB = DIM * 4;
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = s * 8 + 4 * h + j;
            const int cb = 4 * (d + (lane & 31));
            q[j] = *(const uint32_t*)(tile + row * RB + ((((cb >> 4) ^ swz_tr<4, RB>(row)) << 4) | (cb & 15)));
        }
        f[0] = make_uint4(q[0], q[1], q[2], q[3]);
    }
}

template <class Op, int BM, int BN, int WM, int WN, int STAGES, bool ATR, bool BTR, typename TOut>
__global__ __launch_bounds__(WM * WN * 64) __attribute__((amdgpu_waves_per_eu(2, 2))) void linear_tiles(Prod g) {
    constexpr int NWAVE = WM * WN;
    constexpr int TM = BM / (WM * 32), TN = BN / (WN * 32);
    static_assert(TM * WM * 32 == BM && TN * WN * 32 == BN, "tile shape");
    constexpr int STAGE_BYTES = (BM + BN) * 128;
    constexpr int SC_BYTES = Op::MX ? (BM + BN) * 16 : 0;  // scales of four steps
    constexpr int SC_COPIES = (BM + BN) / 64;
    constexpr int PITCH = TN * 32 + 4;                     // floats of a staged output row
    constexpr int EPI_BYTES = NWAVE * 32 * PITCH * 4;
    constexpr int RING = STAGES * STAGE_BYTES + 2 * SC_BYTES;
    constexpr int LDS_BYTES = RING > EPI_BYTES ? RING : EPI_BYTES;
    __shared__ __align__(1024) unsigned char smem[LDS_BYTES];

    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Consecutive tiles of an XCD cover a block of up to 8 row tiles by several column
    // tiles, so that its L2 holds the panels they share.
    const int tile = xcd_tile(blockIdx.x, gridDim.x);
    const int per = 8 * g.tiles_n, grp = tile / per;
    const int first = grp * 8, rows_in = g.tiles_m - first < 8 ? g.tiles_m - first : 8;
    const int tm = first + (tile - grp * per) % rows_in, tn = (tile - grp * per) / rows_in;
    const int64_t m0 = (int64_t)tm * BM;
    const int n0 = tn * BN;
    const int64_t st0 = (int64_t)blockIdx.y * g.steps_per_split;
    const int64_t st1 = st0 + g.steps_per_split < g.steps ? st0 + g.steps_per_split : g.steps;
    const int count = (int)(st1 - st0);

    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    Copies<Op, BM, ATR, NWAVE> ca;
    Copies<Op, BN, BTR, NWAVE> cb;
    ca.init(g.a, g.lda, m0, g.rows, wid, lane);
    cb.init(g.b, g.ldb, n0, g.cols, wid, lane);
    // MX8 scales: 16 bytes (four steps) per tile row, rows of A then of B; wave i copies
    // rows 64i.. of them
    uint32_t sc_off = kOob;
    const char* sc_base = nullptr;
    if constexpr (Op::MX) {
        const bool of_a = wid < BM / 64;
        const int row = (of_a ? wid : wid - BM / 64) * 64 + lane;
        sc_base = of_a ? (const char*)g.a_sc + m0 * g.ld_sc : (const char*)g.b_sc + (int64_t)n0 * g.ld_sc;
        if (wid < SC_COPIES && (of_a ? m0 + row < g.rows : n0 + row < g.cols)) sc_off = (uint32_t)(row * g.ld_sc);
    }
    constexpr int PA = Copies<Op, BM, ATR, NWAVE>::PER, PB = Copies<Op, BN, BTR, NWAVE>::PER;
    constexpr int kCopies = PA + PB;
    uint32_t slot = 0;
    int next = 0;
    auto begin = [&](int i) {  // step st0 + i goes into ring slot i % STAGES
        next = i;
        slot = lds0 + (uint32_t)(i % STAGES) * STAGE_BYTES;
        ca.step(st0 + i, g.R);
        cb.step(st0 + i, g.R);
    };
    auto copy = [&](int c) {  // copy c of kCopies of the step begun last; MX8's scales with the last one
        if (c < PA) ca.copy(c, slot, wid);
        else cb.copy(c - PA, slot + BM * 128, wid);
        if constexpr (Op::MX)
            if (c == kCopies - 1 && (next & 3) == 0 && wid < SC_COPIES)
                dma16_buf(sc_off, make_rsrc(sc_base + ((st0 + next) >> 2) * 16, kRecords),
                          __builtin_amdgcn_readfirstlane(lds0 + STAGES * STAGE_BYTES +
                                                         (uint32_t)((next >> 2) & 1) * SC_BYTES + (uint32_t)wid * 1024));
    };

    const int wm = wid / WN, wn = wid % WN;
    floatx16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    // Sums of A over r (the bias gradient) ride along in the workgroups of the first column
    // tile: wave column c adds up the fragments of sub-steps c, c + WN, ...  (With all of it
    // on one wave column these workgroups finished 48 us late at 8192 x 4096 x 4096 bf16.)
    float dsum[TM];
#pragma unroll
    for (int t = 0; t < TM; ++t) dsum[t] = 0.0f;
    const bool sums = ATR && g.db && tn == 0;

    // One step's products.  The copies of a later step are issued between them, over the
    // first half of the step: in a burst at its start they hold up every wave's products
    // while the CU's 64-byte-per-cycle path takes them (8192 x 4096 x 4096 bf16: 243.5 ->
    // 237.7 us; on zeros, where the clock is not power-limited, 202 -> 187).  MX8, with
    // half as many products between two reads, measured the other way (141.8 against
    // 147.6 us) and issues them before the step.
    constexpr int SPREAD = Op::NSUB / 2, PER_GROUP = (kCopies + SPREAD * TM - 1) / (SPREAD * TM);
    uint4 sa4[Op::MX ? TM : 1], sb4[Op::MX ? TN : 1];
    auto compute = [&](int i, bool more) {
        const unsigned char* As = smem + (i % STAGES) * STAGE_BYTES;
        const unsigned char* Bs = As + BM * 128;
        if (Op::MX && more)
#pragma unroll
            for (int c = 0; c < kCopies; ++c) copy(c);
        uint32_t sa[TM], sb[TN];
        if constexpr (Op::MX) {
            if ((i & 3) == 0) {  // the scale bytes of four steps, 16 per row
                const unsigned char* sc = smem + STAGES * STAGE_BYTES + ((i >> 2) & 1) * SC_BYTES;
#pragma unroll
                for (int t = 0; t < TM; ++t)
                    sa4[t] = *(const uint4*)(sc + (wm * TM * 32 + t * 32 + (lane & 31)) * 16);
#pragma unroll
                for (int t = 0; t < TN; ++t)
                    sb4[t] = *(const uint4*)(sc + (BM + wn * TN * 32 + t * 32 + (lane & 31)) * 16);
            }
            // this step's four per row are the lowest word: byte 2s + h belongs to sub-step s
            const int sh = 8 * (lane >> 5);
#pragma unroll
            for (int t = 0; t < TM; ++t) {
                sa[t] = sa4[t].x >> sh;
                sa4[t] = make_uint4(sa4[t].y, sa4[t].z, sa4[t].w, 0u);
            }
#pragma unroll
            for (int t = 0; t < TN; ++t) {
                sb[t] = sb4[t].x >> sh;
                sb4[t] = make_uint4(sb4[t].y, sb4[t].z, sb4[t].w, 0u);
            }
        }
#pragma unroll
        for (int s = 0; s < Op::NSUB; ++s) {
            uint4 af[TM][Op::FV], bf[TN][Op::FV];
#pragma unroll
            for (int t = 0; t < TM; ++t) read_frag<Op, BM, ATR>(As, wm * TM * 32 + t * 32, s, lane, af[t]);
#pragma unroll
            for (int t = 0; t < TN; ++t) read_frag<Op, BN, BTR>(Bs, wn * TN * 32 + t * 32, s, lane, bf[t]);
            if constexpr (ATR)
                if (sums && s % WN == wn)
#pragma unroll
                    for (int t = 0; t < TM; ++t) dsum[t] = Op::add_all(af[t][0], dsum[t]);
#pragma unroll
            for (int p = 0; p < TM; ++p) {
#pragma unroll
                for (int q = 0; q < TN; ++q)
                    Op::run(acc[p][q], bf[q], af[p], Op::MX ? sb[q] >> (16 * s) : 0u,
                            Op::MX ? sa[p] >> (16 * s) : 0u);
                if (!Op::MX && s < SPREAD && more) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int c = 0; c < PER_GROUP; ++c)
                        if ((s * TM + p) * PER_GROUP + c < kCopies) copy((s * TM + p) * PER_GROUP + c);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };

#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
        if (i < count) {
            begin(i);
#pragma unroll
            for (int c = 0; c < kCopies; ++c) copy(c);
        }
    for (int i = 0; i < count; ++i) {
        // this wave's copies of the steps after i that are already on their way
        const int later = count - 1 - i < STAGES - 2 ? count - 1 - i : STAGES - 2;
        int flying = later * kCopies;
        if constexpr (Op::MX && STAGES > 2)
            for (int l = 1; l <= later; ++l) flying += ((i + l) & 3) == 0 && wid < SC_COPIES;
        wait_dma(flying);
        __syncthreads();
        const bool more = i + STAGES - 1 < count;
        if (more) begin(i + STAGES - 1);
        compute(i, more);
    }
    __syncthreads();

    if constexpr (ATR)
        if (sums) {  // the same for the whole workgroup
            float* ds = (float*)smem;
#pragma unroll
            for (int t = 0; t < TM; ++t) {  // lanes i and i + 32 hold halves of row i's sum
                const float v = dsum[t] + lane_xor32(dsum[t]);
                if (lane < 32) ds[wn * BM + wm * TM * 32 + t * 32 + lane] = v;
            }
            __syncthreads();
            for (int i = threadIdx.x; i < BM && m0 + i < g.rows; i += NWAVE * 64) {
                float v = 0.0f;
#pragma unroll
                for (int c = 0; c < WN; ++c) v += ds[c * BM + i];
                float* o = g.db + (g.part ? (int64_t)blockIdx.y * g.rows : 0) + m0 + i;
                *o = g.db_add ? *o + v : v;
            }
            __syncthreads();
        }

    // ---- each wave: 32 rows at a time through its own piece of LDS
    float* Cs = (float*)smem + wid * 32 * PITCH;
    constexpr int LPR = TN * 4, RPP = 64 / LPR;  // lanes per row, rows per pass
    const int lc = (lane % LPR) * kPiece;
    const int col = n0 + wn * TN * 32 + lc, n = g.cols - col;
    float bias[kPiece];
    load_piece(g.epi.bias + col, g.epi.bias && !g.part ? n : 0, bias);
    // One copy of the output code for all TM row groups: the accumulators move down one
    // group per turn, so that every index is a constant and they stay in registers.
    constexpr int NP = 32 / RPP;
#pragma unroll 1
    for (int p = 0; p < TM; ++p) {
        const int64_t row0 = m0 + wm * TM * 32 + p * 32 + lane / LPR;
        float res[NP][kPiece];
#pragma unroll
        for (int k = 0; k < NP; ++k)
            load_residual<TOut>(g.epi, row0 + k * RPP, col, row0 + k * RPP < g.rows && !g.part ? n : 0, res[k]);
#pragma unroll
        for (int q = 0; q < TN; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *(float4*)(Cs + (lane & 31) * PITCH + q * 32 + 8 * e + 4 * (lane >> 5)) =
                    make_float4(acc[0][q][4 * e], acc[0][q][4 * e + 1], acc[0][q][4 * e + 2], acc[0][q][4 * e + 3]);
#pragma unroll
        for (int t = 1; t < TM; ++t)
#pragma unroll
            for (int q = 0; q < TN; ++q) acc[t - 1][q] = acc[t][q];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int64_t row = row0 + k * RPP;
            float v[kPiece];
            load_piece(Cs + (lane / LPR + k * RPP) * PITCH + lc, kPiece, v);
            const int live = row < g.rows ? n : 0;
            if (g.part) {
                if (live > 0) store_piece(g.part + ((int64_t)blockIdx.y * g.rows + row) * g.cols + col, live, v);
            } else {
                emit<TOut>(g.epi, row, col, live, v, bias, res[k], (lane & 3) == 0);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// v += the partials of splits s, s + 1, ... in order, U of them loaded together, while U are
// left; returns the first split not added.
template <int U>
__device__ __forceinline__ int add_splits(const float* p, int64_t stride, int s, int splits, int n, float (&v)[kPiece]) {
    for (; s + U <= splits; s += U) {
        float u[U][kPiece];
#pragma unroll
        for (int t = 0; t < U; ++t) load_piece(p + (s + t) * stride, n, u[t]);
#pragma unroll
        for (int t = 0; t < U; ++t)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) v[j] += u[t][j];
    }
    return s;
}
template <int U> __device__ __forceinline__ int add_splits(const float* p, int64_t stride, int s, int splits, float& v) {
    for (; s + U <= splits; s += U) {
        float u[U];
#pragma unroll
        for (int t = 0; t < U; ++t) u[t] = p[(s + t) * stride];
#pragma unroll
        for (int t = 0; t < U; ++t) v += u[t];
    }
    return s;
}

// Sum of the splits' partial products, in order, then the epilogue.  Bound by the partials'
// bytes from the last-level cache; small ones by the launch (8 splits of 256 x 512: 4.1 us)
// and by round trips, so that loads go out in groups (dW of 131072 x 64 by 64 bf16, 64
// splits, when the step was made: 43.2 us with one db partial at a time, 29.7 with groups of
// 16; 128 splits now, 29.6).
template <typename TOut>
__global__ __launch_bounds__(256) void linear_join(const float* __restrict__ part, int splits, Epi e, int per_row,
                                                   int64_t count, FastDiv fdr) {
    for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < count; p += (int64_t)gridDim.x * 256) {
        const int64_t row = count < (1LL << 31) ? (int64_t)fdiv((int)p, fdr) : p / per_row;
        const int i = (int)(p - row * per_row), col = i * kPiece, n = e.cols - col;
        const float* src = part + row * e.cols + col;
        const int64_t stride = e.rows * e.cols;
        float v[kPiece] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, bias[kPiece], res[kPiece];
        load_piece(e.bias + col, e.bias ? n : 0, bias);
        load_residual<TOut>(e, row, col, n, res);
        int s = add_splits<8>(src, stride, 0, splits, n, v);
        s = add_splits<4>(src, stride, s, splits, n, v);
        add_splits<1>(src, stride, s, splits, n, v);
        emit<TOut>(e, row, col, n, v, bias, res, (i & 3) == 0);
    }
    if (e.db_part)
        for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < e.rows; r += (int64_t)gridDim.x * 256) {
            float v = 0.0f;
            int s = add_splits<16>(e.db_part + r, e.rows, 0, splits, v);
            s = add_splits<4>(e.db_part + r, e.rows, s, splits, v);
            add_splits<1>(e.db_part + r, e.rows, s, splits, v);
            e.db[r] = e.db_add ? e.db[r] + v : v;
        }
}

// ---------------------------------------------------------------- few rows
// Forward of up to 16 rows: a workgroup owns NC strips of 16 columns (rows of w), its eight
// waves take every eighth 128-byte step of r.  Lane i%16 loads its quarter of each half
// step of w row i and of x row i (the order of r is the same on both sides, so it does
// not matter to the sum; it is the one in which the MX8 instruction assigns its scales).
// U steps are in flight.  Loads go straight to registers at any alignment, so odd row
// lengths need no copy.  The waves' sums meet in LDS.  Bound by the weights' bytes: one row,
// 4096 -> 8192 bf16, 16.3 us with the weights in the last-level cache, 18.0 from HBM (3.7
// TB/s), of which a small launch's latency is 3-4; fp32 36.1 (3.7 TB/s), MX8 13.0 (2.7); rows of
// an odd number of bf16, whose loads split, 36.  The reduction stays in one workgroup, so few
// columns over a long one are slow: 16 rows, 65536 -> 64 bf16 take 118 us (17 rows, in split
// tiles, 17), 2^20 -> 16 take 3.1 ms (72 us).
constexpr int kSkinnyRows = 16, kSkinnyWaves = 8;
struct Skinny {
    const void *x, *w;
    const uint8_t *x_sc, *w_sc;
    int M, N;
    int64_t K;  // bytes of a row
    int nb;     // scale bytes of a row
    Epi epi;
};
// The lane's two chunks of a step at p, of which n bytes exist.
__device__ __forceinline__ void load_step(const char* p, int64_t n, int gq, uint4 (&v)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int o = 64 * i + 16 * gq;
        if (o + 16 <= n) {
            __builtin_memcpy(&v[i], p + o, 16);
        } else {
            uint32_t d[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int b = 0; b < 16; ++b)
                if (o + b < n) d[b >> 2] |= (uint32_t)(uint8_t)p[o + b] << (8 * (b & 3));
            v[i] = make_uint4(d[0], d[1], d[2], d[3]);
        }
    }
}

template <class Op, int NC, typename TOut>
__global__ __launch_bounds__(kSkinnyWaves * 64) void linear_skinny(Skinny g) {
    constexpr int U = 8;
    constexpr int PITCH = NC * 16 + 4;
    __shared__ float red[kSkinnyWaves][16][PITCH];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int i16 = lane & 15, gq = lane >> 4;
    const int n0 = blockIdx.x * NC * 16;
    // rows past the end repeat the last one; nothing is stored for them
    const char* wp[NC];
    const uint8_t* ws[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t row = n0 + c * 16 + i16 < g.N ? n0 + c * 16 + i16 : g.N - 1;
        wp[c] = (const char*)g.w + row * g.K;
        ws[c] = Op::MX ? g.w_sc + row * g.nb + gq : nullptr;
    }
    const int64_t xrow = i16 < g.M ? i16 : g.M - 1;
    const char* xp = (const char*)g.x + xrow * g.K;
    const uint8_t* xs = Op::MX ? g.x_sc + xrow * g.nb + gq : nullptr;
    floatx4 acc[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[c] = floatx4{0.f, 0.f, 0.f, 0.f};

    const int64_t full = g.K >> 7;
    int64_t st = wid;
    for (; st + (U - 1) * kSkinnyWaves < full; st += U * kSkinnyWaves) {
        uint4 wv[U][NC][2], xv[U][2];
        uint32_t wsc[U][NC], xsc[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = (st + u * kSkinnyWaves) * 128;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                load_step(wp[c] + at, 128, gq, wv[u][c]);
                wsc[u][c] = Op::MX ? ws[c][at >> 5] : 0;
            }
            load_step(xp + at, 128, gq, xv[u]);
            xsc[u] = Op::MX ? xs[at >> 5] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < NC; ++c) Op::run16(acc[c], wv[u][c], xv[u], wsc[u][c], xsc[u]);
    }
    for (; st * 128 < g.K; st += kSkinnyWaves) {  // the last steps, the very last one maybe cut
        uint4 wv[2], xv[2];
        const int64_t at = st * 128, left = g.K - at;
        const bool scaled = Op::MX && left > 32 * gq;
        load_step(xp + at, left, gq, xv);
        const uint32_t xsc = scaled ? xs[at >> 5] : 0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            load_step(wp[c] + at, left, gq, wv);
            Op::run16(acc[c], wv, xv, scaled ? ws[c][at >> 5] : 0, xsc);
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
        *(float4*)&red[wid][i16][c * 16 + gq * 4] = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
    __syncthreads();
    constexpr int PPR = NC * 2;  // pieces per row
    if (threadIdx.x < 16 * PPR) {
        const int row = threadIdx.x / PPR, lc = (threadIdx.x % PPR) * kPiece;
        const int col = n0 + lc, n = row < g.M ? g.N - col : 0;
        float v[kPiece] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, bias[kPiece], res[kPiece];
        load_piece(g.epi.bias + col, g.epi.bias ? n : 0, bias);
        load_residual<TOut>(g.epi, row, col, n, res);
#pragma unroll
        for (int k = 0; k < kSkinnyWaves; ++k)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) v[j] += red[k][row][lc + j];
        emit<TOut>(g.epi, row, col, n, v, bias, res, (threadIdx.x & 3) == 0);
    }
}

// ---------------------------------------------------------------- host side
enum LinType { LT_BF16, LT_F32, LT_MX8 };
LinType type_of(const LinearDims& d, int op) {
    if (op == LIN_FORWARD && d.x_mx8) return LT_MX8;
    return d.dtype == DT_BF16 ? LT_BF16 : LT_F32;
}
int type_size(LinType t) { return t == LT_MX8 ? 1 : t == LT_BF16 ? 2 : 4; }

struct LinPlan {
    bool skinny;
    int tile;                 // block tile side
    int splits;
    int64_t steps, steps_per_split;
    // workspace: operands and scales padded (dW of an MX8 x: unpacked), partials
    size_t pad_a, pad_b, pad_sa, pad_sb, part, db_part, total;
};
int64_t pad16(int64_t n, int es) { return (n * es + 15) / 16 * 16 / es; }

// i, j, r sizes of an operation.
void sizes_of(const LinearDims& d, int op, int64_t& I, int64_t& J, int64_t& R) {
    if (op == LIN_FORWARD) { I = d.M; J = d.N; R = d.K; }
    else if (op == LIN_BACKWARD_DATA) { I = d.M; J = d.K; R = d.N; }
    else { I = d.N; J = d.K; R = d.M; }
}

// A launch has fewer than 2^32 threads along x: 256 per tile (512 of side 256).
constexpr int64_t kMaxTiles = 1LL << 24;

LinPlan make_plan(const LinearDims& d, int op) {
    LinPlan p{};
    int64_t I, J, R;
    sizes_of(d, op, I, J, R);
    const LinType t = type_of(d, op);
    const int es = type_size(t);
    p.skinny = op == LIN_FORWARD && d.M <= kSkinnyRows;
    if (p.skinny || d.M == 0) return p;
    p.steps = ceil_div(R * es, 128);
    // Least estimated time over tile sides and splits of the reduction.  A CU takes n
    // workgroups; two of 128- or 64-sided tiles run together, one of 256.  one, two: us per
    // step of a workgroup alone and of two together; fixed: copies' first latency and the
    // output.  Fitted to sweeps of the three operations at up to 29 shapes per type (8..32768
    // rows and columns, 64..2^20 of r; every side, 1..256 splits): on the present kernels the
    // pick is on average within 0.4-1.5 % of the best by operation and type, at most 21 % off.
    struct Cand { int side; double one, two, fixed; };
    static const Cand cands[5][3] = {
        {{256, 1.62, 0, 12}, {128, 0.62, 1.15, 7}, {64, 0.27, 0.42, 3.5}},  // bf16, forward
        {{256, 1.62, 0, 12}, {128, 0.72, 1.2, 7}, {64, 0.40, 0.50, 3.5}},   // bf16, an operand with r slowest
        {{0, 0, 0, 0}, {128, 2.1, 3.6, 7}, {64, 0.65, 1.2, 3.5}},           // f32, forward
        {{0, 0, 0, 0}, {128, 2.2, 3.6, 7}, {64, 0.75, 1.25, 3.5}},          // f32, an operand with r slowest
        {{256, 1.6, 0, 12}, {128, 0.70, 1.36, 7}, {64, 0.52, 0.60, 3.5}}};  // mx8
    const Cand* cand = cands[t == LT_MX8 ? 4 : (t == LT_F32 ? 2 : 0) + (op != LIN_FORWARD)];
    double best = 1e300;
    for (int i = 0; i < 3; ++i) {
        const Cand& c = cand[i];
        if (c.side == 0) continue;
        const int64_t tiles = ceil_div(I, c.side) * ceil_div(J, c.side);
        if (tiles >= kMaxTiles / (c.side == 256 ? 2 : 1)) continue;
        for (int S = 1; S <= 256 && (S == 1 || S * 2 <= p.steps); S *= 2) {
            int64_t per = ceil_div(p.steps, S);
            if (t == LT_MX8) per = ceil_div(per, 4) * 4;  // scales come four steps at a time
            const int64_t splits = ceil_div(p.steps, per), n = ceil_div(tiles * splits, 256);
            double us = c.side == 256 ? n * (c.fixed + per * c.one)
                                      : (n + 1) / 2 * c.fixed + per * (n / 2 * c.two + n % 2 * c.one);
            if (splits > 1) us += 4.0 + 0.08 * splits + (double)splits * I * J * 8.0 / 6e6;  // second launch, partials
            if (us < best) {
                best = us;
                p.tile = c.side;
                p.splits = (int)splits;
                p.steps_per_split = per;
            }
        }
    }
    // workspace
    size_t at = 0;
    auto take = [&](size_t bytes) { const size_t o = at; at = align_up(at + bytes, 256); return o; };
    p.pad_a = p.pad_b = p.pad_sa = p.pad_sb = (size_t)-1;
    const int64_t wa = op == LIN_FORWARD ? d.K : d.N, ra = d.M;             // A as stored
    const int64_t wb = d.K, rb = op == LIN_BACKWARD_WEIGHT ? d.M : d.N;     // B as stored
    if (wa * es % 16) p.pad_a = take((size_t)ra * pad16(wa, es) * es);
    if (wb * es % 16 || (op == LIN_BACKWARD_WEIGHT && d.x_mx8)) p.pad_b = take((size_t)rb * pad16(wb, es) * es);
    if (t == LT_MX8) {
        const int64_t nb = ceil_div(d.K, kMxBlock);
        if (nb % 16) {
            p.pad_sa = take((size_t)ra * pad16(nb, 1));
            p.pad_sb = take((size_t)rb * pad16(nb, 1));
        }
    }
    if (p.splits > 1) {
        p.part = take((size_t)p.splits * I * J * sizeof(float));
        if (op == LIN_BACKWARD_WEIGHT) p.db_part = take((size_t)p.splits * I * sizeof(float));
    }
    p.total = at;
    return p;
}

template <class Op, int SIDE, bool ATR, bool BTR, typename TOut>
hipError_t launch_tiles(const Prod& g, int splits, hipStream_t s) {
    constexpr int WM = 2, WN = SIDE == 256 ? 4 : 2, STAGES = SIDE == 64 ? 4 : 2;
    linear_tiles<Op, SIDE, SIDE, WM, WN, STAGES, ATR, BTR, TOut>
        <<<dim3((unsigned)(g.tiles_m * g.tiles_n), (unsigned)splits), WM * WN * 64, 0, s>>>(g);
    return hipGetLastError();
}
template <class Op, bool ATR, bool BTR, typename TOut>
hipError_t launch_sides(const LinPlan& p, Prod g, hipStream_t s) {
    g.tiles_m = (int)ceil_div(g.rows, p.tile);
    g.tiles_n = (int)ceil_div(g.cols, p.tile);
    g.steps = p.steps;
    g.steps_per_split = p.steps_per_split;
    hipError_t e;
    if (p.tile == 64) e = launch_tiles<Op, 64, ATR, BTR, TOut>(g, p.splits, s);
    else if (p.tile == 128) e = launch_tiles<Op, 128, ATR, BTR, TOut>(g, p.splits, s);
    else if constexpr (Op::ES < 4) e = launch_tiles<Op, 256, ATR, BTR, TOut>(g, p.splits, s);
    else e = hipErrorInvalidValue;
    if (e != hipSuccess || p.splits == 1) return e;
    const int per_row = (int)ceil_div(g.cols, kMxBlock) * (kMxBlock / kPiece);
    const int64_t count = g.rows * per_row, blocks = ceil_div(count, 256);
    linear_join<TOut><<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, s>>>(g.part, p.splits, g.epi, per_row,
                                                                               count, make_fastdiv((uint32_t)per_row));
    return hipGetLastError();
}

template <class Op, typename TOut> hipError_t launch_skinny(const Skinny& g, hipStream_t s) {
    // 32 columns per workgroup where the 8-bit z needs whole blocks, and where that still
    // gives every CU a workgroup (1x4096 by 8192 columns, bf16, when it was chosen: 14.4 us
    // against 15.8)
    constexpr int threads = kSkinnyWaves * 64;
    if (g.epi.z8 || g.N >= 32 * 256)
        linear_skinny<Op, 2, TOut><<<(unsigned)ceil_div(g.N, 32), threads, 0, s>>>(g);
    else
        linear_skinny<Op, 1, TOut><<<(unsigned)ceil_div(g.N, 16), threads, 0, s>>>(g);
    return hipGetLastError();
}

}  // namespace

bool linear_fits(int64_t M, int64_t K, int64_t N) {
    auto tiles = [](int64_t i, int64_t j) { return ceil_div(i, 128) * ceil_div(j, 128); };
    return tiles(M, N) < kMaxTiles && tiles(M, K) < kMaxTiles && tiles(N, K) < kMaxTiles;
}

size_t linear_ws_bytes(const LinearDims& d, int op) { return make_plan(d, op).total; }

void linear_plan_text(const LinearDims& d, int op, char* buf, size_t len) {
    const LinPlan p = make_plan(d, op);
    static const char* const names[3] = {"bf16", "f32", "mx8"};
    const char* ty = names[type_of(d, op)];
    if (d.M == 0) snprintf(buf, len, "empty");
    else if (p.skinny) snprintf(buf, len, "rows %s", ty);
    else
        snprintf(buf, len, "tiles %s %dx%d split %d%s", ty, p.tile, p.tile, p.splits,
                 p.pad_a != (size_t)-1 || p.pad_b != (size_t)-1 ? " prep" : "");
}

hipError_t launch_linear_fwd(const LinearDims& d, const void* x, const void* x_sc, const void* w, const void* w_sc,
                             const float* bias, const void* residual, void* z, void* z8_scales, void* y, void* ws,
                             hipStream_t s) {
    if (d.M == 0) return hipSuccess;
    const LinPlan p = make_plan(d, LIN_FORWARD);
    const LinType t = type_of(d, LIN_FORWARD);
    const int es = type_size(t);
    Epi e{};
    e.bias = bias;
    e.residual = residual;
    e.z = d.z_mx8 ? nullptr : z;
    e.z8 = d.z_mx8 ? (uint8_t*)z : nullptr;
    e.z8_scales = (uint8_t*)z8_scales;
    e.out = y;
    e.rows = d.M;
    e.cols = (int)d.N;
    e.nb = (int)ceil_div(d.N, kMxBlock);
    e.act = d.act;
    const int64_t nb = ceil_div(d.K, kMxBlock);
    if (p.skinny) {
        const Skinny g{x, w, (const uint8_t*)x_sc, (const uint8_t*)w_sc, (int)d.M, (int)d.N, d.K * es, (int)nb, e};
        if (t == LT_BF16) return launch_skinny<Bf16Op, bf16>(g, s);
        if (t == LT_F32) return launch_skinny<F32Op, float>(g, s);
        return launch_skinny<Mx8Op, bf16>(g, s);
    }
    Prod g{};
    g.a = x;
    g.b = w;
    g.a_sc = (const uint8_t*)x_sc;
    g.b_sc = (const uint8_t*)w_sc;
    const int64_t kp = pad16(d.K, es);
    g.lda = g.ldb = kp * es;
    g.ld_sc = (int)pad16(nb, 1);
    char* base = (char*)ws;
    Prep prep{};
    if (p.pad_a != (size_t)-1) {
        g.a = base + p.pad_a;
        g.b = base + p.pad_b;
        add_prep(prep, x, nullptr, base + p.pad_a, d.M, d.K * es, es);
        add_prep(prep, w, nullptr, base + p.pad_b, d.N, d.K * es, es);
    }
    if (p.pad_sa != (size_t)-1) {
        g.a_sc = (const uint8_t*)base + p.pad_sa;
        g.b_sc = (const uint8_t*)base + p.pad_sb;
        add_prep(prep, x_sc, nullptr, base + p.pad_sa, d.M, nb, es);
        add_prep(prep, w_sc, nullptr, base + p.pad_sb, d.N, nb, es);
    }
    if (const hipError_t err = launch_prep(prep, d.dtype, s); err != hipSuccess) return err;
    g.rows = d.M;
    g.cols = (int)d.N;
    g.R = d.K;
    g.part = p.splits > 1 ? (float*)(base + p.part) : nullptr;
    g.epi = e;
    if (t == LT_BF16) return launch_sides<Bf16Op, false, false, bf16>(p, g, s);
    if (t == LT_F32) return launch_sides<F32Op, false, false, float>(p, g, s);
    return launch_sides<Mx8Op, false, false, bf16>(p, g, s);
}

hipError_t launch_linear_dx(const LinearDims& d, const void* dz, const void* w, void* dx, void* ws, hipStream_t s) {
    if (d.M == 0) return hipSuccess;
    const LinPlan p = make_plan(d, LIN_BACKWARD_DATA);
    const int es = (int)dtype_size(d.dtype);
    char* base = (char*)ws;
    Prod g{};
    g.a = dz;
    g.b = w;
    g.lda = pad16(d.N, es) * es;
    g.ldb = pad16(d.K, es) * es;
    Prep prep{};
    if (p.pad_a != (size_t)-1) add_prep(prep, dz, nullptr, base + p.pad_a, d.M, d.N * es, es), g.a = base + p.pad_a;
    if (p.pad_b != (size_t)-1) add_prep(prep, w, nullptr, base + p.pad_b, d.N, d.K * es, es), g.b = base + p.pad_b;
    if (const hipError_t err = launch_prep(prep, d.dtype, s); err != hipSuccess) return err;
    g.rows = d.M;
    g.cols = (int)d.K;
    g.R = d.N;
    g.part = p.splits > 1 ? (float*)(base + p.part) : nullptr;
    g.epi.out = dx;
    g.epi.rows = d.M;
    g.epi.cols = (int)d.K;
    if (d.dtype == DT_BF16) return launch_sides<Bf16Op, false, true, bf16>(p, g, s);
    return launch_sides<F32Op, false, true, float>(p, g, s);
}

// dw = db = 0 for an empty batch (a fill kernel: memset nodes do not belong in captured graphs).
__global__ __launch_bounds__(256) void zero_floats(float* p, int64_t n, float* q, int64_t m) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n + m; i += (int64_t)gridDim.x * 256)
        (i < n ? p[i] : q[i - n]) = 0.0f;
}

hipError_t launch_linear_dw(const LinearDims& d, const void* x, const void* x_sc, const void* dz, float* dw, float* db,
                            int accumulate, void* ws, hipStream_t s) {
    const LinPlan p = make_plan(d, LIN_BACKWARD_WEIGHT);
    const int es = (int)dtype_size(d.dtype);
    char* base = (char*)ws;
    hipError_t e = hipSuccess;
    if (d.M == 0) {
        if (!accumulate) zero_floats<<<1024, 256, 0, s>>>(dw, d.N * d.K, db, db ? d.N : 0);
        return hipGetLastError();
    }
    Prod g{};
    g.a = dz;
    g.b = x;
    g.lda = pad16(d.N, es) * es;
    g.ldb = pad16(d.K, es) * es;
    Prep prep{};
    if (p.pad_a != (size_t)-1) add_prep(prep, dz, nullptr, base + p.pad_a, d.M, d.N * es, es), g.a = base + p.pad_a;
    if (p.pad_b != (size_t)-1) {  // odd rows, or MX8 codes to unpack
        add_prep(prep, x, d.x_mx8 ? x_sc : nullptr, base + p.pad_b, d.M, d.x_mx8 ? d.K : d.K * es, es);
        g.b = base + p.pad_b;
    }
    if ((e = launch_prep(prep, d.dtype, s)) != hipSuccess) return e;
    g.rows = d.N;
    g.cols = (int)d.K;
    g.R = d.M;
    g.part = p.splits > 1 ? (float*)(base + p.part) : nullptr;
    if (db) {
        g.db = p.splits > 1 ? (float*)(base + p.db_part) : db;
        g.db_add = accumulate && p.splits == 1;
        g.epi.db_part = p.splits > 1 ? g.db : nullptr;
        g.epi.db = db;
        g.epi.db_add = accumulate;
    }
    g.epi.out = dw;
    g.epi.residual = accumulate ? dw : nullptr;
    g.epi.rows = d.N;
    g.epi.cols = (int)d.K;
    if (d.dtype == DT_BF16) return launch_sides<Bf16Op, true, true, float>(p, g, s);
    return launch_sides<F32Op, true, true, float>(p, g, s);
}

}  // namespace convmi
