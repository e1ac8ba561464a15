// k_mx8.hip -- activations kept in 8 bits (format: mx8.hpp): packing, unpacking and the
// activation derivative taken at the kept values.
//
//   pack      top = max |v| over the block's finite values; e = scale byte of top;
//             code = e4m3(v * 2^(127-e)), nearest even
//   unpack    v = e4m3(code) * 2^(e-127), exact in fp32 and (above 2^-126) in bf16
//   backward  dz = act'(v) * dy, act' at v = z or written in terms of v = y
//
// All three are one pass over memory: per value, pack moves 2 (bf16) or 4 bytes in and
// 1 + 1/32 out, unpack the reverse, the derivative 1 + 1/32 + es in and es out; HBM is
// the bound.  8192 x 4096 bf16, from HBM: pack 20.8 us (4.9 TB/s), unpack 20.9 (4.9), GELU
// derivative 34-37 (4.6-4.9); a plain 1 GiB copy runs at 5.1.  On tensors that stay in the
// last-level cache 16.8 (6.0), 16.6 (6.1) and 29.8 (5.7).  A lane holds 8
// consecutive values of a row (16 bytes of bf16, 8 of codes, so a wave's accesses are whole
// cache lines), the four lanes of a block agree on the scale with two DPP exchanges, and
// the first of them stores it.
#include "internal.hpp"
#include "mx8.hpp"

namespace convmi {
namespace {

constexpr int kThreads = 256;

// Pieces of a [rows][cols] tensor, kPiece values each; a row has 4 * ceil(cols/32) of
// them, so that a block's four pieces sit in four neighbouring lanes.  With whole blocks
// (cols % 32 == 0) piece p covers values 8p.. of the flat tensor and no division is due.
struct Pieces {
    int64_t count;
    int cols, per_row, nb;
    int flat;     // cols % 32 == 0
    FastDiv fdr;  // by per_row, for counts below 2^31
};
Pieces make_pieces(int64_t rows, int cols) {
    const int nb = (int)ceil_div(cols, kMxBlock), per_row = nb * (kMxBlock / kPiece);
    return Pieces{rows * per_row, cols, per_row, nb, cols % kMxBlock == 0, make_fastdiv((uint32_t)per_row)};
}

struct PackOp {
    const void* x;
    uint8_t *q, *scales;
    template <typename T> __device__ __forceinline__ void run(int64_t at, int64_t sc, int n, bool first) const {
        float v[kPiece];
        load_piece((const T*)x + at, n, v);
        uint32_t e;
        const uint2 c = mx_pack(v, e);
        if (n > 0) store_codes(q + at, n, c);
        if (first) scales[sc] = (uint8_t)e;
    }
};
struct UnpackOp {
    const uint8_t *q, *scales;
    void* x;
    template <typename T> __device__ __forceinline__ void run(int64_t at, int64_t sc, int n, bool) const {
        if (n <= 0) return;
        float v[kPiece];
        mx_decode(load_codes(q + at, n), mx_scale(scales[sc]), v);
        store_piece((T*)x + at, n, v);
    }
};
template <int ACT, bool FROM_OUT> struct ActBwdOp {
    const uint8_t *q, *scales;
    const void* dy;  // may be dz
    void* dz;
    template <typename T> __device__ __forceinline__ void run(int64_t at, int64_t sc, int n, bool) const {
        if (n <= 0) return;
        float v[kPiece], g[kPiece];
        load_piece((const T*)dy + at, n, g);
        mx_decode(load_codes(q + at, n), mx_scale(scales[sc]), v);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) g[j] *= FROM_OUT ? act_slope_out<ACT>(v[j]) : act_slope<ACT>(v[j]);
        store_piece((T*)dz + at, n, g);
    }
};

template <typename T, class Op> __global__ __launch_bounds__(kThreads) void mx_pieces(Op op, Pieces g) {
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t p = (int64_t)blockIdx.x * kThreads + threadIdx.x; p < g.count; p += step) {
        const bool first = (threadIdx.x & 3) == 0;
        if (g.flat) {
            op.template run<T>(p * kPiece, p >> 2, kPiece, first);
        } else {
            const int64_t row = g.count < (1LL << 31) ? (int64_t)fdiv((int)p, g.fdr) : p / g.per_row;
            const int i = (int)(p - row * g.per_row);
            op.template run<T>(row * g.cols + i * kPiece, row * g.nb + (i >> 2), g.cols - i * kPiece, first);
        }
    }
}

template <class Op> hipError_t launch_pieces(int dt, const Op& op, int64_t rows, int cols, hipStream_t s) {
    if (rows == 0) return hipSuccess;
    const Pieces g = make_pieces(rows, cols);
    const int64_t blocks = ceil_div(g.count, kThreads);
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192)), block(kThreads);
    if (dt == DT_BF16)
        mx_pieces<bf16><<<grid, block, 0, s>>>(op, g);
    else
        mx_pieces<float><<<grid, block, 0, s>>>(op, g);
    return hipGetLastError();
}

// Rows copied to a pitch of whole 16-byte chunks, or unpacked (see PrepSeg): one chunk per
// thread, one pass over memory (8192 x 4096 MX8 to bf16: 20.9 us in a trace, 4.9 TB/s).
template <typename T> __global__ __launch_bounds__(kThreads) void prep_rows(Prep p) {
    constexpr int VEC = 16 / (int)sizeof(T);
    for (int i = 0; i < p.n; ++i) {
        const PrepSeg& g = p.seg[i];
        for (int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x; c < g.chunks; c += (int64_t)gridDim.x * kThreads) {
            const int64_t row = g.chunks < (1LL << 31) ? (int64_t)fdiv((int)c, g.fdr) : c / g.per_row;
            const int k = (int)(c - row * g.per_row);
            const char* src = g.src + row * g.row_bytes;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            const int at = k * (g.scales ? VEC : 16), left = g.row_bytes - at;
            if (c >= g.src_chunks || left <= 0) {  // behind the last row, or behind a row's end
            } else if (g.scales) {                 // codes
                uint2 q = make_uint2(0u, 0u);
                if (left >= VEC) {
                    __builtin_memcpy(&q, src + at, VEC);
                } else {
#pragma unroll
                    for (int b = 0; b < VEC; ++b)
                        if (b < left) (b < 4 ? q.x : q.y) |= (uint32_t)(uint8_t)src[at + b] << (8 * (b & 3));
                }
                float f[kPiece];
                mx_decode(q, mx_scale(g.scales[row * g.nb + at / kMxBlock]), f);
                if constexpr (VEC == 8)
                    v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                   pack_bf16x2(f[6], f[7]));
                else
                    v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                   __float_as_uint(f[3]));
                if (left < VEC) {  // zeros behind the row whatever its last scale is
                    uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int b = 0; b < VEC; ++b)
                        if (b >= left) d[b * (int)sizeof(T) / 4] &= VEC == 8 && !(b & 1) ? 0xffff0000u : VEC == 8 ? 0x0000ffffu : 0u;
                    v = make_uint4(d[0], d[1], d[2], d[3]);
                }
            } else {
                if (left >= 16) {
                    __builtin_memcpy(&v, src + at, 16);
                } else {
                    uint32_t d[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int b = 0; b < 16; ++b)
                        if (b < left) d[b >> 2] |= (uint32_t)(uint8_t)src[at + b] << (8 * (b & 3));
                    v = make_uint4(d[0], d[1], d[2], d[3]);
                }
            }
            *(uint4*)(g.dst + c * 16) = v;
        }
    }
}

// The reverse: the first `cols` of every `pitch` values, copied or added to what is there.
template <typename T> __device__ __forceinline__ void compact(const CompactSeg& g) {
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < g.rows * g.cols; i += (int64_t)gridDim.x * kThreads) {
        const int64_t row = i / g.cols;
        const T v = ((const T*)g.src)[row * g.pitch + (i - row * g.cols)];
        T* o = (T*)g.dst + i;
        *o = g.add ? from_f32<T>(to_f32(*o) + to_f32(v)) : v;
    }
}
__global__ __launch_bounds__(kThreads) void compact_rows(Compact p) {
    for (int i = 0; i < p.n; ++i) {
        if (p.seg[i].dt == DT_BF16) compact<bf16>(p.seg[i]);
        else compact<float>(p.seg[i]);
    }
}

}  // namespace

void add_prep(Prep& p, const void* src, const void* scales, void* dst, int64_t rows, int64_t row_bytes, int es,
              int64_t pitch, int64_t zero_rows) {
    const int per_row = (int)ceil_div(pitch ? pitch : scales ? row_bytes * es : row_bytes, 16);
    p.seg[p.n++] = PrepSeg{(const char*)src, (const uint8_t*)scales, (char*)dst, (rows + zero_rows) * per_row,
                           rows * per_row, (int)row_bytes, per_row, (int)ceil_div(row_bytes, kMxBlock),
                           make_fastdiv((uint32_t)per_row)};
}
hipError_t launch_prep(const Prep& p, int dt, hipStream_t s) {
    int64_t most = 0;
    for (int i = 0; i < p.n; ++i) most = p.seg[i].chunks > most ? p.seg[i].chunks : most;
    if (most == 0) return hipSuccess;
    const int64_t n = ceil_div(most, kThreads);
    const unsigned blocks = (unsigned)(n < 8192 ? n : 8192);
    if (dt == DT_BF16) prep_rows<bf16><<<blocks, kThreads, 0, s>>>(p);
    else prep_rows<float><<<blocks, kThreads, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_compact(const Compact& p, hipStream_t s) {
    int64_t most = 1;
    for (int i = 0; i < p.n; ++i) most = p.seg[i].rows * p.seg[i].cols > most ? p.seg[i].rows * p.seg[i].cols : most;
    const int64_t n = ceil_div(most, kThreads);
    compact_rows<<<(unsigned)(n < 8192 ? n : 8192), kThreads, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_mx8_pack(int dt, const void* x, int64_t rows, int cols, void* q, void* scales, hipStream_t s) {
    return launch_pieces(dt, PackOp{x, (uint8_t*)q, (uint8_t*)scales}, rows, cols, s);
}

hipError_t launch_mx8_unpack(int dt, const void* q, const void* scales, int64_t rows, int cols, void* x,
                             hipStream_t s) {
    return launch_pieces(dt, UnpackOp{(const uint8_t*)q, (const uint8_t*)scales, x}, rows, cols, s);
}

hipError_t launch_mx8_act_bwd(int dt, const void* q, const void* scales, int from_output, const void* dy, void* dz,
                              int64_t rows, int cols, int act, hipStream_t s) {
    if (from_output && act == ACT_GELU) return hipErrorInvalidValue;
    hipError_t e = hipSuccess;
    const uint8_t *qc = (const uint8_t*)q, *sc = (const uint8_t*)scales;
    CONVMI_ACT_SWITCH(act, A, {
        if (from_output)
            e = launch_pieces(dt, ActBwdOp<A, true>{qc, sc, dy, dz}, rows, cols, s);
        else
            e = launch_pieces(dt, ActBwdOp<A, false>{qc, sc, dy, dz}, rows, cols, s);
    });
    return e;
}

}  // namespace convmi
