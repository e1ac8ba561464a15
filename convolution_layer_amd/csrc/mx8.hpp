// mx8.hpp -- the 8-bit activation format and the row pieces that its kernels work on.
//
// MX8 holds a [rows][cols] tensor as one e4m3 code per value (sign, 4 exponent bits of
// bias 7, 3 mantissa bits; largest finite 448; 0x7f and 0xff are NaN; no infinities) and
// one scale byte e per 32 consecutive values of a row, standing for 2^(e-127).  Packing
// takes the smallest power of two that brings the block's largest finite magnitude to
// 448 or below, so no finite value saturates and each value that is not subnormal in its
// block is off by at most 2^-4 of itself (half a unit in the last of 4 significant bits).
// Powers of two make scaling exact; 32-value blocks along the row are what the scaled
// MFMA instructions take directly.
#pragma once

#include "common.hpp"

namespace convmi {
namespace {

constexpr int kMxBlock = 32;
constexpr int kPiece = 8;  // consecutive values a lane holds; four lanes hold a block

// Eight values from / to memory at any element alignment (gfx950 global accesses may be
// unaligned; the copies become 16-byte loads and stores), or the first n of them.
template <typename T> struct RawPiece {  // as loaded: 32 bytes of fp32, 16 of bf16
    uint32_t u[kPiece * sizeof(T) / 4];
};
template <typename T> __device__ __forceinline__ RawPiece<T> load_raw(const T* p, int n) {
    RawPiece<T> w;
    if (n >= kPiece) {
        __builtin_memcpy(&w, p, sizeof(w));
        return w;
    }
#pragma unroll
    for (int i = 0; i < (int)(sizeof(w) / 4); ++i) w.u[i] = 0u;
#pragma unroll
    for (int j = 0; j < kPiece; ++j)
        if (j < n) {
            if constexpr (sizeof(T) == 4) w.u[j] = __float_as_uint(p[j]);
            else w.u[j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
        }
    return w;
}
__device__ __forceinline__ void widen(const RawPiece<float>& w, float (&v)[kPiece]) {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) v[j] = __uint_as_float(w.u[j]);
}
__device__ __forceinline__ void widen(const RawPiece<bf16>& w, float (&v)[kPiece]) {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) v[j] = __uint_as_float(j & 1 ? w.u[j / 2] & 0xffff0000u : w.u[j / 2] << 16);
}
template <typename T> __device__ __forceinline__ void load_piece(const T* p, int n, float (&v)[kPiece]) {
    widen(load_raw(p, n), v);
}
template <typename T> __device__ __forceinline__ void store_piece(T* p, int n, const float (&v)[kPiece]);
template <> __device__ __forceinline__ void store_piece<float>(float* p, int n, const float (&v)[kPiece]) {
    if (n >= kPiece) {
        __builtin_memcpy(p, v, sizeof(v));
    } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (j < n) p[j] = v[j];
    }
}
template <> __device__ __forceinline__ void store_piece<bf16>(bf16* p, int n, const float (&v)[kPiece]) {
    if (n >= kPiece) {
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        __builtin_memcpy(p, r, sizeof(r));
    } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (j < n) p[j] = f32_to_bf16(v[j]);
    }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int n) {
    uint2 c = make_uint2(0u, 0u);
    if (n >= kPiece) {
        __builtin_memcpy(&c, p, sizeof(c));
    } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (j < n) (j < 4 ? c.x : c.y) |= (uint32_t)p[j] << (8 * (j & 3));
    }
    return c;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint2 c) {
    if (n >= kPiece) {
        __builtin_memcpy(p, &c, sizeof(c));
    } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (j < n) p[j] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
    }
}

// Largest of four neighbouring lanes' unsigned values (the lanes of one block).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true);  // lanes 1,0,3,2
    v = v > o ? v : o;
    o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true);  // lanes 2,3,0,1
    return v > o ? v : o;
}

// Bits of the largest finite magnitude among a lane's values (0 if none).
__device__ __forceinline__ uint32_t top_bits(const float (&v)[kPiece]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
        uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
        b = b < 0x7f800000u ? b : 0u;
        m = m > b ? m : b;
    }
    return m;
}

// Scale byte for a block whose largest finite magnitude has these bits: 448 = 1.75 * 2^8,
// so with top = 1.f * 2^x the power is 2^(x-8), one more where 1.f > 1.75 (the addition
// carries into the exponent exactly then).  At least 1, so that the scale and its
// reciprocal (254 - e; e <= 247) are normal float32 numbers; blocks below 448 * 2^-126
// lie on the coarser grid of 2^-126.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
    const int e = (int)((top + 0x1FFFFFu) >> 23) - 8;
    return (uint32_t)(e > 1 ? e : 1);
}
// Codes of eight values under scale byte e: round to nearest even; infinities and NaN
// become the NaN code (the format has no infinity).  Under the largest scale that packing
// chooses, 2^120, 256 would stand for 2^128, beyond fp32: the top magnitudes are kept as
// 240 * 2^120 there (still within 2^-4 of themselves), so that finite values stay finite.
__device__ __forceinline__ uint2 mx_encode(const float (&v)[kPiece], uint32_t e) {
    const float inv = __uint_as_float((254u - e) << 23);
    const float lim = e < 247u ? 448.0f : 240.0f;
    float u[kPiece];
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
        const bool fin = (__float_as_uint(v[j]) & 0x7fffffffu) < 0x7f800000u;
        u[j] = fin ? __builtin_amdgcn_fmed3f(v[j] * inv, -lim, lim) : __uint_as_float(0x7fc00000u);
    }
    uint2 c;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], 0, false);
    c.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(u[2], u[3], w, true);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(u[4], u[5], 0, false);
    c.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(u[6], u[7], w, true);
    return c;
}
// Scale byte and codes of eight values, in whole groups of four lanes that hold a block.
// The magnitudes' bits order like the magnitudes, so one integer maximum finds the top and
// shows whether anything is infinite, NaN or close to fp32's limit; only such blocks take
// the checked path (the 8-bit pre-activations of an 8192 x 4096 product: 3.4 vector
// instructions a value instead of 10).
__device__ __forceinline__ uint2 mx_pack(const float (&v)[kPiece], uint32_t& e) {
    uint32_t b[kPiece];
#pragma unroll
    for (int j = 0; j < kPiece; ++j) b[j] = __float_as_uint(v[j]) & 0x7fffffffu;
    uint32_t top = b[0];
#pragma unroll
    for (int j = 1; j < kPiece; ++j) top = top > b[j] ? top : b[j];
    top = quad_max(top);
    if (top > 0x7f600000u) {  // a scale byte of 247 or more, or not finite
        e = mx_scale_byte(quad_max(top_bits(v)));
        return mx_encode(v, e);
    }
    e = mx_scale_byte(top);
    const float inv = __uint_as_float((254u - e) << 23);
    uint2 c;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    c.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, w, true);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, 0, false);
    c.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, w, true);
    return c;
}
// 2^(e-127) for any scale byte: 0 is the subnormal 2^-127, 255 stands for NaN.
__device__ __forceinline__ float mx_scale(uint32_t e) {
    const uint32_t b = e << 23;
    return __uint_as_float(e == 0u ? 0x00400000u : e == 255u ? 0x7fc00000u : b);
}
__device__ __forceinline__ void mx_decode(uint2 c, float s, float (&v)[kPiece]) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true);
    const f2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false), f = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
    v[0] = a.x * s; v[1] = a.y * s; v[2] = b.x * s; v[3] = b.y * s;
    v[4] = d.x * s; v[5] = d.y * s; v[6] = f.x * s; v[7] = f.y * s;
}

}  // namespace
}  // namespace convmi
