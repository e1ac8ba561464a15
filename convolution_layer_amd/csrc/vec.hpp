// vec.hpp -- V consecutive values of a row at any element alignment, or the first n of them.
#pragma once

#include "common.hpp"

namespace convmi {
namespace {

template <typename T, int V> struct Vec {  // as loaded
    uint32_t u[V * sizeof(T) / 4];
};
// gfx950 global accesses may be unaligned; the copies become loads and stores of up to 16 bytes.
template <typename T, int V> __device__ __forceinline__ Vec<T, V> load_vec(const T* p, int n) {
    Vec<T, V> w;
    if (n >= V) {
        __builtin_memcpy(&w, p, sizeof(w));
        return w;
    }
#pragma unroll
    for (int i = 0; i < (int)(sizeof(w) / 4); ++i) w.u[i] = 0u;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < n) {
            if constexpr (sizeof(T) == 4) w.u[j] = __float_as_uint(p[j]);
            else w.u[j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
        }
    return w;
}
template <typename T, int V> __device__ __forceinline__ void widen(const Vec<T, V>& w, float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if constexpr (sizeof(T) == 4) v[j] = __uint_as_float(w.u[j]);
        else v[j] = __uint_as_float(j & 1 ? w.u[j / 2] & 0xffff0000u : w.u[j / 2] << 16);
    }
}
template <typename T, int V> __device__ __forceinline__ void load_wide(const T* p, int n, float (&v)[V]) {
    widen<T, V>(load_vec<T, V>(p, n), v);
}
template <typename T, int V> __device__ __forceinline__ void store_vec(T* p, int n, const float (&v)[V]) {
    if (n >= V) {
        Vec<T, V> w;
#pragma unroll
        for (int i = 0; i < (int)(sizeof(w) / 4); ++i) {
            if constexpr (sizeof(T) == 4) w.u[i] = __float_as_uint(v[i]);
            else w.u[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        }
        __builtin_memcpy(p, &w, sizeof(w));
        return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < n) p[j] = from_f32<T>(v[j]);
}

}  // namespace
}  // namespace convmi
