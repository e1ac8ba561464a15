// lane_sums.hpp -- cross-lane sums of a wave64, shared by the reduction kernels.
#pragma once

#include "common.hpp"

namespace convmi {
namespace {

// ---------------------------------------------------------------- cross-lane sums
// Lanes l and l + k of a wave64 exchange values without LDS memory: rotations within
// 16-lane rows through DPP (row_ror), the two halves of each 32-lane group through
// ds_swizzle (bit mode, xor 16), the two 32-lane halves through ds_bpermute (xor 32).
__device__ __forceinline__ float dpp_ror(float v, int k) {  // k in {1, 2, 4, 8}; lane i gets lane (i + k) % 16 of its row
    const int x = __builtin_bit_cast(int, v);
    int r;
    switch (k) {
    case 8: r = __builtin_amdgcn_update_dpp(0, x, 0x128, 0xf, 0xf, false); break;
    case 4: r = __builtin_amdgcn_update_dpp(0, x, 0x124, 0xf, 0xf, false); break;
    case 2: r = __builtin_amdgcn_update_dpp(0, x, 0x122, 0xf, 0xf, false); break;
    default: r = __builtin_amdgcn_update_dpp(0, x, 0x121, 0xf, 0xf, false); break;
    }
    return __builtin_bit_cast(float, r);
}
__device__ __forceinline__ float lane_xor16(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), (0x10 << 10) | 0x1f));
}
__device__ __forceinline__ float lane_xor32(float v) {
    const int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    return __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute((lane ^ 32) << 2, __builtin_bit_cast(int, v)));
}

// Sum over the lanes of a wave congruent modulo `stride` (a power of two <= 64): every
// lane ends with the sum of its class.  Each lane adds the same terms in the same
// pairing (IEEE addition is commutative), so all lanes of a class agree bit for bit and
// the result depends only on the data.
__device__ __forceinline__ float wave_class_sum(float v, int stride) {
    for (int k = 8; k >= stride && k >= 1; k >>= 1) v += dpp_ror(v, k);
    if (stride <= 16) v += lane_xor16(v);
    if (stride <= 32) v += lane_xor32(v);
    return v;
}

}  // namespace
}  // namespace convmi
