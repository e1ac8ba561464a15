// seq.hpp -- sequences that lie one behind the other in the rows of a tensor, as the
// sequence-mixing kernels see them.
#pragma once

#include "common.hpp"

namespace convmi {

// Sequence i holds the rows starts[i] .. starts[i+1]-1, or without starts the i-th `len` rows.
// starts is device data that the host has not seen: every value is brought into [0, rows] before
// it becomes an address, so that no content of it leads out of a tensor.
struct Seqs {
    const int32_t* starts;
    int rows, batch, len;
};

// States of one-token calls: row r uses state slots[r] of `count`, without slots the r-th.
struct Slots {
    const int32_t* slots;
    int64_t count;
};

namespace {

__device__ __forceinline__ int seq_clamp(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }
__device__ __forceinline__ int seq_begin(const Seqs& q, int i) {
    return q.starts ? seq_clamp(q.starts[i], 0, q.rows) : i * q.len;
}
__device__ __forceinline__ int seq_end(const Seqs& q, int i, int begin) {
    return q.starts ? seq_clamp(q.starts[i + 1], begin, q.rows) : begin + q.len;
}

// Largest i in [0, n) with holds(i), which is true up to some i and false behind it; -1 if for
// none.  Whole waves call it with the same arguments: 64 candidates a round, one round for up
// to 64 sequences.
template <typename F> __device__ __forceinline__ int wave_last(int n, F holds) {
    const int lane = threadIdx.x & 63;
    int lo = 0;
    while (n > 64) {
        const int step = (n + 63) >> 6;
        const int at = lane * step;
        const int c = __builtin_popcountll(__ballot(at < n && holds(lo + at)));
        if (c == 0) return -1;
        lo += (c - 1) * step;
        n = n - (c - 1) * step < step ? n - (c - 1) * step : step;
    }
    const int c = __builtin_popcountll(__ballot(lane < n && holds(lo + lane)));
    return c == 0 ? -1 : lo + c - 1;
}

// The sequence that a row lies in or, between none, the last one that begins at or before it
// (-1: none does).  Whole waves, one row.
__device__ __forceinline__ int wave_seq_of_row(const Seqs& q, int row) {
    if (!q.starts) return row / q.len;
    return wave_last(q.batch, [&](int i) { return q.starts[i] <= row; });
}

// The state that a row of a one-token call uses: that of its slot, or the row's own without slots.
// Rows with a negative slot are padding; a slot that does not exist gives kSlotBad.
constexpr int kSlotNone = -1, kSlotBad = -2;
__device__ __forceinline__ int slot_of(const Slots& s, int row) {
    if (!s.slots) return row;
    const int v = s.slots[row];
    return v < 0 ? kSlotNone : v < s.count ? v : kSlotBad;
}
// Whether the row may not use its slot, because there is no such slot or an earlier row has taken it:
// two rows never touch one state.  All threads of the workgroup call it.
__device__ __forceinline__ bool slot_taken(const Slots& s, int row, int slot) {
    if (!s.slots) return false;
    int bad = slot == kSlotBad;
    for (int j = threadIdx.x; j < row; j += blockDim.x) bad |= s.slots[j] == slot;
    return __syncthreads_or(bad);
}
// The same of R rows from row0 on, a bit each.  flags: one int of the workgroup's LDS.
template <int R> __device__ __forceinline__ int slots_taken(const Slots& s, int row0, const int (&slot)[R], int* flags) {
    if (!s.slots) return 0;
    if (threadIdx.x == 0) *flags = 0;
    __syncthreads();
    int bad = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) bad |= (slot[r] == kSlotBad) << r;
    for (int j = threadIdx.x; j < row0; j += blockDim.x) {
        const int v = s.slots[j];
#pragma unroll
        for (int r = 0; r < R; ++r) bad |= (slot[r] >= 0 && v == slot[r]) << r;
    }
#pragma unroll
    for (int r = 1; r < R; ++r)
#pragma unroll
        for (int e = 0; e < r; ++e) bad |= (slot[r] >= 0 && slot[e] == slot[r]) << r;
    if (bad) atomicOr(flags, bad);
    __syncthreads();
    return *flags;
}

}  // namespace
}  // namespace convmi
