// Work items of the window attention kernels: blocks of a sequence's rows and the tiles of the other side
// that they meet, found on the device from the packed offsets.
#pragma once

#include "seq_offsets.cuh"

namespace ttt {
namespace win {

// Sequence s of an array has at most floor(rows_s / R) + 1 blocks of R rows; counting from
// begin(s) / R + s gives every sequence enough numbers without a pass over the offsets (some stay unused).
template <int R>
__host__ __device__ inline long long block_numbers(long long rows, long long n_seq) { return rows / R + n_seq; }

// The sequence that owns block number b, or -1 where the number is unused; `first` is the block's first row.
template <int R>
__device__ __forceinline__ int block_of(const SeqOffsets& c, int b, int& first, int& rows) {
    int lo = 0, hi = c.n - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (c.begin(mid) / R + mid <= b) lo = mid;
        else hi = mid - 1;
    }
    const int r0 = c.begin(lo), r1 = c.begin(lo + 1);
    const int k = b - (r0 / R + lo);
    if (k < 0 || r1 - r0 <= k * R) return -1;
    first = r0 + k * R;
    rows = min(R, r1 - first);
    return lo;
}

// n low bits (n may lie outside 0..32)
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Keys that a block of query rows sees: the first `sk` keys of its sequence (sinks in front of the window)
// and the window's [lo, hi).  Positions and keys count from the sequence's start.
struct KeyRange {
    int sk, lo, hi;
};
__device__ __forceinline__ KeyRange keys_of(int pos0, int rows, int nk, int left, int right, int sinks) {
    KeyRange r;
    r.lo = min(max(pos0 - left, 0), nk);
    r.hi = max(min(pos0 + rows + right, nk), r.lo);
    r.sk = min(sinks, r.lo);
    return r;
}

}  // namespace win
}  // namespace ttt
