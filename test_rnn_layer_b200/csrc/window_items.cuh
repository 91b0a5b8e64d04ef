// Work items of the window attention kernels: blocks of a sequence's rows and the tiles of the other side
// that they meet, found on the device from the packed offsets.
#pragma once

#include "seq_offsets.cuh"
#include "tc_prims.cuh"

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

// The items a persistent CTA works on: its first is its own number, the others come from a counter in global memory
// (items differ in length, and a fixed share left some CTAs with 1.4 times the average).  The producer thread draws
// them and hands them to the CTA's other roles through four slots.
constexpr int kItemSlots = 4;
constexpr uint64_t kItemWait = 60000000000ull;   // ns: others may work on one item for long
struct ItemQueue {
    uint64_t *full, *empty;     // [kItemSlots] barriers: 1 arrival, and one of each taker
    volatile int* slot;         // [kItemSlots]
    const volatile int* abort;

    __device__ __forceinline__ void init(int takers) const {
        for (int s = 0; s < kItemSlots; ++s) {
            tc::mbar_init(full + s, 1);
            tc::mbar_init(empty + s, takers);
        }
    }
    // the n-th item of this CTA (-1: no more)
    __device__ __forceinline__ bool put(int n, int w) const {
        const int s = n % kItemSlots, use = n / kItemSlots;
        if (use > 0 && !tc::mbar_wait(empty + s, (use - 1) & 1, abort, kItemWait)) return false;
        slot[s] = w;
        tc::mbar_arrive(full + s);
        return true;
    }
    // by one thread; -2 where the wait ran out
    __device__ __forceinline__ int take(int n) const {
        const int s = n % kItemSlots, use = n / kItemSlots;
        if (!tc::mbar_wait(full + s, use & 1, abort, kItemWait)) return -2;
        const int w = slot[s];
        tc::mbar_arrive(empty + s);
        return w;
    }
    // by a warp
    __device__ __forceinline__ int take_warp(int n) const {
        const int s = n % kItemSlots, use = n / kItemSlots;
        const bool ok = tc::mbar_wait(full + s, use & 1, abort, kItemWait);
        if (!__all_sync(0xffffffffu, ok)) return -2;
        const int w = slot[s];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(empty + s);
        return w;
    }
};
// The order in which few blocks of unequal work are drawn: the longest first, so that the CTAs end together (forward
// pass of 13 requests of up to 1,725 rows, 12 heads, window 1,024: 60 -> 49 us).  Ranking them takes 2 to 4 us of a
// launch, so it is left out where blocks differ little: one sequence (16,384 rows, forward and backward: 580 us, 584
// with it), a narrow window (5 sequences, 256 keys to both sides: 148 us, 152 with it), and where every CTA has one item.
// A warp ranks up to kOrder blocks; with more, an item is a small part of a CTA's work.
// The window's width is a rough sign of unequal work.  On 13 requests of 20 to 760 rows behind up to 1,500 cached ones
// the order is worth nothing at 256 keys, and 8 us at 512 to 768, where it is not used (53 -> 45, 57 -> 47); short
// sequences under a wide window are all alike and pay for it (40 of 128 rows: forward 35 -> 39 us, backward 80 -> 84).
constexpr int kOrder = 128;
inline bool ordered(const WindowArgs& p, long long n_blocks, int ctas) {
    return n_blocks <= kOrder && n_blocks * p.Hq > ctas && p.n_seq > 1 && (long long)p.left + p.right >= 768;
}
// By a warp: block numbers by falling work(b) (-1: unused) into order[]; returns how many are used.
template <class Work>
__device__ __forceinline__ int order_blocks(uint8_t* order, int n, Work work) {
    const int lane = threadIdx.x & 31;
    int mine[kOrder / 32], rank[kOrder / 32], used = 0;
#pragma unroll
    for (int i = 0; i < kOrder / 32; ++i) {
        mine[i] = 32 * i + lane < n ? work(32 * i + lane) : -1;
        rank[i] = 0;
        used += __popc(__ballot_sync(0xffffffffu, mine[i] >= 0));
    }
#pragma unroll
    for (int k = 0; k < kOrder / 32; ++k) {
        if (32 * k >= n) break;
#pragma unroll 4
        for (int l = 0; l < min(32, n - 32 * k); ++l) {
            const int other = __shfl_sync(0xffffffffu, mine[k], l), b = 32 * k + l;
#pragma unroll
            for (int i = 0; i < kOrder / 32; ++i) {
                if (32 * i >= n) break;
                rank[i] += other >= mine[i] + (b >= 32 * i + lane);   // equal work: by number
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kOrder / 32; ++i)
        if (mine[i] >= 0) order[rank[i]] = (uint8_t)(32 * i + lane);
    __syncwarp();
    return used;
}

}  // namespace win
}  // namespace ttt
