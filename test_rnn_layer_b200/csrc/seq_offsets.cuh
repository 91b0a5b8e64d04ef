// Packed sequences on the device: offsets cu[0..n] cut to the array they index.
#pragma once

#include "internal.h"

namespace ttt {

struct SeqOffsets {
    const int* cu;   // device, or null: one sequence of every row
    int n, rows;

    __device__ __forceinline__ int begin(int s) const {
        return cu ? min(max(__ldg(cu + s), 0), rows) : (s ? rows : 0);
    }
    // the last s in [0, n) with begin(s) <= t: t's sequence if t < begin(s + 1) (empty ones share their start
    // with the sequence after them)
    __device__ __forceinline__ int find(int t) const {
        int lo = 0, hi = n - 1;
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (begin(mid) <= t) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
    // whether offset s is out of order or out of the array (s in [0, n])
    __device__ __forceinline__ bool bad(int s) const {
        if (!cu) return false;
        const int v = __ldg(cu + s);
        return v < 0 || v > rows || (s == 0 ? v != 0 : v < __ldg(cu + s - 1));
    }
};

}  // namespace ttt
