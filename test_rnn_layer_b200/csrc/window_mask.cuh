// The window's visibility rule, shared by the window attention kernels.
#pragma once

#include "seq_offsets.cuh"

namespace ttt {

// Query at position p (possibly negative: it sees nothing unless `right` reaches a key) and key u.
__device__ __forceinline__ bool window_sees(int p, int u, int left, int right, int sinks) {
    return u <= p + right && (u >= p - left || u < sinks);
}

}  // namespace ttt
