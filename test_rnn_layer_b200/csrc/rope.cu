// Rotary positions: y0 = A (x0 cos u - x1 sin u), y1 = A (x0 sin u + x1 cos u)
// for each pair of a head's first `rot` columns, u = position * frequency.
//
// The angle is taken in turns: position * turns[i] in 64 bits, less its whole
// part, so that a far position (2^20 and more radians) keeps its angle to
// 2^-31 turns; the rest is sinpi/cospi in fp32.  One angle serves every head
// of a row, so a block first fills a table of cos and sin for its rows in
// shared memory and then streams the heads past it.
#include "common.cuh"

namespace ttt {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs p) {
    const int pairs = p.rot / 2, units = p.H * p.d / 2;
    __shared__ float2 cs[kRopeMaxPairs];
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        const long long pos = p.positions ? p.positions[t] : p.pos0 + t;
        for (int i = threadIdx.x; i < pairs; i += kThreads) {
            const double u = (double)pos * p.turns[i];
            const float r = (float)(u - rint(u));
            float sn, c;
            sincospif(2.f * r, &sn, &c);
            cs[i] = make_float2(p.amplitude * c, p.amplitude * (p.inverse ? -sn : sn));
        }
        __syncthreads();
        const int rest = (p.d - p.rot) / 2;
        for (int k = threadIdx.x; k < units; k += kThreads) {
            const int h = k / (p.d / 2), i = k - h * (p.d / 2);
            int j0, j1;
            if (i < pairs) {
                j0 = p.half ? i : 2 * i;
                j1 = p.half ? i + pairs : 2 * i + 1;
            } else {
                j0 = p.rot + (i - pairs);
                j1 = j0 + rest;
            }
            const long long x = t * p.ld_x + h * p.d, y = t * p.ld_y + h * p.d;
            const float a = load_elem(p.X, x + j0, p.bf16), b = load_elem(p.X, x + j1, p.bf16);
            const float2 w = i < pairs ? cs[i] : make_float2(1.f, 0.f);
            store_elem(p.Y, y + j0, p.bf16, i < pairs ? a * w.x - b * w.y : a);
            store_elem(p.Y, y + j1, p.bf16, i < pairs ? a * w.y + b * w.x : b);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
    LaunchScope scope("rope", s);
    rope_kernel<<<min(a.T, 148 * 8), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ttt
