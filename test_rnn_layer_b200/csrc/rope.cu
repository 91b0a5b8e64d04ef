// Rotary positions: y0 = A (x0 cos u - x1 sin u), y1 = A (x0 sin u + x1 cos u)
// for each pair of a head's first `rot` columns, u = position * frequency.
//
// The angle is taken in turns: position * turns[i] in 64 bits, less its whole
// part, so that a far position (2^20 and more radians) keeps its angle: to
// 2^-31 turns or better there, to 2^-26 once the rest, at most half a turn, is
// cast to fp32 for sinpi/cospi.  One angle serves every head
// of a row, so a block first fills a table of cos and sin for its rows in
// shared memory and then streams the heads past it, 16 bytes at a time and
// three units a thread under way while the table is made.  Bound by memory:
// each element is read and written once.
//
// A unit is what one thread turns at once: two 16-byte pieces, the pairs'
// halves (HALF layout) or two neighbouring pieces of whole pairs.  Layouts
// whose pieces do not fall on 16 bytes (rot / 2 or rot no multiple of the
// piece) go pair by pair.
#include "common.cuh"

namespace ttt {
namespace {

constexpr int kThreads = 128, kMaxRows = 8, kBatch = 3;   // 72 us for 32,768 x 48 heads; 256 x 4 and 128 x 6: 78

__device__ __forceinline__ void fill_table(const RopeArgs& p, int t0, int rows, float2* cs) {
    const int pairs = p.rot / 2;
    for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
        const int r = i / pairs, j = i - r * pairs;
        const long long pos = p.positions ? p.positions[t0 + r] : p.pos0 + t0 + r;
        const double u = (double)pos * p.turns[j];
        float sn, c;
        sincospif(2.f * (float)(u - rint(u)), &sn, &c);
        cs[i] = make_float2(p.amplitude * c, p.amplitude * (p.inverse ? -sn : sn));
    }
}

// Piece: 16 bytes as fp32 values
template <bool BF>
struct Piece {
    static constexpr int N = BF ? 8 : 4;
    static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[N]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF) {
                v[2 * i] = __uint_as_float(u[i] << 16);
                v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            } else {
                v[i] = __uint_as_float(u[i]);
            }
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[N]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
                u[i] = __float_as_uint(v[i]);
            }
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

// rows [t0, t0 + rows) of a block; `turned` units a head, then `copied` pieces behind the turned columns
template <bool BF, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs p, int block_rows, int turned, int copied) {
    constexpr int N = Piece<BF>::N, E = BF ? 2 : 4;
    extern __shared__ float2 cs[];
    const int t0 = blockIdx.x * block_rows, rows = min(block_rows, p.T - t0), pairs = p.rot / 2;
    const int per_head = turned + copied, per_row = p.H * per_head, units = rows * per_row;
    const char* X = static_cast<const char*>(p.X) + (long long)t0 * p.ld_x * E;
    char* Y = static_cast<char*>(p.Y) + (long long)t0 * p.ld_y * E;
    // a unit's row, its first column in the row, the second piece's distance and its first pair (-1: to copy)
    struct Unit {
        int r, col, second, pair;
    };
    auto unit_of = [&](int u) {
        Unit q;
        q.r = u / per_row;
        const int in_row = u - q.r * per_row, h = in_row / per_head, k = in_row - h * per_head;
        if (k < turned) {
            q.col = h * p.d + (HALF ? k * N : 2 * k * N);
            q.second = HALF ? pairs : N;
            q.pair = k * N;
            if (!HALF && 2 * k * N + N >= p.rot) q.second = 0;   // the last piece of an odd number
        } else {
            q.col = h * p.d + p.rot + (k - turned) * N;
            q.second = 0;
            q.pair = -1;
        }
        return q;
    };
    bool made = false;
    for (int u0 = threadIdx.x; u0 - threadIdx.x < units; u0 += kBatch * kThreads) {
        uint4 a[kBatch], b[kBatch];
        Unit q[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int u = u0 + i * kThreads;
            if (u < units) {
                q[i] = unit_of(u);
                const char* x = X + (q[i].r * p.ld_x + q[i].col) * E;
                a[i] = __ldcs(reinterpret_cast<const uint4*>(x));
                if (q[i].second) b[i] = __ldcs(reinterpret_cast<const uint4*>(x + q[i].second * E));
            }
        }
        if (!made) {
            fill_table(p, t0, rows, cs);
            __syncthreads();
            made = true;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int u = u0 + i * kThreads;
            if (u >= units) continue;
            char* y = Y + (q[i].r * p.ld_y + q[i].col) * E;
            if (q[i].pair >= 0) {
                const float2* w = cs + q[i].r * pairs + q[i].pair;
                float v0[N], v1[N];
                Piece<BF>::unpack(a[i], v0);
                if (q[i].second) Piece<BF>::unpack(b[i], v1);
                if constexpr (HALF) {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float x0 = v0[e], x1 = v1[e];
                        v0[e] = x0 * w[e].x - x1 * w[e].y;
                        v1[e] = x0 * w[e].y + x1 * w[e].x;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < N; e += 2) {
                        const float x0 = v0[e], x1 = v0[e + 1];
                        const float2 c = w[e / 2];
                        v0[e] = x0 * c.x - x1 * c.y;
                        v0[e + 1] = x0 * c.y + x1 * c.x;
                    }
                    if (q[i].second) {
#pragma unroll
                        for (int e = 0; e < N; e += 2) {
                            const float x0 = v1[e], x1 = v1[e + 1];
                            const float2 c = w[(N + e) / 2];
                            v1[e] = x0 * c.x - x1 * c.y;
                            v1[e + 1] = x0 * c.y + x1 * c.x;
                        }
                    }
                }
                a[i] = Piece<BF>::pack(v0);
                if (q[i].second) b[i] = Piece<BF>::pack(v1);
            }
            __stcs(reinterpret_cast<uint4*>(y), a[i]);
            if (q[i].second) __stcs(reinterpret_cast<uint4*>(y + q[i].second * E), b[i]);
        }
    }
}

// Pair by pair, for layouts whose pieces do not fall on 16 bytes.
__global__ void __launch_bounds__(kThreads) rope_pairs_kernel(const __grid_constant__ RopeArgs p) {
    const int pairs = p.rot / 2, units = p.H * p.d / 2, rest = (p.d - p.rot) / 2;
    __shared__ float2 cs[kRopeMaxPairs];
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        fill_table(p, t, 1, cs);
        __syncthreads();
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
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    LaunchScope scope("rope", s);
    const int n = a.bf16 ? 8 : 4;
    // strides are multiples of 8 elements and d of 8, so only the split columns can fall off 16 bytes
    const bool pieces = a.half ? a.rot / 2 % n == 0 : a.rot % n == 0;
    if (!pieces) {
        rope_pairs_kernel<<<min(a.T, sms * 8), kThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    const int turned = a.half ? a.rot / 2 / n : (a.rot / n + 1) / 2;
    const int copied = a.X == a.Y ? 0 : (a.d - a.rot) / n;
    // rows of a block: enough for three units a thread, fewer where blocks would be short of the SMs
    int rows = 1;
    while (rows < kMaxRows && (long long)rows * a.H * (turned + copied) < kBatch * kThreads && a.T / (2 * rows) >= 2 * sms) rows *= 2;
    const unsigned grid = (unsigned)((a.T + rows - 1) / rows);
    const size_t smem = (size_t)rows * (a.rot / 2) * sizeof(float2);
    if (a.bf16) {
        if (a.half) rope_kernel<true, true><<<grid, kThreads, smem, s>>>(a, rows, turned, copied);
        else rope_kernel<true, false><<<grid, kThreads, smem, s>>>(a, rows, turned, copied);
    } else {
        if (a.half) rope_kernel<false, true><<<grid, kThreads, smem, s>>>(a, rows, turned, copied);
        else rope_kernel<false, false><<<grid, kThreads, smem, s>>>(a, rows, turned, copied);
    }
    return cudaGetLastError();
}

}  // namespace ttt
