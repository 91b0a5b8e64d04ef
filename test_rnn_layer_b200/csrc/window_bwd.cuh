// Parts shared by the two kernels of the window attention's backward pass.
#pragma once

#include "attn_prims.cuh"
#include "internal.h"
#include "window_items.cuh"

namespace ttt {
namespace winb {

using namespace attn;

constexpr int DH = 64, BT = 128, HALF = 64, TILE = BT * DH * 2;
// Sixteen softmax warps (four per scheduler; eight, with 64 scores a thread, left 60% of the issue slots empty) and
// four others.  A thread holds COLS scores and as many products.
constexpr int SOFT = 16, THREADS = 32 * (SOFT + 4), COLS = 32;
constexpr int EMU = 1;          // pairs of every 8 whose 2^x runs on the FMA pipe
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 2^x0, 2^x1 on the FMA pipe: fma_exp2.cuh's cubic (relative error 7.6e-5, 25 times below the bf16
// rounding P and dS get) on a pair.
__device__ __forceinline__ void ex2_poly2(uint64_t x, float& p0, float& p1) {
    ex2_cubic2(x, fexp::kC3_0, fexp::kC3_1, fexp::kC3_2, fexp::kC3_3, p0, p1);
}

// Rows of a 128-row tile in shared memory that must not enter a product (not finite, or not the sequence's: a weight
// of zero would not keep them out) are zeroed; bit `lane` of word g is row 32 g + lane.  A warp calls it.
// Which rows of the inputs are not finite is found by the pass that computes delta: looking through every tile here
// took longer (3,100 cycles of one warp a step) than the step's products and exponentials.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int lane, const uint32_t (&word)[4]) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        if ((word[g] >> lane) & 1u) {
            uint4* row = reinterpret_cast<uint4*>(tile + (32 * g + lane) * 128);   // a row's 128 bytes lie together
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) row[ch] = make_uint4(0, 0, 0, 0);
        }
    }
}
// whether one of eight bf16 values is not finite
__device__ __forceinline__ bool odd_values(const uint4& v) {
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
    __nv_bfloat162 a = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v.x), zero);
    a = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.y), zero, a);
    a = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.z), zero, a);
    a = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.w), zero, a);
    return !(__low2float(a) == 0.f && __high2float(a) == 0.f);
}

// P = exp2(c S - lse2) and dS = P (dP - delta) of COLS scores of one row, as bf16 pairs in the front of s (KEEP_P) and
// dp.  neg(k4, a, b, c, d) gives the packed pairs (-lse2) and (-delta) of columns 4 k4 .. 4 k4 + 3.  Unless WHOLE,
// `vis` has the bits of the columns seen.  `bad`: columns whose other operand was not finite and was zeroed: seen,
// they make the row NaN.
template <bool WHOLE, bool KEEP_P, class Neg>
__device__ __forceinline__ void grad_scores(uint32_t (&s)[COLS], uint32_t (&dp)[COLS], float c, uint32_t vis, uint32_t bad, Neg neg) {
    if (bad) {
#pragma unroll
        for (int k = 0; k < COLS; ++k)
            if ((bad >> k) & 1u) s[k] = dp[k] = 0x7fffffffu;   // (both: the FMA pipe's exponential of a NaN may be finite)
    }
    const uint64_t c2 = f2(c, c);
#pragma unroll
    for (int k4 = 0; k4 < COLS / 4; ++k4) {
        uint64_t nl[2], nd[2];
        neg(k4, nl[0], nl[1], nd[0], nd[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k2 = 2 * k4 + j;
            const uint32_t v = WHOLE ? 3u : vis >> (2 * k2);
            const uint64_t x = f2_fma(f2(__uint_as_float(s[2 * k2]), __uint_as_float(s[2 * k2 + 1])), c2, nl[j]);
            float p0, p1;
            if ((k2 & 7) >= 8 - EMU) {
                ex2_poly2(x, p0, p1);
            } else {
                float x0, x1;
                f2_split(x, x0, x1);
                p0 = ex2(x0);
                p1 = ex2(x1);
            }
            const uint64_t t = f2_add(f2(__uint_as_float(dp[2 * k2]), __uint_as_float(dp[2 * k2 + 1])), nd[j]);
            float d0, d1;
            f2_split(f2_mul(f2(p0, p1), t), d0, d1);
            if (!WHOLE) {   // selected, not multiplied: a masked score or product may be anything
                d0 = v & 1u ? d0 : 0.f;
                d1 = v & 2u ? d1 : 0.f;
                p0 = v & 1u ? p0 : 0.f;
                p1 = v & 2u ? p1 : 0.f;
            }
            if (KEEP_P) s[k2] = pack_bf16(p0, p1);
            dp[k2] = pack_bf16(d0, d1);
        }
    }
}

// COLS fp32 values of one row, times `f`, as bf16 to global memory; returns whether one is not finite.
__device__ __forceinline__ bool store_row(__nv_bfloat16* dst, const uint32_t (&o)[COLS], float f) {
    bool bad = false;
#pragma unroll
    for (int c8 = 0; c8 < COLS / 8; ++c8) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = __uint_as_float(o[8 * c8 + e]) * f;
            bad |= !isfinite(v[e]);
        }
        reinterpret_cast<uint4*>(dst)[c8] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                       pack_bf16(v[6], v[7]));
    }
    return bad;
}

// ------------------------------------------------------------------ the sinks' share of dK and dV
// Every later query sees a sink, so a block of keys with sinks in it has a long list of query rows while the
// others have a window's.  The rows past its window are cut into chunks that are items of their own; their sums
// go to slots of the workspace in fp32 and are added in a fixed order.
constexpr int CHUNK = 16 * BT;              // query rows of a chunk
constexpr int SINK_BLOCKS = 2;              // key blocks (of 128) that are cut up like this; with more sinks none
// Rows of at most FEW keys get their dQ from the delta pass (there in fp32), not from the dQ kernel.  20 is a choice for
// accuracy that short calls pay for.  dQ's error in the norm: 0.0017 with the delta pass at any number of keys, without
// it 0.0038 at 2 keys, 0.0027 at 8, 0.0025 at 20, 0.0024 at 64, so that rows of few keys are no worse than long ones.
// Time of the backward pass with FEW = 0 / 8 / 20 / 32: 700 rows of 4 heads 37 / 44 / 52 / 64 us, 40 sequences of 128
// rows 62 / 74 / 84 / 94, 16,384 rows with a window of 1,024 424 / 432 / 434 / 444; where every row has that few keys,
// a window of 16, 154 / 160 / 299 / 299 (the keys one after the other, and the dQ kernel runs all the same).
constexpr int FEW = 20;
// The keys that a row at position pos sees: the first `sk`, then [lo, lo + n)
struct RowKeys {
    int sk, lo, n;
    __device__ __forceinline__ RowKeys(const WindowArgs& p, int pos, int nk) {
        const int end = min(pos + p.right + 1, nk);
        lo = min(max(pos - p.left, 0), nk);
        n = max(end - lo, 0);
        sk = max(min(min(p.sinks, lo), end), 0);
    }
    __device__ __forceinline__ int all() const { return sk + n; }
    __device__ __forceinline__ bool few() const { return all() > 0 && all() <= FEW; }
};

constexpr long long SLOT = 2LL * BT * DH;   // floats: dK and dV of one block
// 256 MB.  Calls with more rows, sequences and heads leave the lists whole: one CTA then walks a sink block's every query,
// from 131,072 rows of 32 heads or 262,144 of 16 on (131,072 rows, 32 / 8 heads, 16 sinks: dK and dV take 5.9 ms at a
// window of 256, 1.2 without sinks; 6.3 and 2.7 at 1,024).
constexpr long long MAX_SLOTS = 4096;

__host__ __device__ inline long long chunk_slots(const WindowArgs& p) {
    return win::block_numbers<CHUNK>(p.Tq, p.n_seq) * p.Hq * SINK_BLOCKS;
}
__host__ __device__ inline long long window_slots(const WindowArgs& p) { return (long long)p.n_seq * p.Hk * SINK_BLOCKS; }
__host__ __device__ inline long long all_slots(const WindowArgs& p) {
    const long long n = chunk_slots(p) + window_slots(p);
    return n <= MAX_SLOTS ? n : 0;
}
inline bool cuts_sinks(const WindowArgs& p) { return p.sinks > 0 && p.sinks <= SINK_BLOCKS * BT && all_slots(p) > 0; }

// A sequence's queries [ia, ib) that see keys [u0, u1) inside their window (query i has position first + i).
struct QueryRange {
    int ia, ib;
};
__device__ __forceinline__ QueryRange queries_of(int u0, int u1, int first, int nq, int left, int right) {
    QueryRange r;
    r.ia = min(max(u0 - right - first, 0), nq);
    r.ib = max(min(u1 + left - first, nq), r.ia);
    return r;
}

}  // namespace winb
}  // namespace ttt
