// Gated linear recurrence h_t = a_t h_{t-1} + s(a_t) x_t, a = sigmoid(f), over long packed sequences: what the
// forward and the backward kernel share.
//
// Each pass reads its inputs and writes its outputs once.  A thread-block cluster owns a strip of channels (LC
// lanes of two bf16 or one fp32 channel) and walks the whole length; in a step each of its CTAs takes 32 / LC groups
// of 8 rows a warp, a thread keeping its rows' (a, s x) in registers.  The effect of a run of rows on the state is
// h -> A h + B: groups combine theirs in their warp, warps leave theirs in shared memory, and a warp of its own sends
// the CTA's to every CTA of the cluster (asynchronous stores to distributed shared memory that count on the
// receiver's barrier) and walks the state over the runs, one after the other.  Meanwhile the other warps compute the
// gates of the next step: two steps are in registers.  So the state never leaves the cluster, nothing waits on
// global memory, and the order of every operation is fixed.  The inputs come by TMA into a ring of stages.  The
// backward pass is the same walk the other way, lambda -> a (lambda + dy), with h recomputed from states that the
// forward pass keeps every 8 rows.
//
// A sequence's first row in walking order does not take the state before it: such a run has A = -0.  A state that
// is not finite would still reach through as 0 times it, so where a walk's result is not finite it is done again
// with the runs' signs looked at.
//
// In a strip of fewer channels the lanes beyond them do the last one's work once more (the same values to the same
// places), which spares a predicate on every access.
//
// Narrow strips (LC = 16 or 8) serve few channels, so that the grid is about one wave.  (Tiles that look back at
// each other's states in global memory in place of the clusters were slower: 2.25 ms for 313,344 rows of 1,024
// channels, the hand-over between tiles being the bound.)  Every wait is bounded.
#pragma once

#include <algorithm>
#include <type_traits>

#include "attn_prims.cuh"
#include "common.cuh"
#include "seq_offsets.cuh"

namespace ttt {
namespace scan {

constexpr int kKeep = 8;          // rows between two kept states, and of a group
constexpr int kRows = kKeep;
constexpr int kMaxCluster = 8;    // the portable size; of 16 CTAs only 14 clusters at two CTAs per SM fit the card
constexpr int kStages = 4;
constexpr float kReset = -0.f;
// Warps that walk rows (one more exchanges) and CTAs of them per SM: two steps' rows of the forward pass take 64
// registers of a thread, of the backward pass 128.
constexpr int kWarpsF = 7, kPerSmF = 2, kWarpsB = 11, kPerSmB = 1;

// ------------------------------------------------------------------ V channels' values, in fp32
// (Two channels in packed fp32 pairs took as many instructions: the moves that build and split the pairs.)
template <int V>
struct alignas(4 * V) Vec {
    float x[V];
    __device__ __forceinline__ float get(int v) const { return x[v]; }
    __device__ __forceinline__ void set(int v, float c) { x[v] = c; }
};
template <int V>
__device__ __forceinline__ Vec<V> fma(Vec<V> a, Vec<V> b, Vec<V> c) {
#pragma unroll
    for (int v = 0; v < V; ++v) c.x[v] = fmaf(a.x[v], b.x[v], c.x[v]);
    return c;
}
template <int V>
__device__ __forceinline__ Vec<V> mul(Vec<V> a, Vec<V> b) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.x[v] *= b.x[v];
    return a;
}
template <int V>
__device__ __forceinline__ Vec<V> add(Vec<V> a, Vec<V> b) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.x[v] += b.x[v];
    return a;
}
template <int V>
__device__ __forceinline__ Vec<V> sub(Vec<V> a, Vec<V> b) {
#pragma unroll
    for (int v = 0; v < V; ++v) a.x[v] -= b.x[v];
    return a;
}
template <int V>
__device__ __forceinline__ Vec<V> all(float c) {
    Vec<V> r;
#pragma unroll
    for (int v = 0; v < V; ++v) r.x[v] = c;
    return r;
}
// whether some channel is not finite
template <int V>
__device__ __forceinline__ bool wild(Vec<V> a) {
    const Vec<V> z = mul(a, all<V>(0.f));   // 0 or NaN
    return !(z.get(0) == 0.f && z.get(V - 1) == 0.f);
}

// ------------------------------------------------------------------ gates
// a = sigmoid(f) and rest = 1 - a = sigmoid(-f) from t = exp(-f): 1 / (1 + t) and t / (1 + t), with the rounding
// of f log2(e) made good (t is good to 2^-22 where the product alone would lose |f| 2^-24).  f is cut to
// [-80, 128], where a is below 2^-115 and rest zero (exp(-f) leaves fp32 at 87); NaN stays.
template <int V>
__device__ __forceinline__ void gates(Vec<V> f, Vec<V>& a, Vec<V>& rest) {
    constexpr float kL = 1.44269502f, kLow = 1.92596299e-8f, kLn2 = 0.693147182f;   // log2(e) in two parts
    Vec<V> z, t, r;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float c;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(f.get(v)), "f"(-80.f));
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(c), "f"(128.f));
        z.set(v, c);
    }
    const Vec<V> y = mul(z, all<V>(-kL));
    Vec<V> e = fma(z, all<V>(kL), y);
    e = fma(z, all<V>(kLow), e);
    e = mul(e, all<V>(-kLn2));
#pragma unroll
    for (int v = 0; v < V; ++v) t.set(v, attn::ex2(y.get(v)));
    t = fma(t, e, t);
    const Vec<V> d = add(t, all<V>(1.f));
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float q;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(d.get(v)));
        r.set(v, q);
    }
    a = r;
    rest = mul(t, r);
}

// b = s(a) x
template <int FORM, int V>
__device__ __forceinline__ Vec<V> input(Vec<V> a, Vec<V> rest, Vec<V> x) {
    if (FORM == 0) return x;
    if (FORM == 1) return mul(rest, x);
    Vec<V> s;
    const Vec<V> w = fma(rest, a, rest);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float q;
        asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(w.get(v)));
        s.set(v, q);
    }
    return mul(s, x);
}
// s(a) and dh/df = h_before a (1 - a) + x ds/df
template <int FORM, int V>
__device__ __forceinline__ void slopes(Vec<V> a, Vec<V> rest, Vec<V> h, Vec<V> x, Vec<V>& s, Vec<V>& d) {
    if (FORM == 0) {
        s = all<V>(1.f);
        d = mul(mul(a, rest), h);
    } else if (FORM == 1) {
        s = rest;
        d = mul(mul(a, rest), sub(h, x));
    } else {
        // sqrt(1 - a^2) and its a (1 - a) d/da = -a^2 sqrt((1 - a) / (1 + a)) from one reciprocal root of
        // 1 - a^2, kept off zero (and a NaN kept)
        Vec<V> q;
        const Vec<V> w = fma(rest, a, rest);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float c;
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(w.get(v)), "f"(1e-37f));
            asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(c));
            q.set(v, c);
        }
        s = mul(w, q);
        d = mul(a, sub(mul(rest, h), mul(mul(a, mul(rest, q)), x)));
    }
}

// ------------------------------------------------------------------ elements: V of 4 bytes in all
template <bool BF>
struct Elem {
    static constexpr int V = BF ? 2 : 1;
    using type = std::conditional_t<BF, __nv_bfloat16, float>;
    static __device__ __forceinline__ Vec<V> get(uint32_t w) {
        Vec<V> r;
        r.x[0] = __uint_as_float(BF ? w << 16 : w);
        if constexpr (BF) r.x[1] = __uint_as_float(w & 0xffff0000u);
        return r;
    }
    static __device__ __forceinline__ uint32_t put(Vec<V> x) {
        if constexpr (BF) return attn::pack_bf16(x.get(0), x.get(1));
        else return __float_as_uint(x.get(0));
    }
};

// ------------------------------------------------------------------ rows
// Whether R rows lie inside one sequence and none is its first or last one ([b, e): the sequence that the last
// look-up found).  Where they do not, each row's marks say what it is
// and the rows stay in registers like the others.  (Walking them one by one from shared memory, in rolled loops, held
// the cluster up for 3 us a border: 9,001 rows in 7 sequences, fp32, both passes 115 us against 91, in 40
// sequences 163 against 129; one sequence of 313,344 rows takes 523 us with the larger code, 517 with the smaller.)
template <int R>
__device__ __forceinline__ bool plain_rows(const SeqOffsets& c, int first, int dir, int& b, int& e) {
    const int lo = dir > 0 ? first : first - (R - 1), hi = lo + R - 1;
    if (!(lo > b && hi < e - 1)) {
        const int s = c.find(min(max(lo, 0), c.rows));
        b = c.begin(s);
        e = c.begin(s + 1);
    }
    return __all_sync(0xffffffffu, lo > b && hi < e - 1);
}
// Marks of eight rows: bit k for row t0 + dir k in a sequence, bit 8 + k for the first one of a sequence in walking
// order, bit 16 + k for the last one.  kBorder is set for rows that are not all plain ones.
constexpr uint32_t kBorder = 1u << 31;
__device__ __forceinline__ uint32_t marks_of(const SeqOffsets& c, int t0, int dir, int reverse) {
    const int lo = dir > 0 ? t0 : t0 - (kRows - 1), stop = min(lo + kRows, c.rows);
    uint32_t in = 0, low = 0, high = 0;   // bit r for row lo + r
    for (int t = max(lo, 0); t < stop;) {
        const int s = c.find(t), b = c.begin(s), e = c.begin(s + 1);
        if (t < b || t >= e) {   // behind the last sequence (or between offsets that fall)
            if (t >= c.begin(c.n)) break;
            ++t;
            continue;
        }
        const int u = min(e, stop);
        in |= (1u << (u - lo)) - (1u << (t - lo));
        if (t == b) low |= 1u << (t - lo);
        if (u == e) high |= 1u << (u - 1 - lo);
        t = u;
    }
    uint32_t first = reverse ? high : low, last = reverse ? low : high;
    if (dir < 0) {
        in = __brev(in) >> 24;
        first = __brev(first) >> 24;
        last = __brev(last) >> 24;
    }
    return kBorder | in | first << 8 | last << 16;
}
__device__ __forceinline__ bool in_sequence(uint32_t marks, int k) { return marks >> k & 1; }
__device__ __forceinline__ bool first_of(uint32_t marks, int k) { return marks >> (8 + k) & 1; }
__device__ __forceinline__ bool last_of(uint32_t marks, int k) { return marks >> (16 + k) & 1; }
static_assert(kRows == 8, "marks");
// Keeps the compiler from computing a border's addresses in front of the branch, where plain rows would pay for them.
template <class T>
__device__ __forceinline__ T* apart(T* p) {
    asm volatile("" : "+l"(p));
    return p;
}

// Sequence s's values of an fp32 array [n_seq, D] (null: zeros).
template <int V>
__device__ __forceinline__ Vec<V> state_of(const float* p, int s, int D, int ch) {
    Vec<V> r = all<V>(0.f);
    if (p) {
        const long long at = (long long)s * D + ch;
#pragma unroll
        for (int v = 0; v < V; ++v) r.set(v, p[at + v]);
    }
    return r;
}
// The same for the rows whose bits are set (the others' places are left).
template <int V>
__device__ __forceinline__ void states_at(Vec<V>* to, uint32_t bits, const SeqOffsets& c, int t0, int dir, const float* p, int D, int ch) {
    for (; bits; bits &= bits - 1) {
        const int k = __ffs(bits) - 1;
        to[k] = p ? state_of<V>(p, c.find(t0 + dir * k), D, ch) : all<V>(0.f);
    }
}
template <int V>
__device__ __forceinline__ void put_state(float* p, int s, int D, int ch, Vec<V> h) {
    if (!p) return;
    const long long at = (long long)s * D + ch;
#pragma unroll
    for (int v = 0; v < V; ++v) p[at + v] = h.get(v);
}

// States of empty sequences, and a look over the offsets.
__device__ __forceinline__ void empty_sequences(const SeqOffsets& c, int D, const float* from, float* to, int* status) {
    for (int s = blockIdx.x; s < c.n; s += gridDim.x) {
        if (threadIdx.x == 0 && (c.bad(s) || c.bad(s + 1))) atomicOr(status, kStatusBadOffsets);
        if (to && c.begin(s) >= c.begin(s + 1))
            for (int ch = threadIdx.x; ch < D; ch += blockDim.x)
                to[(long long)s * D + ch] = from ? from[(long long)s * D + ch] : 0.f;
    }
}

// ------------------------------------------------------------------ runs
template <int V>
struct alignas(8 * V) Run {
    Vec<V> a, b;
};
// run `p` followed by run `q`
template <int V>
__device__ __forceinline__ Run<V> then(Run<V> p, Run<V> q) {
    Run<V> r{mul(p.a, q.a), fma(q.a, p.b, q.b)};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const bool pr = signbit(p.a.get(v)), qr = signbit(q.a.get(v));
        if (pr || qr) r.a.set(v, kReset);
        if (qr) r.b.set(v, q.b.get(v));
    }
    return r;
}
template <int V>
__device__ __forceinline__ Vec<V> over(Run<V> p, Vec<V> h) { return fma(p.a, h, p.b); }
template <int V>
__device__ __forceinline__ Vec<V> over_exact(Run<V> p, Vec<V> h) {
    Vec<V> r = over(p, h);
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (signbit(p.a.get(v))) r.set(v, p.b.get(v));
    return r;
}
template <int V>
__device__ __forceinline__ Run<V> from_lane(Run<V> p, int lane) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        p.a.x[v] = __shfl_sync(0xffffffffu, p.a.x[v], lane);
        p.b.x[v] = __shfl_sync(0xffffffffu, p.b.x[v], lane);
    }
    return p;
}

// Several runs in a row; the exact form only where one of them has a reset.
template <int V, int N>
__device__ __forceinline__ Run<V> compose(const Run<V> (&q)[N]) {
    bool reset = false;
#pragma unroll
    for (int i = 0; i < N; ++i) reset |= signbit(q[i].a.get(0)) || signbit(q[i].a.get(V - 1));
    Run<V> r = q[0];
    if (__any_sync(0xffffffffu, reset)) {
#pragma unroll
        for (int i = 1; i < N; ++i) r = then<V>(r, q[i]);
    } else {
#pragma unroll
        for (int i = 1; i < N; ++i) r = Run<V>{mul(r.a, q[i].a), fma(q[i].a, r.b, q[i].b)};
    }
    return r;
}

template <int LC, int V, int W>
struct Shared {
    // each for two steps in turn
    Run<V> cta[2][kMaxCluster][LC];   // each CTA's run
    Run<V> part[2][W][LC];            // each warp's
    Vec<V> enter[2][W][LC];           // the state that enters each warp's rows
    uint64_t full[kStages];           // inputs landed
    uint64_t ready[2];                // part is written (W warps)
    uint64_t sent[2];                 // cta is written (bytes)
    uint64_t entered[2];              // enter is written
    volatile int abort;
};

template <int LC, int V, int W>
__device__ __forceinline__ void init_barriers(Shared<LC, V, W>& sh) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) tc::mbar_init(sh.full + s, 1);
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(sh.ready + s, W);
            tc::mbar_init(sh.sent + s, 1);
            tc::mbar_init(sh.entered + s, 1);
        }
        sh.abort = 0;
        tc::fence_mbar_init();
    }
    tc::cluster_sync();   // every CTA runs and has its barriers: its shared memory may be written
}

// A step's first half, by a walking warp: its groups' runs to the exchange.  Returns, for G > 1, the runs of the
// warp's groups in front of this one.
template <int LC, int V, int W>
__device__ __forceinline__ Run<V> hand_over(Shared<LC, V, W>& sh, int step, int col, Run<V> mine) {
    constexpr int G = 32 / LC;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane / LC;
    Run<V> before = mine;
    if constexpr (G == 1) {
        sh.part[step & 1][warp][col] = mine;
    } else {
        const Run<V> none{all<V>(1.f), all<V>(0.f)};
        Run<V> groups[G], front[G];
#pragma unroll
        for (int g = 0; g < G; ++g) groups[g] = from_lane<V>(mine, g * LC + col);
        front[0] = none;
#pragma unroll
        for (int g = 0; g < G - 1; ++g) front[g + 1] = g < group ? groups[g] : none;
        before = compose<V, G>(front);
        const Run<V> total = compose<V, G>(groups);
        if (lane < LC) sh.part[step & 1][warp][col] = total;
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(sh.ready + (step & 1));
    return before;
}
// Its second half: the state that enters this thread's rows.
template <int LC, int V, int W>
__device__ __forceinline__ bool take_over(Shared<LC, V, W>& sh, int step, int col, Run<V> before, Vec<V>& h) {
    if (!tc::mbar_wait(sh.entered + (step & 1), (step >> 1) & 1, &sh.abort)) return false;
    const Vec<V> e = sh.enter[step & 1][threadIdx.x >> 5][col];
    h = e;
    if constexpr (LC < 32) {
        h = over<V>(before, e);
        if (wild<V>(h)) h = over_exact<V>(before, e);
    }
    return true;
}

// The exchanging warp: issues the inputs' copies (issue(step)), sends the CTA's run of each step to the cluster and
// walks the state over the runs of the CTAs and of the warps.  (Every warp doing this for itself took 40% of all
// instructions; one of the walking warps doing it between two barriers left the others waiting 60% of the time.)
template <int LC, int V, int W, class Issue>
__device__ __forceinline__ bool exchange(Shared<LC, V, W>& sh, int steps, int cs, int rank, int cols, Issue issue) {
    constexpr int G = 32 / LC;
    const int lane = threadIdx.x & 31, col = min(lane % LC, cols - 1), group = lane / LC;
    Vec<V> state = all<V>(0.f);
    if (lane == 0)
        for (int s = 0; s < 2; ++s) issue(s);
    for (int step = 0; step < steps; ++step) {
        const int p = step & 1, phase = (step >> 1) & 1;
        if (!__all_sync(0xffffffffu, tc::mbar_wait(sh.ready + p, phase, &sh.abort))) return false;
        Run<V> q[W];
#pragma unroll
        for (int i = 0; i < W; ++i) q[i] = sh.part[p][i][col];
        const Run<V> total = compose<V, W>(q);
        if (lane == 0) tc::mbar_arrive_expect_tx(sh.sent + p, cs * LC * V * 8);
        __syncwarp();
        const uint32_t to0 = tc::smem_u32(&sh.cta[p][rank][col]), on0 = tc::smem_u32(sh.sent + p);
#pragma unroll
        for (int j = 0; j < kMaxCluster; j += G) {
            const int i = j + group;
            if (i < cs) {
                const uint32_t to = tc::mapa_shared(to0, i), on = tc::mapa_shared(on0, i);
                if constexpr (V == 2)
                    tc::st_async_v4(to, __float_as_uint(total.a.x[0]), __float_as_uint(total.a.x[1]),
                                    __float_as_uint(total.b.x[0]), __float_as_uint(total.b.x[1]), on);
                else
                    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(to),
                                 "r"(__float_as_uint(total.a.x[0])), "r"(__float_as_uint(total.b.x[0])), "r"(on) : "memory");
            }
        }
        // every warp has handed this step over, so is through with the one before the last: its stage is free
        if (lane == 0) issue(step + 2);
        // A slot is written again two steps on: its sender has then seen every CTA's next step, which each sends
        // after it has walked over this one.
        if (!__all_sync(0xffffffffu, tc::mbar_wait_cluster_abort(sh.sent + p, phase, &sh.abort))) return false;
        const Run<V>(*slot)[LC] = sh.cta[p];
        const Vec<V> s0 = state;
        auto walk = [&](auto step_over) {
            Vec<V> s = s0, e = s0;
#pragma unroll
            for (int i = 0; i < kMaxCluster; ++i) {
                if (i < cs) {
                    if (i == rank) e = s;
                    s = step_over(slot[i][col], s);
                }
            }
            state = s;
            if (lane < LC) sh.enter[p][0][col] = e;
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                e = step_over(q[i], e);
                if (lane < LC) sh.enter[p][i + 1][col] = e;
            }
            return wild<V>(s) || wild<V>(e);
        };
        if (__any_sync(0xffffffffu, walk([](Run<V> r, Vec<V> s) { return over<V>(r, s); })))
            walk([](Run<V> r, Vec<V> s) { return over_exact<V>(r, s); });
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(sh.entered + p);
    }
    return true;
}

struct Maps {
    CUtensorMap f, x, dy, h;   // boxes of a strip x a tile's rows; h: a tile's kept states
};

__device__ __forceinline__ int cluster_size() {
    int n;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

// A tile of more rows than a box may have (256) comes in two.
__host__ __device__ constexpr int box_rows(int tile) { return tile <= 256 ? tile : tile / 2; }

// Copies in flight land before a block that gave up leaves its memory.
__device__ __forceinline__ void settle() {
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
}

// ------------------------------------------------------------------ host
// rows of `cols` elements, boxes of `width` x `height`, no swizzle, zeros outside
inline bool map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, long long rows, int cols, long long ld, int width, int height) {
    auto fn = attn::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * (dt == CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 ? 2 : 4)};
    cuuint32_t box[2] = {(cuuint32_t)width, (cuuint32_t)height};
    cuuint32_t es[2] = {1, 1};
    return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One launch: kernel(args, maps) on strips x cluster CTAs.
template <bool BF, int LC, class Kernel>
cudaError_t launch(Kernel kernel, const GatedScanArgs& a, bool backward, int cs, cudaStream_t s) {
    constexpr int W = LC * Elem<BF>::V, ARRAYS_F = 2, ARRAYS_B = 3;
    const int warps = backward ? kWarpsB : kWarpsF, TILE = 32 / LC * warps * kRows, BOX = box_rows(TILE), HBOX = TILE / kKeep;
    Maps m{};
    const CUtensorMapDataType dt = BF ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const long long keeps = ((long long)a.T + kKeep - 1) / kKeep;
    if (a.T > 0 && (!map_2d(&m.f, dt, a.F, a.T, a.D, a.ld_f, W, BOX) || !map_2d(&m.x, dt, a.X, a.T, a.D, a.ld_x, W, BOX) ||
                    (backward && (!map_2d(&m.dy, dt, a.dY, a.T, a.D, a.ld_dy, W, BOX) ||
                                  !map_2d(&m.h, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.chunk_states, keeps, a.D, a.D, W, HBOX)))))
        return cudaErrorInvalidValue;
    const int smem = kStages * (((backward ? ARRAYS_B : ARRAYS_F) * TILE * LC * 4 + (backward ? HBOX * W * 4 : 0) + 127) / 128 * 128);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.D + W - 1) / W * cs));
    cfg.blockDim = dim3(32 * (warps + 1));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, m);
}

// The strip's width and the cluster's size: those that have most rows under way at once, the wider strip (whole
// 128-byte lines) where a narrower one has not a fifth more.  All clusters have to run at once, or the last ones
// double the time: clusters of up to eight CTAs fill at least 86% of the card's places (120 of 148 with one CTA per
// SM and eight, 264 of 296 with two).  120 of 148 is less, so the backward pass stops at six: with eight 102,400 x 1,024
// takes 444 us instead of 266 and x 512 263 instead of 154; only 9,001 x 776 in fp32 gains (44 -> 43).  With four x 256
// takes 152 us instead of 108.
struct Shape {
    int lanes, cs;
};
inline Shape shape_of(const GatedScanArgs& a, bool backward) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int V = a.bf16 ? 2 : 1, room = sms * (backward ? kPerSmB : kPerSmF) * 865 / 1000, most = backward ? 6 : kMaxCluster;
    Shape best{32, 1};
    long long best_rows = 0;
    for (int lanes = 32; lanes >= 8; lanes /= 2) {
        const int strips = (a.D + lanes * V - 1) / (lanes * V), tile = 32 / lanes * (backward ? kWarpsB : kWarpsF) * kRows;
        int cs = std::max(1, std::min(most, room / strips));
        while (cs > 1 && (long long)(cs - 1) * tile >= a.T) --cs;
        const long long rows = std::min<long long>((long long)cs * tile, a.T);
        if (5 * rows > 6 * best_rows) {
            best = Shape{lanes, cs};
            best_rows = rows;
        }
    }
    return best;
}

}  // namespace scan
}  // namespace ttt
