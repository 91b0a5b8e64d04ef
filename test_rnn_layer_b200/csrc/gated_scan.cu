// Gated linear recurrence h_t = a_t h_{t-1} + s(a_t) x_t, a = sigmoid(f), over long packed sequences: forward,
// backward and the single token.
//
// Each pass reads its inputs and writes its outputs once.  A thread-block cluster owns 32 threads' channels (64
// in bf16, 32 in fp32) and walks the whole length; in a step each of its CTAs takes 8 warps x R rows, a thread
// keeping its R rows' (a, s x) in registers.  The effect of a run of rows on the state is h -> A h + B: warps
// leave theirs in shared memory, CTAs send theirs to every CTA of the cluster (asynchronous stores to distributed
// shared memory that count on the receiver's barrier), and everyone walks the state over those before its own,
// one after the other, before it runs its rows from registers.  So the state never leaves the cluster, nothing
// waits on global memory, and the order of every operation is fixed.  The inputs of the next steps are on their
// way meanwhile (TMA into a ring of stages).  The backward pass is the same walk the other way,
// lambda -> a (lambda + dy), with h recomputed from states that the forward pass keeps every 8 rows.
//
// A sequence's first row in walking order does not take the state before it (not even as zero times it: what
// lies there may not be finite); such a run has A = -1, which no product of gates can be.
//
// (A single pass whose tiles look back at each other's states in global memory was slower: 2.25 ms for 313,344
// rows of 1,024 channels, its hand-over of about 1 us a tile being the bound.)  Every wait is bounded.
#include <type_traits>

#include "attn_prims.cuh"
#include "common.cuh"
#include "seq_offsets.cuh"

namespace ttt {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kKeep = 8;          // rows between two kept states
constexpr int kRowsF = 16;        // rows of a warp, forward
constexpr int kRowsB = kKeep;     // and backward
constexpr float kReset = -1.f;

struct Gate {
    float a, rest;                // sigmoid(f), 1 - a as sigmoid(-f)
};
// Two gates.  t = exp(-|f|) with the rounding of |f| log2(e) made good (2^-22 for every |f|, where the product
// alone would lose |f| 2^-24); beyond 128 it is zero all the same.  The minimum keeps a NaN.
__device__ __forceinline__ void gates(float f0, float f1, Gate& g0, Gate& g1) {
    constexpr float kL = 1.44269502f, kLow = 1.92596299e-8f, kLn2 = 0.693147182f;   // log2(e) in two parts
    float z0, z1, t0, t1, r0, r1, y0, y1, d0, d1, u0, u1;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(z0) : "f"(fabsf(f0)), "f"(128.f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(z1) : "f"(fabsf(f1)), "f"(128.f));
    const uint64_t z = attn::f2(z0, z1), y = attn::f2_fma(z, attn::f2(-kL, -kL), attn::f2(0.f, 0.f));
    uint64_t e = attn::f2_fma(z, attn::f2(kL, kL), y);
    e = attn::f2_fma(z, attn::f2(kLow, kLow), e);
    e = attn::f2_fma(e, attn::f2(-kLn2, -kLn2), attn::f2(0.f, 0.f));
    attn::f2_split(y, y0, y1);
    t0 = attn::ex2(y0);
    t1 = attn::ex2(y1);
    uint64_t t = attn::f2(t0, t1);
    t = attn::f2_fma(t, e, t);
    attn::f2_split(attn::f2_add(t, attn::f2(1.f, 1.f)), d0, d1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d1));
    attn::f2_split(attn::f2_fma(t, attn::f2(r0, r1), attn::f2(0.f, 0.f)), u0, u1);
    g0 = f0 < 0.f ? Gate{u0, r0} : Gate{r0, u0};
    g1 = f1 < 0.f ? Gate{u1, r1} : Gate{r1, u1};
}

// the input's scale s(a)
template <int FORM>
__device__ __forceinline__ float input_scale(const Gate& g) {
    if (FORM == 0) return 1.f;
    if (FORM == 1) return g.rest;
    float s;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(g.rest * (1.f + g.a)));
    return s;
}
// s(a) and dh/df = h_before a (1 - a) + x ds/df
template <int FORM>
__device__ __forceinline__ void slopes(const Gate& g, float h, float x, float& s, float& d) {
    if (FORM == 0) {
        s = 1.f;
        d = h * g.a * g.rest;
    } else if (FORM == 1) {
        s = g.rest;
        d = g.a * g.rest * (h - x);
    } else {
        // sqrt(1 - a^2) and its a (1 - a) d/da = -a^2 sqrt((1 - a) / (1 + a)) from one reciprocal root of
        // 1 - a^2, kept off zero
        float q;
        const float w = g.rest * (1.f + g.a);
        asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(fmaxf(w, 1e-37f)));
        s = w * q;
        d = g.a * (g.rest * h - x * (g.a * (g.rest * q)));
        if (g.rest != g.rest) s = d = g.rest;   // the maximum above drops a NaN
    }
}

// V elements of 4 bytes in all: two bf16 or one fp32
template <bool BF>
struct Elem {
    static constexpr int V = BF ? 2 : 1;
    using type = std::conditional_t<BF, __nv_bfloat16, float>;
    static __device__ __forceinline__ float get(uint32_t w, int v) {
        if (!BF) return __uint_as_float(w);
        return __uint_as_float(v ? w & 0xffff0000u : w << 16);
    }
    static __device__ __forceinline__ void store(void* p, long long i, const float (&x)[V]) {
        uint32_t w;
        if constexpr (BF) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[0], x[1]);
            w = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            w = __float_as_uint(x[0]);
        }
        __stcs(reinterpret_cast<uint32_t*>(static_cast<type*>(p) + i), w);
    }
};

__device__ __forceinline__ float carry(float A, float B, float h) { return A < 0.f ? B : fmaf(A, h, B); }

constexpr int kMaxCluster = 8;    // the portable size; with 16 only 14 clusters of two CTAs per SM fit the card
constexpr int kStages = 3;
template <int V>
struct Shared {
    float2 cta[2][kMaxCluster][32 * V];   // (A, B) of each CTA's rows, for two steps in turn
    float2 part[kWarps][32 * V];
    uint64_t full[kStages], sent[2];
};

// From the warps' (A, B) to the state that enters this warp's rows; `run` (the state that enters the cluster's
// step, the same in every thread of a channel) moves on to the next step.  `consumed` runs once every warp has
// its inputs in registers.
template <int V, class Consumed>
__device__ __forceinline__ bool exchange(Shared<V>& sh, int step, int cs, int rank, const float (&A)[V], const float (&B)[V],
                                         float (&run)[V], float (&h)[V], bool ok, Consumed consumed) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int v = 0; v < V; ++v) sh.part[warp][lane * V + v] = make_float2(A[v], B[v]);
    __syncthreads();
    uint64_t* bar = sh.sent + (step & 1);
    if (warp == 0) {
        float a[V], b[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            a[v] = 1.f;
            b[v] = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const float2 p = sh.part[i][lane * V + v];
                b[v] = carry(p.x, p.y, b[v]);
                a[v] = p.x < 0.f || a[v] < 0.f ? kReset : a[v] * p.x;
            }
        }
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, cs * 32 * V * 8);
        const uint32_t mine = tc::smem_u32(&sh.cta[step & 1][rank][lane * V]), at = tc::smem_u32(bar);
        for (int i = 0; i < cs; ++i) {
            const uint32_t to = tc::mapa_shared(mine, i), on = tc::mapa_shared(at, i);
            if constexpr (V == 2)
                tc::st_async_v4(to, __float_as_uint(a[0]), __float_as_uint(b[0]), __float_as_uint(a[1]), __float_as_uint(b[1]), on);
            else
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(to),
                             "r"(__float_as_uint(a[0])), "r"(__float_as_uint(b[0])), "r"(on) : "memory");
        }
    } else if (threadIdx.x == 32) {
        consumed();
    }
    // A slot is written again two steps on: its sender has then seen every CTA's next step, which each sends
    // after it has read this one.
    ok = tc::mbar_wait_cluster(bar, (step >> 1) & 1) && ok;
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = run[v];
    for (int i = 0; i < cs; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (i == rank) h[v] = run[v];
            const float2 p = sh.cta[step & 1][i][lane * V + v];
            run[v] = carry(p.x, p.y, run[v]);
        }
    }
    for (int i = 0; i < warp; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 p = sh.part[i][lane * V + v];
            h[v] = carry(p.x, p.y, h[v]);
        }
    return __syncthreads_and(ok);   // the same for the whole CTA; part is free again
}

// A warp's rows: bit k of the masks is row first + dir * k.
struct Rows {
    uint32_t valid, start, end;   // in a sequence; its first and its last row in walking order
    int seq;                      // lane k: row k's sequence
    bool plain;                   // all valid, none first or last
};
template <int R>
__device__ __forceinline__ Rows rows_of(const SeqOffsets& c, long long first, int dir, int reverse) {
    const int lane = threadIdx.x & 31;
    const long long t = first + (long long)dir * lane;
    Rows r{0, 0, 0, 0, false};
    bool valid = false, lo = false, hi = false;
    if (lane < R && t >= 0 && t < c.rows) {
        r.seq = c.find((int)t);
        const int b = c.begin(r.seq), e = c.begin(r.seq + 1);
        valid = t >= b && t < e;
        lo = valid && t == b;
        hi = valid && t == e - 1;
    }
    r.valid = __ballot_sync(0xffffffffu, valid);
    const uint32_t l = __ballot_sync(0xffffffffu, lo), h = __ballot_sync(0xffffffffu, hi);
    r.start = reverse ? h : l;
    r.end = reverse ? l : h;
    r.plain = r.valid == (uint32_t)((1ull << R) - 1) && !(l | h);
    return r;
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

struct Maps {
    CUtensorMap f, x, dy, h;   // boxes of 128 bytes x a tile's rows; h: a tile's kept states
};

__device__ __forceinline__ int cluster_size() {
    int n;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

template <bool BF, int FORM>
__global__ void __launch_bounds__(kThreads, 2) gated_fwd_kernel(const __grid_constant__ GatedScanArgs p, const __grid_constant__ Maps m) {
    constexpr int R = kRowsF, V = Elem<BF>::V, TILE = kWarps * R;
    __shared__ Shared<V> sh;
    extern __shared__ __align__(128) uint8_t stages[];
    const SeqOffsets c{p.cu, p.n_seq, p.T};
    const int cs = cluster_size(), rank = tc::cluster_ctarank(), chunks = (p.T + TILE - 1) / TILE, steps = (chunks + cs - 1) / cs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, dir = p.reverse ? -1 : 1;
    const int ch = (blockIdx.x / cs * 32 + lane) * V;
    const bool on = ch < p.D;
    empty_sequences(c, p.D, p.H_0, p.H_T, p.status);

    auto first_row = [&](int step) {   // the warp's first row in walking order; past the last chunk outside [0, T)
        const long long chunk = (long long)step * cs + rank;
        return p.reverse ? (chunks - chunk) * TILE - 1 - warp * R : chunk * TILE + warp * R;
    };
    // stage s: TILE rows of 128 bytes of F, then of X
    auto issue = [&](int step) {
        const int chunk = step * cs + rank, s = step % kStages;
        if (step >= steps || chunk >= chunks) return;
        const int row = (p.reverse ? chunks - 1 - chunk : chunk) * TILE, x = blockIdx.x / cs * 32 * V;
        uint8_t* to = stages + s * 2 * TILE * 128;
        tc::mbar_arrive_expect_tx(sh.full + s, 2 * TILE * 128);
        tc::tma_load_2d(to, &m.f, x, row, sh.full + s);
        tc::tma_load_2d(to + TILE * 128, &m.x, x, row, sh.full + s);
    };
    float run[V] = {};
    bool bad = false;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) tc::mbar_init(sh.full + s, 1);
        for (int s = 0; s < 2; ++s) tc::mbar_init(sh.sent + s, 1);
        tc::fence_mbar_init();
    }
    tc::cluster_sync();   // every CTA runs and has its barriers: its shared memory may be written
    if (threadIdx.x == 32)
        for (int s = 0; s < kStages; ++s) issue(s);
    bool ok = true;
    for (int step = 0; step < steps && ok; ++step) {
        const long long t0 = first_row(step);
        const Rows r = rows_of<R>(c, t0, dir, p.reverse);
        uint32_t fw[R], xw[R];
        if (step * cs + rank < chunks) ok = tc::mbar_wait(sh.full + step % kStages, (step / kStages) & 1, nullptr);
        {
            const uint32_t* in = reinterpret_cast<const uint32_t*>(stages + step % kStages * 2 * TILE * 128) +
                                 (p.reverse ? TILE - 1 - warp * R : warp * R) * 32 + lane;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                fw[k] = in[dir * k * 32];
                xw[k] = in[(TILE + dir * k) * 32];
            }
        }
        float a[R][V], b[R][V], A[V], B[V], h[V];
        // gates, two at a time (two channels, or two rows of one)
#pragma unroll
        for (int i = 0; i < R * V; i += 2) {
            const int k0 = i / V, v0 = i % V, k1 = (i + 1) / V, v1 = (i + 1) % V;
            Gate g0, g1;
            gates(Elem<BF>::get(fw[k0], v0), Elem<BF>::get(fw[k1], v1), g0, g1);
            a[k0][v0] = g0.a;
            a[k1][v1] = g1.a;
            b[k0][v0] = input_scale<FORM>(g0) * Elem<BF>::get(xw[k0], v0);
            b[k1][v1] = input_scale<FORM>(g1) * Elem<BF>::get(xw[k1], v1);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f;
            B[v] = 0.f;
        }
        if (r.plain) {
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    B[v] = fmaf(a[k][v], B[v], b[k][v]);
                    A[v] *= a[k][v];
                }
        } else {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int s = __shfl_sync(0xffffffffu, r.seq, k);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if ((r.start >> k) & 1u) {   // the first row: b includes what the initial state leaves
                        const float h0 = p.H_0 && on ? p.H_0[(long long)s * p.D + ch + v] : 0.f;
                        b[k][v] = fmaf(a[k][v], h0, b[k][v]);
                        A[v] = kReset;
                        B[v] = b[k][v];
                    } else if ((r.valid >> k) & 1u) {
                        B[v] = fmaf(a[k][v], B[v], b[k][v]);
                        A[v] = A[v] < 0.f ? kReset : A[v] * a[k][v];
                    }
                }
            }
        }
        ok = exchange<V>(sh, step, cs, rank, A, B, run, h, ok, [&]() { issue(step + kStages); });
        const long long keep0 = t0 < 0 ? -1 : t0 / kKeep;   // a warp's rows are whole segments
        auto keep = [&](int k) {
            const long long seg = keep0 + dir * (k / kKeep);
            if (p.chunk_states && on && keep0 >= 0 && seg * kKeep < p.T) {
#pragma unroll
                for (int v = 0; v < V; ++v) p.chunk_states[seg * p.D + ch + v] = h[v];
            }
        };
        if (r.plain) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (k % kKeep == 0) keep(k);
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = fmaf(a[k][v], h[v], b[k][v]);
                if (on) Elem<BF>::store(p.Y, (t0 + dir * k) * p.ld_y + ch, h);
            }
            // inside a sequence a state that is not finite stays so
#pragma unroll
            for (int v = 0; v < V; ++v) bad |= on && !isfinite(h[v]);
        } else {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (k % kKeep == 0) keep(k);
                if (!((r.valid >> k) & 1u)) continue;
                const bool start = (r.start >> k) & 1u;
                const int s = __shfl_sync(0xffffffffu, r.seq, k);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    h[v] = start ? b[k][v] : fmaf(a[k][v], h[v], b[k][v]);
                    bad |= on && !isfinite(h[v]);
                }
                if (!on) continue;
                Elem<BF>::store(p.Y, (t0 + dir * k) * p.ld_y + ch, h);
                if (p.H_T && ((r.end >> k) & 1u)) {
#pragma unroll
                    for (int v = 0; v < V; ++v) p.H_T[(long long)s * p.D + ch + v] = h[v];
                }
            }
        }
    }
    if (bad) atomicOr(p.status, kStatusNonFinite);
    if (!ok) atomicOr(p.status, kStatusTimeout);
    if (!ok) {   // copies in flight land before the block's memory goes away
        const uint64_t t0 = tc::globaltimer_ns();
        while (tc::globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
    tc::cluster_sync();   // nobody leaves while another may still write to its shared memory
}

// Backward: rows in the order of lambda's walk, against the forward walk.
template <bool BF, int FORM>
__global__ void __launch_bounds__(kThreads, 2) gated_bwd_kernel(const __grid_constant__ GatedScanArgs p, const __grid_constant__ Maps m) {
    constexpr int R = kRowsB, V = Elem<BF>::V, TILE = kWarps * R;
    __shared__ Shared<V> sh;
    extern __shared__ __align__(128) uint8_t stages[];
    const SeqOffsets c{p.cu, p.n_seq, p.T};
    const int cs = cluster_size(), rank = tc::cluster_ctarank(), chunks = (p.T + TILE - 1) / TILE, steps = (chunks + cs - 1) / cs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, dir = p.reverse ? 1 : -1;
    const int ch = (blockIdx.x / cs * 32 + lane) * V;
    const bool on = ch < p.D;
    empty_sequences(c, p.D, p.dH_T, p.dH_0, p.status);

    auto first_row = [&](int step) {
        const long long chunk = (long long)step * cs + rank;
        return p.reverse ? chunk * TILE + warp * R : (chunks - chunk) * TILE - 1 - warp * R;
    };
    // stage s: TILE rows of 128 bytes of F, X and dY, then the kept states of the tile's segments
    constexpr int STAGE = 3 * TILE * 128 + kWarps * 32 * V * 4;
    auto issue = [&](int step) {
        const int chunk = step * cs + rank, s = step % kStages;
        if (step >= steps || chunk >= chunks) return;
        const int row = (p.reverse ? chunk : chunks - 1 - chunk) * TILE, x = blockIdx.x / cs * 32 * V;
        uint8_t* to = stages + s * STAGE;
        tc::mbar_arrive_expect_tx(sh.full + s, STAGE);
        tc::tma_load_2d(to, &m.f, x, row, sh.full + s);
        tc::tma_load_2d(to + TILE * 128, &m.x, x, row, sh.full + s);
        tc::tma_load_2d(to + 2 * TILE * 128, &m.dy, x, row, sh.full + s);
        tc::tma_load_2d(to + 3 * TILE * 128, &m.h, x, row / kKeep, sh.full + s);
    };
    float run[V] = {};
    bool bad = false;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) tc::mbar_init(sh.full + s, 1);
        for (int s = 0; s < 2; ++s) tc::mbar_init(sh.sent + s, 1);
        tc::fence_mbar_init();
    }
    tc::cluster_sync();   // every CTA runs and has its barriers: its shared memory may be written
    if (threadIdx.x == 32)
        for (int s = 0; s < kStages; ++s) issue(s);
    bool ok = true;
    for (int step = 0; step < steps && ok; ++step) {
        const long long t0 = first_row(step);
        const Rows r = rows_of<R>(c, t0, dir, p.reverse);
        uint32_t fw[R], xw[R], gw[R];
        float hw[V];
        if (step * cs + rank < chunks) ok = tc::mbar_wait(sh.full + step % kStages, (step / kStages) & 1, nullptr);
        {
            const uint8_t* st = stages + step % kStages * STAGE;
            const uint32_t* in = reinterpret_cast<const uint32_t*>(st) + (p.reverse ? warp * R : TILE - 1 - warp * R) * 32 + lane;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                fw[k] = in[dir * k * 32];
                xw[k] = in[(TILE + dir * k) * 32];
                gw[k] = in[(2 * TILE + dir * k) * 32];
            }
            const float* kept = reinterpret_cast<const float*>(st + 3 * TILE * 128) + (p.reverse ? warp : kWarps - 1 - warp) * 32 * V + lane * V;
#pragma unroll
            for (int v = 0; v < V; ++v) hw[v] = kept[v];
        }
        float a[R][V], sc[R][V], sl[R][V], dy[R][V], A[V], B[V], lam[V];
        // gates, and the forward walk over the warp's rows: scales and slopes
#pragma unroll
        for (int i = R * V - 2; i >= 0; i -= 2) {
            const int k0 = i / V, v0 = i % V, k1 = (i + 1) / V, v1 = (i + 1) % V;
            Gate g[2];
            gates(Elem<BF>::get(fw[k0], v0), Elem<BF>::get(fw[k1], v1), g[0], g[1]);
#pragma unroll
            for (int j = 1; j >= 0; --j) {
                const int k = j ? k1 : k0, v = j ? v1 : v0;
                const float x = Elem<BF>::get(xw[k], v);
                const bool start = !r.plain && ((r.start >> k) & 1u), valid = r.plain || ((r.valid >> k) & 1u);
                if (start) {
                    const int s = __shfl_sync(0xffffffffu, r.seq, k);
                    hw[v] = p.H_0 && on ? p.H_0[(long long)s * p.D + ch + v] : 0.f;
                }
                slopes<FORM>(g[j], hw[v], x, sc[k][v], sl[k][v]);
                if (valid) hw[v] = fmaf(g[j].a, hw[v], sc[k][v] * x);
                a[k][v] = g[j].a;
                dy[k][v] = Elem<BF>::get(gw[k], v);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f;
            B[v] = 0.f;
        }
        if (r.plain) {
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    B[v] = a[k][v] * (B[v] + dy[k][v]);
                    A[v] *= a[k][v];
                }
        } else {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int s = __shfl_sync(0xffffffffu, r.seq, k);
                if (!((r.valid >> k) & 1u)) continue;
                const bool end = (r.end >> k) & 1u;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (end) {   // lambda starts anew: dy takes the final state's gradient along
                        if (p.dH_T && on) dy[k][v] += p.dH_T[(long long)s * p.D + ch + v];
                        A[v] = kReset;
                        B[v] = a[k][v] * dy[k][v];
                    } else {
                        B[v] = a[k][v] * (B[v] + dy[k][v]);
                        A[v] = A[v] < 0.f ? kReset : A[v] * a[k][v];
                    }
                }
            }
        }
        ok = exchange<V>(sh, step, cs, rank, A, B, run, lam, ok, [&]() { issue(step + kStages); });
        float seen = 0.f;   // 0 times what is stored: NaN where it is not finite
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (!r.plain && !((r.valid >> k) & 1u)) continue;
            const bool end = !r.plain && ((r.end >> k) & 1u);
            float df[V], dx[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float l = end ? dy[k][v] : lam[v] + dy[k][v];
                df[v] = l * sl[k][v];
                dx[v] = l * sc[k][v];
                seen = fmaf(0.f, df[v], seen);
                lam[v] = a[k][v] * l;
            }
            if (!r.plain) bad |= on && !(isfinite(lam[0]) && isfinite(lam[V - 1]));
            const int s = r.plain ? 0 : __shfl_sync(0xffffffffu, r.seq, k);
            if (!on) continue;
            Elem<BF>::store(p.dF, (t0 + dir * k) * p.ld_df + ch, df);
            Elem<BF>::store(p.dX, (t0 + dir * k) * p.ld_dx + ch, dx);
            if (!r.plain && p.dH_0 && ((r.start >> k) & 1u)) {
#pragma unroll
                for (int v = 0; v < V; ++v) p.dH_0[(long long)s * p.D + ch + v] = lam[v];
            }
        }
        if (r.plain) bad |= on && !(isfinite(lam[0]) && isfinite(lam[V - 1]));
        bad |= on && seen != 0.f;
    }
    if (bad) atomicOr(p.status, kStatusNonFinite);
    if (!ok) atomicOr(p.status, kStatusTimeout);
    if (!ok) {   // copies in flight land before the block's memory goes away
        const uint64_t t0 = tc::globaltimer_ns();
        while (tc::globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
    tc::cluster_sync();   // nobody leaves while another may still write to its shared memory
}

// One token of each row: a thread takes eight channels, 16 or 32 bytes at a time.
template <bool BF, int FORM>
__global__ void __launch_bounds__(128) gated_step_kernel(int D, long long units, const void* F, long long ld_f, const void* X,
                                                         long long ld_x, const float* H, float* H_out, void* Y, long long ld_y) {
    constexpr int N = BF ? 4 : 8;   // 32-bit words of eight elements
    const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= units) return;
    const int per = D / 8;
    const long long b = u / per, ch = u % per * 8;
    uint4 fw[N / 4], xw[N / 4];
    float4 h[2];
    const uint4* f = reinterpret_cast<const uint4*>(static_cast<const typename Elem<BF>::type*>(F) + b * ld_f + ch);
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const typename Elem<BF>::type*>(X) + b * ld_x + ch);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        fw[i] = f[i];
        xw[i] = x[i];
    }
    const float4* hp = reinterpret_cast<const float4*>(H + b * D + ch);
    h[0] = hp[0];
    h[1] = hp[1];
    float* hv = reinterpret_cast<float*>(h);
    const uint32_t* fv = reinterpret_cast<const uint32_t*>(fw);
    const uint32_t* xv = reinterpret_cast<const uint32_t*>(xw);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const int w0 = BF ? i / 2 : i, w1 = BF ? i / 2 : i + 1;
        Gate g0, g1;
        gates(Elem<BF>::get(fv[w0], 0), Elem<BF>::get(fv[w1], 1), g0, g1);
        hv[i] = fmaf(g0.a, hv[i], input_scale<FORM>(g0) * Elem<BF>::get(xv[w0], 0));
        hv[i + 1] = fmaf(g1.a, hv[i + 1], input_scale<FORM>(g1) * Elem<BF>::get(xv[w1], 1));
    }
    float4* ho = reinterpret_cast<float4*>(H_out + b * D + ch);
    ho[0] = h[0];
    ho[1] = h[1];
    if (!Y) return;
    uint32_t yw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (BF) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(hv[2 * i], hv[2 * i + 1]);
            yw[i] = *reinterpret_cast<const uint32_t*>(&v);
        } else {
            yw[i] = __float_as_uint(hv[i]);
        }
    }
    uint4* y = reinterpret_cast<uint4*>(static_cast<typename Elem<BF>::type*>(Y) + b * ld_y + ch);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) y[i] = make_uint4(yw[4 * i], yw[4 * i + 1], yw[4 * i + 2], yw[4 * i + 3]);
}

// rows of `cols` elements, boxes of `width` x `height`, no swizzle, zeros outside
bool map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, long long rows, int cols, long long ld, int width, int height) {
    auto fn = attn::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * (dt == CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 ? 2 : 4)};
    cuuint32_t box[2] = {(cuuint32_t)width, (cuuint32_t)height};
    cuuint32_t es[2] = {1, 1};
    return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF, int FORM>
cudaError_t scan(const GatedScanArgs& a, bool backward, int sms, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(a.status, 0, 16, s);
    if (e != cudaSuccess) return e;
    auto kernel = backward ? gated_bwd_kernel<BF, FORM> : gated_fwd_kernel<BF, FORM>;
    const int tile = kWarps * (backward ? kRowsB : kRowsF), ctiles = (a.D + 32 * Elem<BF>::V - 1) / (32 * Elem<BF>::V);
    // as many CTAs along the rows as two per SM leave room for (all clusters then run at once) and there are tiles
    int cs = 1;
    while (cs < kMaxCluster && 2LL * cs * ctiles <= 2 * sms && (long long)cs * tile < a.T) cs *= 2;
    Maps m{};
    constexpr int W = 32 * Elem<BF>::V;
    const CUtensorMapDataType dt = BF ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    const long long keeps = gated_scan_chunk_state_floats(a.T, a.D) / a.D;
    if (a.T > 0 && (!map_2d(&m.f, dt, a.F, a.T, a.D, a.ld_f, W, tile) || !map_2d(&m.x, dt, a.X, a.T, a.D, a.ld_x, W, tile) ||
                    (backward && (!map_2d(&m.dy, dt, a.dY, a.T, a.D, a.ld_dy, W, tile) ||
                                  !map_2d(&m.h, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.chunk_states, keeps, a.D, a.D, W, kWarps)))))
        return cudaErrorInvalidValue;
    const int smem = kStages * (backward ? 3 * tile * 128 + kWarps * W * 4 : 2 * tile * 128);
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ctiles * cs));
    cfg.blockDim = dim3(kThreads);
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

cudaError_t scan_any(const GatedScanArgs& a, bool backward, cudaStream_t s) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    LaunchScope scope(backward ? "gated_scan_backward" : "gated_scan", s);
    if (a.bf16)
        return a.form == 0 ? scan<true, 0>(a, backward, sms, s) : a.form == 1 ? scan<true, 1>(a, backward, sms, s) : scan<true, 2>(a, backward, sms, s);
    return a.form == 0 ? scan<false, 0>(a, backward, sms, s) : a.form == 1 ? scan<false, 1>(a, backward, sms, s) : scan<false, 2>(a, backward, sms, s);
}

}  // namespace

long long gated_scan_chunk_state_floats(int T, int D) { return ((long long)T + kKeep - 1) / kKeep * D; }

cudaError_t launch_gated_scan(const GatedScanArgs& a, cudaStream_t s) { return scan_any(a, false, s); }
cudaError_t launch_gated_scan_backward(const GatedScanArgs& a, cudaStream_t s) { return scan_any(a, true, s); }

cudaError_t launch_gated_scan_step(int B, int D, int form, int bf16, const void* F, long long ld_f, const void* X,
                                   long long ld_x, const float* H, float* H_out, void* Y, long long ld_y,
                                   cudaStream_t s) {
    LaunchScope scope("gated_scan_step", s);
    const long long units = (long long)B * (D / 8);
    const unsigned grid = (unsigned)((units + 127) / 128);
    auto go = [&](auto kernel) { kernel<<<grid, 128, 0, s>>>(D, units, F, ld_f, X, ld_x, H, H_out, Y, ld_y); };
    if (bf16) form == 0 ? go(gated_step_kernel<true, 0>) : form == 1 ? go(gated_step_kernel<true, 1>) : go(gated_step_kernel<true, 2>);
    else form == 0 ? go(gated_step_kernel<false, 0>) : form == 1 ? go(gated_step_kernel<false, 1>) : go(gated_step_kernel<false, 2>);
    return cudaGetLastError();
}

}  // namespace ttt
