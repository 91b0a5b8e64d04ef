// Window attention with sinks, forward, on the tcgen05 tensor cores (head dim 64, bf16, fp32 accumulation):
//   Out[i, h] = Xres[i, h] + sum_u softmax_u(scale q_i . k_u) v_u over the keys u that row i sees:
//   u <= p + right and (u >= p - left or u < sinks), p = nk - nq + i.
//
// Work: an item is 256 query rows of a sequence (tiles A and B of 128) of one head; a persistent grid draws the
// items, heads fastest, so that the CTAs running at a time share the keys and values of few windows in L2.  An
// item's key tiles are those of its sinks and those of the window of its rows, 128 keys each.  A tile's halves of 64
// keys go to two softmax groups with a running maximum, a sum and an output of their own (two threads a row, joined
// at the item's end), so there are four streams (A and B, first and second half) that take turns on the tensor
// cores and the issue slots; a half that a stream's rows do not see is skipped.  Per half tile, as in the
// segment-local kernel: S = Q K^T (tensor memory), P = exp2(c S - m) with a lazily raised maximum, O += P V.  P lies
// where S was.  Masks are two 32-bit words per row, applied only where the half tile is not seen whole.
// (Two streams of whole rows, eight softmax warps: 4,000 cycles a tile of A and B, 44% of the issue slots used.)
//
// A weight of zero times a non-finite value is NaN, and a tile's rows behind the sequence's end may hold
// anything: warp 11 looks through each value tile in shared memory (one product by zero per pair of elements,
// well below a tenth of the tile's softmax), zeroes the rows that are not finite and leaves their bits for the
// softmax, which spoils exactly the query rows that see them.
//
// Roles (640 threads): warps 0-7 the softmax of tile A, 8-15 that of tile B (first half, second half; a thread per
// query row), warp 16 the TMA producer, warps 17 and 18 the MMA issuers of A and B, warp 19 the value screen.
// Tensor memory (512 columns), tile X: S 256 X (second half + 64), P in the first 32 columns of each, O 256 X + 128
// (second half + 64).
// Every wait is bounded; on a timeout the CTA sets the status word, lets its copies and products in flight
// land and returns.
#include <type_traits>

#include "attn_prims.cuh"
#include "internal.h"
#include "window_items.cuh"

namespace ttt {
namespace {

using namespace attn;

constexpr int DH = 64, BQ = 128, BKV = 128, HALF = 64, ROWS = 2 * BQ, NST = 4, SOFT = 16, THREADS = 32 * (SOFT + 4);
constexpr int TILE = BQ * DH * 2;                 // 16 KB: a 128 x 64 bf16 tile
constexpr int OFF_Q = 0;                          // Q_A, Q_B
constexpr int OFF_KV = 2 * TILE;                  // stage s: K at OFF_KV + 2 s TILE, V after it
constexpr int OFF_BAR = OFF_KV + NST * 2 * TILE;
constexpr int OFF_ML = OFF_BAR + 512;             // [2][2][128] float2: a row's maximum and sum in each half
constexpr int OFF_ORDER = OFF_ML + 4096;          // [kOrder] bytes
constexpr int SMEM_BYTES = OFF_ORDER + win::kOrder + 1024;
constexpr uint32_t TM_X = 256, TM_O = 128;        // tile X's S at TM_X X + 64 y, its O at TM_X X + TM_O + 64 y
constexpr float kLazy = 8.0f;                     // log2 of the largest unscaled exponential
constexpr int EMU = 1;                            // pairs of every 8 whose 2^x runs on the FMA pipe

// Barrier slots (8 bytes each) from OFF_BAR.
enum : int {
    B_QF = 0,              // Q_A, Q_B landed (TMA bytes)
    B_QE = 1,              // the item's S products are done (2 commits)
    B_KF = 2,              // [NST] K tile landed
    B_VF = 2 + NST,        // [NST] V tile landed
    B_VS = 2 + 2 * NST,    // [NST] V tile screened
    B_KVE = 2 + 3 * NST,   // [NST] the streams are done with the stage (4 arrivals)
    B_SF = 2 + 4 * NST,    // [4] a stream's S is in tensor memory, its products before are done (MMA commit)
    B_PF = B_SF + 4,       // [4] its P is written, its O rescaled (4 warp arrivals)
    B_OD = B_PF + 4,       // [4] its O is complete (MMA commit)
    B_SLOT = B_OD + 4,     // tensor memory address (u32) and the abort flag (int)
    B_BAD = 36,            // [NST] 16 bytes: bits of the stage's V rows that are not finite
    B_IF = B_BAD + 2 * NST,  // [4] the CTA's items: handed out, taken; their numbers (4 ints)
    B_IE = B_IF + win::kItemSlots,
    B_ITEM = B_IE + win::kItemSlots
};
static_assert(B_SLOT < B_BAD && B_BAD % 2 == 0 && B_ITEM * 8 + 16 <= 512, "barrier area");
constexpr int kTicket = 1;   // the item counter's place behind the status word (cleared with it)
static_assert(SMEM_BYTES <= 232448, "shared memory");

struct FwdArgs {
    CUtensorMap mapQ, mapK, mapV;   // bf16 [rows x heads*64 columns], 64 x 128 boxes
    WindowArgs w;
    long long n_items;
    int sorted;                     // few blocks of unequal work: drawn by it
    float c;                        // scale * log2(e)
};

struct Item {
    int q_lo, rows, pos0, k0, nk, h, hk;
    int ns, nt;                     // sink tiles, all tiles
    win::KeyRange r;

    __device__ __forceinline__ bool load(const WindowArgs& p, long long w) {
        const SeqOffsets cq{p.cu_q, p.n_seq, p.Tq}, ck{p.cu_k, p.n_seq, p.Tk};
        h = (int)(w % p.Hq);
        hk = h / (p.Hq / p.Hk);
        const int s = win::block_of<ROWS>(cq, (int)(w / p.Hq), q_lo, rows);
        if (s < 0) return false;
        const int q0 = cq.begin(s), nq = cq.begin(s + 1) - q0;
        k0 = ck.begin(s);
        nk = max(ck.begin(s + 1) - k0, 0);
        pos0 = nk - nq + (q_lo - q0);
        r = win::keys_of(pos0, rows, nk, p.left, p.right, p.sinks);
        ns = (r.sk + BKV - 1) / BKV;
        nt = ns + (r.hi - r.lo + BKV - 1) / BKV;
        return true;
    }
    __device__ __forceinline__ int start(int j) const { return j < ns ? BKV * j : r.lo + BKV * (j - ns); }
    // the window keys [a, b) of tile X's rows (sinks that reach into the window begin it)
    __device__ __forceinline__ void range(const WindowArgs& p, int X, int& a, int& b) const {
        const int n = min(rows - BQ * X, BQ), q = pos0 + BQ * X;
        a = p.sinks > r.lo ? r.lo : max(q - p.left, r.lo);
        b = n > 0 ? max(min(q + n + p.right, r.hi), a) : a;
    }
    // whether tile X meets keys of half y of key tile j (sinks lie in front of the window: every row sees them)
    __device__ __forceinline__ bool sees(int X, int j, int y, int a, int b) const {
        const int t0 = start(j) + HALF * y;
        return j < ns ? rows > BQ * X && t0 < r.sk : t0 < b && t0 + HALF > a;
    }
};

struct RowState {
    float m, l;          // reference maximum (log2 units) and the sum of exponentials above it
    bool first;
};

// the keys 32 i .. 32 i + 31 of a tile that a row sees: those from lo on, or before sk, up to hi
__device__ __forceinline__ uint32_t visible(int lo, int hi, int sk, int i) {
    return win::low_bits(hi - 32 * i) & (~win::low_bits(lo - 32 * i) | win::low_bits(sk - 32 * i));
}

// One masked key tile of NC keys: its exponentials as bf16 pairs in the front of s, the row's sum and reference
// brought up to date.  Returns the factor for O (1: none).
template <int NC>
__device__ __forceinline__ float softmax_tile(uint32_t (&s)[NC], float c, RowState& st) {
    // the row maximum in eight independent chains (a NaN anywhere makes it NaN)
    float m8[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m8[i] = max_nan(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
#pragma unroll
    for (int k = 16; k < NC; k += 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m8[i] = max3_nan(m8[i], __uint_as_float(s[k + 2 * i]), __uint_as_float(s[k + 2 * i + 1]));
    }
    const float mt = c * max3_nan(max3_nan(m8[0], m8[1], m8[2]), max3_nan(m8[3], m8[4], m8[5]), max_nan(m8[6], m8[7]));
    float f = 1.f;
    if (mt > st.m + kLazy) {   // raise the reference maximum (always on the first tile with a visible key)
        f = ex2(st.m - mt);
        st.m = mt;
        st.l *= f;
    }
    if (mt != mt) st.l = NAN;   // (the FMA pipe's exponential of a NaN may be finite)
    // nothing seen so far: any finite reference serves, as every weight is zero
    const float ref = st.m == -INFINITY ? 0.f : st.m;
    const uint64_t c2 = f2(c, c), nm2 = f2(-ref, -ref);
    uint64_t ls[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k2 = 0; k2 < NC / 2; ++k2) {
        const uint64_t x = f2_fma(f2(__uint_as_float(s[2 * k2]), __uint_as_float(s[2 * k2 + 1])), c2, nm2);
        float p0, p1;
        if ((k2 & 7) >= 8 - EMU) {
            ex2_poly2_fine(x, p0, p1);   // (a cubic's 7.6e-5 would show in the log-sum-exp of a few keys)
        } else {
            float x0, x1;
            f2_split(x, x0, x1);
            p0 = ex2(x0);
            p1 = ex2(x1);
        }
        ls[k2 & 3] = f2_add(ls[k2 & 3], f2(p0, p1));
        s[k2] = pack_bf16(p0, p1);
    }
    float a0, a1;
    f2_split(f2_add(f2_add(ls[0], ls[1]), f2_add(ls[2], ls[3])), a0, a1);
    st.l += a0 + a1;
    return f;
}

__global__ void __launch_bounds__(THREADS, 1) window_fwd_kernel(const __grid_constant__ FwdArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);   // (an offset: the pointer stays known as shared)
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_SLOT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint4* bad_rows = reinterpret_cast<uint4*>(bars + B_BAD);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const win::ItemQueue items{bars + B_IF, bars + B_IE, reinterpret_cast<volatile int*>(bars + B_ITEM), abort_flag};

    if (tid == 0) {
        items.init(2 + 1 + SOFT);   // MMA issuers, screen, softmax warps
        tc::mbar_init(bars + B_QF, 1);
        tc::mbar_init(bars + B_QE, 2);
        for (int s = 0; s < NST; ++s) {
            tc::mbar_init(bars + B_KF + s, 1);
            tc::mbar_init(bars + B_VF + s, 1);
            tc::mbar_init(bars + B_VS + s, 1);
            tc::mbar_init(bars + B_KVE + s, 4);
        }
        for (int z = 0; z < 4; ++z) {
            tc::mbar_init(bars + B_SF + z, 1);
            tc::mbar_init(bars + B_PF + z, 4);
            tc::mbar_init(bars + B_OD + z, 1);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&p.mapQ);
        tc::tma_prefetch_desc(&p.mapK);
        tc::tma_prefetch_desc(&p.mapV);
    }
    uint8_t* order = sm + OFF_ORDER;
    long long n_items = p.n_items;
    if (warp == SOFT && p.sorted)   // (a tile of one row block costs three fifths of one of both)
        n_items = (long long)p.w.Hq * win::order_blocks(order, (int)p.n_items / p.w.Hq, [&](int b) {
            Item q;
            return q.load(p.w, (long long)b * p.w.Hq) ? q.nt * (q.rows > BQ ? 5 : 3) : -1;
        });
    if (warp == SOFT + 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    if (blockIdx.x == 0) {
        const SeqOffsets cq{p.w.cu_q, p.w.n_seq, p.w.Tq}, ck{p.w.cu_k, p.w.n_seq, p.w.Tk};
        for (int s = tid; s <= p.w.n_seq; s += THREADS)
            if (cq.bad(s) || ck.bad(s)) atomicOr(p.w.status, kStatusBadOffsets);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *tmem_slot;

    auto give_up = [&]() {
        *abort_flag = 1;
        atomicOr(p.w.status, kStatusTimeout);
    };
    Item it;

    if (warp == SOFT) {
        // ---------------- TMA producer: the item's Q tiles, then its K and V tiles through the ring
        if (tc::elect_one()) {
            int gkv = 0, n = 0;
            bool ok = true;
            for (int ticket = blockIdx.x, next, k = 0; ok && !*abort_flag; ticket = next) {
                if (ticket >= n_items) {
                    ok = items.put(k, -1);
                    break;
                }
                next = gridDim.x + atomicAdd(p.w.status + kTicket, 1);
                const int w = p.sorted ? order[ticket / p.w.Hq] * p.w.Hq + ticket % p.w.Hq : ticket;
                if (!it.load(p.w, w)) continue;
                if (!items.put(k++, w)) { ok = false; break; }
                if (n > 0 && !tc::mbar_wait(bars + B_QE, (n - 1) & 1, abort_flag, win::kItemWait)) { ok = false; break; }
                ++n;
                const int xq = it.h * DH, xk = it.hk * DH;
                tc::mbar_arrive_expect_tx(bars + B_QF, 2 * TILE);
                tc::tma_load_2d(sm + OFF_Q, &p.mapQ, xq, it.q_lo, bars + B_QF);
                // tile B past the last row: load tile A's rows again (its rows are never stored)
                tc::tma_load_2d(sm + OFF_Q + TILE, &p.mapQ, xq, it.rows > BQ ? it.q_lo + BQ : it.q_lo, bars + B_QF);
                for (int j = 0; j < it.nt; ++j, ++gkv) {
                    const int s = gkv % NST, use = gkv / NST, row = it.k0 + it.start(j);
                    if (use > 0 && !tc::mbar_wait(bars + B_KVE + s, (use - 1) & 1, abort_flag)) { ok = false; break; }
                    uint8_t* kt = sm + OFF_KV + s * 2 * TILE;
                    tc::mbar_arrive_expect_tx(bars + B_KF + s, TILE);
                    tc::tma_load_2d(kt, &p.mapK, xk, row, bars + B_KF + s);
                    tc::mbar_arrive_expect_tx(bars + B_VF + s, TILE);
                    tc::tma_load_2d(kt + TILE, &p.mapV, xk, row, bars + B_VF + s);
                }
            }
            if (!ok) give_up();
        }
    } else if (warp == SOFT + 3) {
        // ---------------- value screen: lane takes rows lane, lane + 32, ...; a row's 128 bytes are contiguous
        // (the swizzle permutes its 16-byte chunks), chunks taken in a rotated order for the banks
        int gkv = 0;
        bool ok = true;
        const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
        for (int k = 0; ok; ++k) {
            const int w = items.take_warp(k);
            if (w < 0) {
                ok = w == -1;
                break;
            }
            it.load(p.w, w);
            for (int j = 0; j < it.nt; ++j, ++gkv) {
                const int s = gkv % NST, use = gkv / NST;
                if (!__all_sync(0xffffffffu, tc::mbar_wait(bars + B_VF + s, use & 1, abort_flag))) { ok = false; break; }
                uint8_t* vt = sm + OFF_KV + s * 2 * TILE + TILE;
                uint32_t word[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint4* row = reinterpret_cast<uint4*>(vt + (32 * g + lane) * 128);
                    __nv_bfloat162 acc = zero;
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) {
                        const uint4 v = row[(ch + lane) & 7];
                        acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.x), zero, acc);
                        acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.y), zero, acc);
                        acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.z), zero, acc);
                        acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&v.w), zero, acc);
                    }
                    const bool bad = !(__low2float(acc) == 0.f && __high2float(acc) == 0.f);
                    word[g] = __ballot_sync(0xffffffffu, bad);
                    if (bad) {
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch) row[ch] = make_uint4(0, 0, 0, 0);
                    }
                }
                if (lane == 0) bad_rows[s] = make_uint4(word[0], word[1], word[2], word[3]);
                if (word[0] | word[1] | word[2] | word[3]) tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + B_VS + s);
            }
        }
        if (!ok && lane == 0) give_up();
    } else if (warp > SOFT) {
        // ---------------- MMA issuers, one per tile X; its two streams in turn: P V of the stream's last half tile,
        // once P lies in S's place, and the S of its next one in order behind it
        const int X = warp - SOFT - 1;
        if (tc::elect_one()) {
            constexpr uint32_t ID_S = tc::instr_desc(1, BQ, HALF, 0, 0);     // bf16, both K-major
            constexpr uint32_t ID_PV = tc::instr_desc(1, BQ, DH, 0, 1);      // bf16, A in tensor memory, V MN-major
            const uint64_t dQ = kmajor_desc(sm + OFF_Q + X * TILE);
            int gkv = 0, gs[2] = {0, 0}, n = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int w = items.take(k);
                if (w < 0) {
                    ok = w == -1;
                    break;
                }
                it.load(p.w, w);
                int a, b;
                it.range(p.w, X, a, b);
                if (!tc::mbar_wait(bars + B_QF, n & 1, abort_flag, win::kItemWait)) { ok = false; break; }
                ++n;
                tc::tc_fence_after();
                int pending[2] = {-1, -1};   // the stage whose P V is to come
                bool more[2] = {false, false};
                auto pv = [&](int y) {
                    const int s = pending[y];
                    if (!tc::mbar_wait(bars + B_PF + 2 * X + y, gs[y] & 1, abort_flag)) return false;
                    ++gs[y];
                    tc::tc_fence_after();
                    const uint32_t tS = tm + TM_X * X + HALF * y;
                    const uint64_t dV = mnmajor_desc(sm + OFF_KV + s * 2 * TILE + TILE + y * (TILE / 2));
#pragma unroll
                    for (int kk = 0; kk < HALF / 16; ++kk)
                        tc::mma_f16_ts(tS + TM_O, tS + 8 * kk, dV + (uint64_t)(kk * 128), ID_PV, (more[y] || kk > 0) ? 1u : 0u);
                    more[y] = true;
                    tc::mma_commit(bars + B_KVE + s);
                    return true;
                };
                for (int j = 0; j < it.nt && ok; ++j, ++gkv) {
                    const int s = gkv % NST, use = gkv / NST;
                    // (also where a half is not seen: the arrival then counts for this use of the stage)
                    if (!tc::mbar_wait(bars + B_KF + s, use & 1, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        if (pending[y] >= 0 && !pv(y)) { ok = false; break; }
                        pending[y] = -1;
                        if (!it.sees(X, j, y, a, b)) {
                            tc::mbar_arrive(bars + B_KVE + s);
                            continue;
                        }
                        const uint64_t dK = kmajor_desc(sm + OFF_KV + s * 2 * TILE + y * (TILE / 2));
#pragma unroll
                        for (int kk = 0; kk < DH / 16; ++kk)
                            tc::mma_f16_ss(tm + TM_X * X + HALF * y, dQ + 2 * kk, dK + 2 * kk, ID_S, kk > 0);
                        tc::mma_commit(bars + B_SF + 2 * X + y);
                        pending[y] = s;
                    }
                }
                if (ok) tc::mma_commit(bars + B_QE);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    if (ok && pending[y] >= 0) ok = pv(y);
                    if (ok && more[y]) tc::mma_commit(bars + B_OD + 2 * X + y);
                }
            }
            if (!ok) give_up();
        }
    } else {
        // ---------------- softmax groups: thread = query row r of tile X, half y of each key tile
        const int X = warp / (SOFT / 2), y = (warp >> 2) & 1, z = 2 * X + y, qd = warp & 3, r = 32 * qd + lane;
        const uint32_t lanes = (uint32_t)(32 * qd) << 16, tX = tm + lanes + TM_X * X, tS = tX + HALF * y, tO = tS + TM_O;
        float2* ml = reinterpret_cast<float2*>(sm + OFF_ML) + 256 * X;
        const float c = p.c;
        int gs = 0, gkv = 0, nonfinite = 0, complete[2] = {0, 0};
        bool ok = true;
        // every branch below is uniform over the warp (the item, the key tile, the waits' outcome)
        auto wait_all = [&](uint64_t* bar, uint32_t parity) {
            const bool got = tc::mbar_wait(bar, parity, abort_flag);
            return __all_sync(0xffffffffu, got);
        };
        for (int k = 0;; ++k) {
            // the two halves of a row go on or stop together: they meet at barriers below
            int w = ok ? items.take_warp(k) : -2;
            if (w == -2) {
                ok = false;
                w = -1;
            }
            if (tc::bar_sync_or(1 + X, 256, w < 0)) break;
            it.load(p.w, w);
            int a, b;
            it.range(p.w, X, a, b);
            const int pos = it.pos0 + BQ * X + r;
            RowState st{-INFINITY, 0.f, true};
            for (int j = 0; j < it.nt && ok; ++j, ++gkv) {
                if (!it.sees(X, j, y, a, b)) continue;
                // the keys of this half that the row sees, as bits
                const int t0 = it.start(j) + HALF * y;
                int lo = 0, hi = it.r.sk - t0, sk = 0;
                if (j >= it.ns) {
                    lo = pos - p.w.left - t0;
                    hi = min(pos + p.w.right + 1, it.nk) - t0;
                    sk = p.w.sinks - t0;
                }
                const bool whole = __all_sync(0xffffffffu, hi >= HALF && lo <= 0);
                if (!wait_all(bars + B_SF + z, gs & 1)) { ok = false; break; }
                tc::tc_fence_after();
                uint32_t s[HALF];
                tc::tmem_ld_32x32b_x32(tS, *reinterpret_cast<uint32_t(*)[32]>(s));
                tc::tmem_ld_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
                tc::tmem_wait_ld();
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < HALF / 32; ++i) {
                        const uint32_t vis = visible(lo, hi, sk, i);
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[32 * i + e] = (vis >> e) & 1u ? s[32 * i + e] : 0xff800000u;   // -inf
                    }
                }
                const float f = softmax_tile<HALF>(s, c, st);
                // the screened values: a row that sees one that is not finite becomes NaN
                const int stage = gkv % NST;
                if (!wait_all(bars + B_VS + stage, (gkv / NST) & 1)) { ok = false; break; }
                const uint2 bad = reinterpret_cast<const uint2*>(bad_rows + stage)[y];
                if (bad.x | bad.y) {
                    if ((bad.x & visible(lo, hi, sk, 0)) | (bad.y & visible(lo, hi, sk, 1))) st.l = NAN;
                }
                if (__any_sync(0xffffffffu, f != 1.f && !st.first)) {   // S's arrival says that O is stable
                    uint32_t o[16];
#pragma unroll
                    for (int q = 0; q < DH / 16; ++q) {
                        tc::tmem_ld_32x32b_x16(tO + 16 * q, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc::tmem_st_32x32b_x16(tO + 16 * q, o);
                    }
                }
                st.first = false;
                tc::tmem_st_32x32b_x32(tS, *reinterpret_cast<uint32_t(*)[32]>(s));
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + B_PF + z);
                ++gs;
            }
            // ---- epilogue: the halves' O joined, / l (+ residual) as bf16, 32 columns a thread; log-sum-exp
            ml[128 * y + r] = make_float2(st.m, st.first ? -1.f : st.l);   // (no step: a sum of -1)
            if (tc::bar_sync_or(1 + X, 256, !ok)) {
                ok = false;
                continue;
            }
            const bool has[2] = {ml[r].y != -1.f, ml[128 + r].y != -1.f};   // (the same for every row)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (has[q]) ok = wait_all(bars + B_OD + 2 * X + q, complete[q]++ & 1) && ok;
            }
            if (!ok) continue;
            tc::tc_fence_after();
            float2 ml0 = ml[r], ml1 = ml[128 + r];
            if (!has[0]) ml0.y = 0.f;
            if (!has[1]) ml1.y = 0.f;
            const float m = fmaxf(ml0.x, ml1.x), ref = m == -INFINITY ? 0.f : m;
            // a row without keys; one whose scores are all -infinity has keys, and is NaN as in the formula
            const int end = min(pos + p.w.right + 1, it.nk);
            const bool empty = end <= max(pos - p.w.left, 0) && min(p.w.sinks, end) <= 0;
            // NaN sums stay (a half whose maximum is -infinity has factor 0 and, unless it saw a NaN, a finite sum)
            const float f0 = ex2(ml0.x - ref), f1 = ex2(ml1.x - ref);
            const float l = m == -INFINITY ? NAN : ml0.y * f0 + ml1.y * f1;
            const float inv = 1.0f / l, g0 = f0 * inv, g1 = f1 * inv;
            uint32_t o0[32], o1[32];
            tc::tmem_ld_32x32b_x32(tX + TM_O + 32 * y, o0);
            tc::tmem_ld_32x32b_x32(tX + TM_O + HALF + 32 * y, o1);
            tc::tmem_wait_ld();
            tc::tc_fence_before();
            if (BQ * X + r < it.rows) {
                const long long t = it.q_lo + BQ * X + r, col = (long long)it.h * DH + 32 * y;
                const uint4* xr = p.w.Xres ? reinterpret_cast<const uint4*>(p.w.Xres + t * p.w.ld_out + col) : nullptr;
                uint4* dst = reinterpret_cast<uint4*>(p.w.Out + t * p.w.ld_out + col);
#pragma unroll
                for (int c8 = 0; c8 < 4; ++c8) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {   // what a half without a step left in tensor memory is not used
                        const float a0 = has[0] ? __uint_as_float(o0[8 * c8 + e]) * g0 : 0.f;
                        const float a1 = has[1] ? __uint_as_float(o1[8 * c8 + e]) * g1 : 0.f;
                        v[e] = empty ? 0.f : l == l ? a0 + a1 : l;
                    }
                    if (xr) {
                        const uint4 xv = xr[c8];
                        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 b2 = *reinterpret_cast<const __nv_bfloat162*>(&xw[e]);
                            v[2 * e] += __low2float(b2);
                            v[2 * e + 1] += __high2float(b2);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) nonfinite |= !isfinite(v[e]);
                    dst[c8] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                         pack_bf16(v[6], v[7]));
                }
                if (p.w.Lse && y == 0)
                    p.w.Lse[(long long)it.h * p.w.Tq + t] = empty ? -INFINITY : ref * 0.69314718055994531f + logf(l);
            }
            // (the next item's first barrier keeps both halves from each other's O until it has been read)
        }
        if (!ok) {
            if (lane == 0) give_up();
        }
        if (__any_sync(0xffffffffu, nonfinite) && lane == 0) atomicOr(p.w.status, kStatusNonFinite);
    }

    if (*abort_flag) {
        // let copies and products already in flight land before the CTA's memory goes away
        const uint64_t t0 = tc::globaltimer_ns();
        while (tc::globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == SOFT + 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tm, 512);
    }
}

}  // namespace

cudaError_t launch_window_attention(const WindowArgs& a, cudaStream_t s) {
    FwdArgs p{};
    p.w = a;
    // without keys the tiles are never loaded; any valid array serves the maps
    const void *K = a.Tk ? a.K : a.Q, *V = a.Tk ? a.V : a.Q;
    if (!make_map(&p.mapQ, a.Q, a.Tq, a.Hq * DH, a.ld_q) ||
        !make_map(&p.mapK, K, a.Tk ? a.Tk : a.Tq, (a.Tk ? a.Hk : a.Hq) * DH, a.Tk ? a.ld_k : a.ld_q) ||
        !make_map(&p.mapV, V, a.Tk ? a.Tk : a.Tq, (a.Tk ? a.Hk : a.Hq) * DH, a.Tk ? a.ld_v : a.ld_q))
        return cudaErrorInvalidValue;
    p.c = a.scale * 1.4426950408889634f;
    p.n_items = win::block_numbers<ROWS>(a.Tq, a.n_seq) * a.Hq;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    p.sorted = win::ordered(a, p.n_items / a.Hq, sms);
    cudaError_t e = cudaFuncSetAttribute(window_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    LaunchScope scope("window_attn", s);
    window_fwd_kernel<<<(unsigned)(p.n_items < sms ? p.n_items : sms), THREADS, SMEM_BYTES, s>>>(p);
    return cudaGetLastError();
}

}  // namespace ttt
