// Window attention, backward: delta = rowsum(dO Out), and dQ on the tcgen05 tensor cores (dK and dV have a
// kernel of their own: each sum has one owner and one order, at the price of computing the scores twice).
//   dQ_i = scale sum_u dS_iu k_u,  dS = P (dO.v - delta),  P = exp(scale q.k - lse)
//
// Work: an item is 256 query rows of a sequence (tiles A and B of 128) of one head, walking the forward pass's
// key tiles in steps of 64 keys: S_X = Q_X K^T and dP_X = dO_X V^T into tensor memory, dS_X back to it as bf16,
// dQ_X += dS_X K.  A thread holds 32 scores and products of its query row; lse and delta are two registers.
// Roles (640 threads): warps 0-7 tile A, 8-15 tile B, warp 16 the TMA producer, warps 17 and 18 the MMA issuers,
// warp 19 zeroes key rows that are not finite.
// Tensor memory, tile X: S 256 X, dP 256 X + 64, dQ 256 X + 128, dS 256 X + 192.
// Every wait is bounded, as in the forward kernel.
#include "window_bwd.cuh"

namespace ttt {
namespace {

using namespace winb;

constexpr int ROWS = 2 * BT, NST = 4;
constexpr int OFF_Q = 0;                          // Q_A, Q_B, dO_A, dO_B
constexpr int OFF_KV = 4 * TILE;                  // stage s: K at OFF_KV + 2 s TILE, V after it
constexpr int OFF_BAR = OFF_KV + NST * 2 * TILE;
constexpr int OFF_ORDER = OFF_BAR + 512;          // [kOrder] bytes
constexpr int SMEM_BYTES = OFF_ORDER + win::kOrder + 1024;
constexpr uint32_t TM_X = 256, TM_S = 0, TM_DP = 64, TM_DQ = 128, TM_DS = 192;

enum : int {
    B_QF = 0,              // Q and dO landed
    B_QE = 1,              // the item's S and dP products are done (2 arrivals)
    B_KF = 2,              // [NST] K and V landed
    B_SC = 2 + NST,        // [NST] K's rows that must not take part are zeroed
    B_KVE = 2 + 2 * NST,   // [NST] both tiles are done with the stage (2 arrivals)
    B_SF = 2 + 3 * NST,    // [2] S_X and dP_X in tensor memory
    B_SR = B_SF + 2,       // [2] the group has read them (4 warps)
    B_PF = B_SR + 2,       // [2] dS_X written (4 warps)
    B_PV = B_PF + 2,       // [2] its product is done
    B_SLOT = B_PV + 2,
    B_BAD = 32,            // [NST] 16 bytes: bits of the stage's key rows that are not finite
    B_IF = B_BAD + 2 * NST,  // [4] the CTA's items: handed out, taken; their numbers (4 ints)
    B_IE = B_IF + win::kItemSlots,
    B_ITEM = B_IE + win::kItemSlots
};
static_assert(B_SLOT < B_BAD && B_BAD % 2 == 0 && B_ITEM * 8 + 16 <= 512, "barrier area");
constexpr int kTicket = 2;   // the item counter's place behind the status word (cleared with it)
static_assert(SMEM_BYTES <= 232448, "shared memory");

struct QArgs {
    CUtensorMap mapQ, mapK, mapV, mapDO;
    WindowArgs w;
    long long n_items;
    int sorted;                     // few blocks of unequal work: drawn by it
    float c;
};

struct Item {
    int q_lo, rows, pos0, k0, nk, h, hk;
    int ns, nt;
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
        ns = (r.sk + BT - 1) / BT;
        nt = ns + (r.hi - r.lo + BT - 1) / BT;
        return true;
    }
    __device__ __forceinline__ int start(int j) const { return j < ns ? BT * j : r.lo + BT * (j - ns); }
    // the window keys [a, b) of tile X's rows (sinks that reach into the window begin it)
    __device__ __forceinline__ void range(const WindowArgs& p, int X, int& a, int& b) const {
        const int n = min(rows - BT * X, BT), q = pos0 + BT * X;
        a = p.sinks > r.lo ? r.lo : max(q - p.left, r.lo);
        b = n > 0 ? max(min(q + n + p.right, r.hi), a) : a;
    }
    // whether tile X meets keys of half hh of key tile j
    __device__ __forceinline__ bool sees(int X, int j, int hh, int a, int b) const {
        const int t0 = start(j) + HALF * hh;
        return j < ns ? rows > BT * X && t0 < r.sk : t0 < b && t0 + HALF > a;
    }
};

__global__ void __launch_bounds__(THREADS, 1) window_dq_kernel(const __grid_constant__ QArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);   // (an offset: the pointer stays known as shared)
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_SLOT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint4* bad_rows = reinterpret_cast<uint4*>(bars + B_BAD);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const win::ItemQueue items{bars + B_IF, bars + B_IE, reinterpret_cast<volatile int*>(bars + B_ITEM), abort_flag};

    if (tid == 0) {
        items.init(2 + 1 + SOFT);   // MMA issuers, side warps, softmax warps
        tc::mbar_init(bars + B_QF, 1);
        tc::mbar_init(bars + B_QE, 2);
        for (int s = 0; s < NST; ++s) {
            tc::mbar_init(bars + B_KF + s, 1);
            tc::mbar_init(bars + B_SC + s, 1);
            tc::mbar_init(bars + B_KVE + s, 2);
        }
        for (int x = 0; x < 2; ++x) {
            tc::mbar_init(bars + B_SF + x, 1);
            tc::mbar_init(bars + B_SR + x, SOFT / 2);
            tc::mbar_init(bars + B_PF + x, SOFT / 2);
            tc::mbar_init(bars + B_PV + x, 1);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&p.mapQ);
        tc::tma_prefetch_desc(&p.mapK);
        tc::tma_prefetch_desc(&p.mapV);
        tc::tma_prefetch_desc(&p.mapDO);
    }
    uint8_t* order = sm + OFF_ORDER;
    long long n_items = p.n_items;
    if (warp == SOFT && p.sorted)
        n_items = (long long)p.w.Hq * win::order_blocks(order, (int)p.n_items / p.w.Hq, [&](int b) {
            Item q;
            return q.load(p.w, (long long)b * p.w.Hq) ? q.nt * (q.rows > BT ? 5 : 3) : -1;
        });
    if (warp == SOFT + 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *tmem_slot;

    auto give_up = [&]() {
        *abort_flag = 1;
        atomicOr(p.w.status, kStatusTimeout);
    };
    // waits of a whole warp, so that every branch after it is uniform
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        const bool got = tc::mbar_wait(bar, parity, abort_flag);
        return __all_sync(0xffffffffu, got);
    };
    Item it;

    if (warp == SOFT) {
        // ---------------- TMA producer
        if (tc::elect_one()) {
            int g = 0, n = 0;
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
                // tile B past the last row: tile A's rows again (its results are never stored)
                const int q_b = it.rows > BT ? it.q_lo + BT : it.q_lo;
                tc::mbar_arrive_expect_tx(bars + B_QF, 4 * TILE);
                tc::tma_load_2d(sm + OFF_Q, &p.mapQ, xq, it.q_lo, bars + B_QF);
                tc::tma_load_2d(sm + OFF_Q + TILE, &p.mapQ, xq, q_b, bars + B_QF);
                tc::tma_load_2d(sm + OFF_Q + 2 * TILE, &p.mapDO, xq, it.q_lo, bars + B_QF);
                tc::tma_load_2d(sm + OFF_Q + 3 * TILE, &p.mapDO, xq, q_b, bars + B_QF);
                for (int j = 0; j < it.nt; ++j, ++g) {
                    const int s = g % NST, use = g / NST, row = it.k0 + it.start(j);
                    if (use > 0 && !tc::mbar_wait(bars + B_KVE + s, (use - 1) & 1, abort_flag)) { ok = false; break; }
                    uint8_t* kt = sm + OFF_KV + s * 2 * TILE;
                    tc::mbar_arrive_expect_tx(bars + B_KF + s, 2 * TILE);
                    tc::tma_load_2d(kt, &p.mapK, xk, row, bars + B_KF + s);
                    tc::tma_load_2d(kt + TILE, &p.mapV, xk, row, bars + B_KF + s);
                }
            }
            if (!ok) give_up();
        }
    } else if (warp == SOFT + 3) {
        // ---------------- key rows that are not finite, or behind the sequence's last key
        int g = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int w = items.take_warp(k);
            if (w < 0) {
                ok = w == -1;
                break;
            }
            it.load(p.w, w);
            for (int j = 0; j < it.nt; ++j, ++g) {
                const int s = g % NST, use = g / NST, u0 = it.start(j);
                const uint8_t* odd = p.w.key_odd + (long long)it.hk * p.w.Tk + it.k0;
                uint32_t bad[4], out[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int u = u0 + 32 * e + lane;
                    bad[e] = __ballot_sync(0xffffffffu, u < it.nk && odd[u]);
                    out[e] = bad[e] | ~win::low_bits(it.nk - u0 - 32 * e);
                }
                if (!wait_all(bars + B_KF + s, use & 1)) { ok = false; break; }
                if (out[0] | out[1] | out[2] | out[3]) {
                    zero_rows(sm + OFF_KV + s * 2 * TILE, lane, out);
                    tc::fence_proxy_async_smem();
                }
                if (lane == 0) bad_rows[s] = make_uint4(bad[0], bad[1], bad[2], bad[3]);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + B_SC + s);
            }
        }
        if (!ok && lane == 0) give_up();
    } else if (warp > SOFT) {
        // ---------------- MMA issuers, one per tile: S_X and dP_X of a step, then the product of the step before
        const int X = warp - SOFT - 1;
        if (tc::elect_one()) {
            constexpr uint32_t ID_S = tc::instr_desc(1, BT, HALF, 0, 0);   // both K-major
            constexpr uint32_t ID_Q = tc::instr_desc(1, BT, DH, 0, 1);     // A in tensor memory, B MN-major
            const uint64_t dQ = kmajor_desc(sm + OFF_Q + X * TILE), dO = kmajor_desc(sm + OFF_Q + (2 + X) * TILE);
            const uint32_t tX = tm + TM_X * X;
            int g = 0, gs = 0, n = 0;
            bool ok = true;
            // the product of step gs - 1: half hh of stage s, and the stage's release after X's last half in it
            auto product = [&](int s, int hh, bool accumulate, bool release) {
                if (!tc::mbar_wait(bars + B_PF + X, (gs - 1) & 1, abort_flag)) return false;
                tc::tc_fence_after();
                const uint64_t mK = mnmajor_desc(sm + OFF_KV + s * 2 * TILE + hh * (TILE / 2));
#pragma unroll
                for (int kk = 0; kk < HALF / 16; ++kk)
                    tc::mma_f16_ts(tX + TM_DQ, tX + TM_DS + 8 * kk, mK + (uint64_t)(kk * 128), ID_Q,
                                   (accumulate || kk > 0) ? 1u : 0u);
                tc::mma_commit(bars + B_PV + X);
                if (release) tc::mma_commit(bars + B_KVE + s);
                return true;
            };
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
                int done = 0, ps = -1, ph = 0;
                bool prel = false;
                for (int j = 0; j < it.nt && ok; ++j, ++g) {
                    const int s = g % NST, use = g / NST;
                    if (!tc::mbar_wait(bars + B_KF + s, use & 1, abort_flag)) { ok = false; break; }
                    const bool first = it.sees(X, j, 0, a, b), second = it.sees(X, j, 1, a, b);
                    if (!first && !second) {
                        tc::mbar_arrive(bars + B_KVE + s);
                        continue;
                    }
                    for (int hh = 0; hh < 2; ++hh) {
                        if (!(hh ? second : first)) continue;
                        if (gs > 0 && !tc::mbar_wait(bars + B_SR + X, (gs - 1) & 1, abort_flag)) { ok = false; break; }
                        tc::tc_fence_after();
                        const uint8_t* kt = sm + OFF_KV + s * 2 * TILE + hh * (TILE / 2);
                        const uint64_t dK = kmajor_desc(kt), dV = kmajor_desc(kt + TILE);
#pragma unroll
                        for (int kk = 0; kk < DH / 16; ++kk)
                            tc::mma_f16_ss(tX + TM_S, dQ + 2 * kk, dK + 2 * kk, ID_S, kk > 0);
#pragma unroll
                        for (int kk = 0; kk < DH / 16; ++kk)
                            tc::mma_f16_ss(tX + TM_DP, dO + 2 * kk, dV + 2 * kk, ID_S, kk > 0);
                        tc::mma_commit(bars + B_SF + X);
                        if (ps >= 0 && !product(ps, ph, done > 1, prel)) { ok = false; break; }
                        ++gs;
                        ++done;
                        ps = s;
                        ph = hh;
                        prel = hh == 1 || !second;
                    }
                }
                if (ok) tc::mma_commit(bars + B_QE);
                if (ok && ps >= 0 && !product(ps, ph, done > 1, prel)) ok = false;
            }
            if (!ok) give_up();
        }
    } else {
        // ---------------- softmax groups: thread = query row r of tile X, part y of each step's keys
        const int X = warp / (SOFT / 2), y = (warp >> 2) & 1, qd = warp & 3, r = 32 * qd + lane;
        const uint32_t tX = tm + TM_X * X + ((uint32_t)(32 * qd) << 16);
        const float c = p.c;
        int g = 0, gs = 0, nonfinite = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int w = items.take_warp(k);
            if (w < 0) {
                ok = w == -1;
                break;
            }
            it.load(p.w, w);
            int a, b;
            it.range(p.w, X, a, b);
            const int pos = it.pos0 + BT * X + r;
            const bool mine = BT * X + r < it.rows;
            const long long at = (long long)it.h * p.w.Tq + it.q_lo + BT * X + r;
            const float nl = mine ? -kLog2e * p.w.Lse[at] : 0.f, nd = mine ? -p.w.delta[at] : 0.f;
            const uint64_t nl2 = f2(nl, nl), nd2 = f2(nd, nd);
            bool any = false;
            for (int j = 0; j < it.nt && ok; ++j, ++g) {
                const int s = g % NST, use = g / NST;
                for (int hh = 0; hh < 2; ++hh) {
                    if (!it.sees(X, j, hh, a, b)) continue;
                    const int t0 = it.start(j) + HALF * hh + COLS * y;
                    int lo = 0, hi = it.r.sk - t0, sk = 0;
                    if (j >= it.ns) {
                        lo = pos - p.w.left - t0;
                        hi = min(pos + p.w.right + 1, it.nk) - t0;
                        sk = p.w.sinks - t0;
                    }
                    const bool whole = __all_sync(0xffffffffu, hi >= COLS && lo <= 0);
                    const uint32_t vis = win::low_bits(hi) & (~win::low_bits(lo) | win::low_bits(sk));
                    if (!wait_all(bars + B_SC + s, use & 1) || !wait_all(bars + B_SF + X, gs & 1)) { ok = false; break; }
                    tc::tc_fence_after();
                    const uint32_t bad = reinterpret_cast<const uint32_t*>(bad_rows + s)[2 * hh + y] & vis;
                    uint32_t sc[COLS], dp[COLS];
                    tc::tmem_ld_32x32b_x32(tX + TM_S + COLS * y, sc);
                    tc::tmem_ld_32x32b_x32(tX + TM_DP + COLS * y, dp);
                    tc::tmem_wait_ld();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bars + B_SR + X);
                    auto neg = [&](int, uint64_t& l0, uint64_t& l1, uint64_t& d0, uint64_t& d1) {
                        l0 = l1 = nl2;
                        d0 = d1 = nd2;
                    };
                    if (whole) grad_scores<true, false>(sc, dp, c, vis, bad, neg);
                    else grad_scores<false, false>(sc, dp, c, vis, bad, neg);
                    if (gs > 0) {
                        if (!wait_all(bars + B_PV + X, (gs - 1) & 1)) { ok = false; break; }
                        tc::tc_fence_after();
                    }
                    tc::tmem_st_32x32b_x16(tX + TM_DS + COLS / 2 * y, *reinterpret_cast<uint32_t(*)[16]>(dp));
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bars + B_PF + X);
                    ++gs;
                    any = true;
                }
            }
            if (!ok) break;
            // ---- epilogue
            if (any) {
                if (!wait_all(bars + B_PV + X, (gs - 1) & 1)) { ok = false; break; }
                tc::tc_fence_after();
            }
            uint32_t o[COLS];
            tc::tmem_ld_32x32b_x32(tX + TM_DQ + COLS * y, o);
            tc::tmem_wait_ld();
            if (!any) {   // rows that see nothing
#pragma unroll
                for (int e = 0; e < COLS; ++e) o[e] = 0;
            }
            if (mine && !RowKeys(p.w, it.pos0 + BT * X + r, it.nk).few()) {
                const long long t = it.q_lo + BT * X + r;
                nonfinite |= store_row(p.w.dQ + t * p.w.ld_dq + it.h * DH + COLS * y, o, p.w.grad_scale);
            }
        }
        if (!ok && lane == 0) give_up();
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
    // this kernel may have begun before the one of dK and dV ended; what follows in the stream waits for both
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// delta[h, t] = sum of dO Out over the head's columns, NaN where the row's q is not finite (so that delta is finite
// only where q, dO and Out are), and key_odd[h, u]: whether the key is not finite.  Eight lanes a row of 64, 16
// bytes each; a warp takes four consecutive rows of a few heads.  Also looks over the offsets.
//
// Out is rounded to bf16, and dP - delta of a row with few keys is small beside dP: with two keys the rounding put
// dQ and dK off by 0.0055 in the norm (0.0025 with many).  So a row of at most FEW keys gets delta = sum_u P_u dP_u,
// which is the same number, from the keys and values themselves, and its dQ here in fp32: scale (sum_u P_u dP_u k_u -
// delta sum_u P_u k_u).  (With the rounded dS, dQ of rows of five keys was off by 0.0026, more than the 0.0024 of long ones.)

__device__ __forceinline__ float dot8(const uint4& x, const uint4& y) {
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&xw[e]), b = *reinterpret_cast<const __nv_bfloat162*>(&yw[e]);
        sum = fmaf(__low2float(a), __low2float(b), sum);
        sum = fmaf(__high2float(a), __high2float(b), sum);
    }
    return sum;
}
__device__ __forceinline__ float sum8(float v) {   // over the eight lanes of a row
#pragma unroll
    for (int m = 1; m < 8; m *= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

constexpr int DELTA_HEADS = 2;   // of a warp: all loads first, the rows' sequences are looked up once

__global__ void __launch_bounds__(256) window_delta_kernel(const WindowArgs p, long long q_warps, long long warps) {
    const SeqOffsets cq{p.cu_q, p.n_seq, p.Tq}, ck{p.cu_k, p.n_seq, p.Tk};
    if (blockIdx.x == 0) {
        for (int s = threadIdx.x; s <= p.n_seq; s += blockDim.x)
            if (cq.bad(s) || ck.bad(s)) atomicOr(p.status, kStatusBadOffsets);
    }
    const int lane = threadIdx.x & 31;
    long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (w >= warps) return;
    const bool key = w >= q_warps;
    if (key) w -= q_warps;
    const int heads = key ? p.Hk : p.Hq, parts = (heads + DELTA_HEADS - 1) / DELTA_HEADS, rows = key ? p.Tk : p.Tq;
    const int h0 = (int)(w % parts) * DELTA_HEADS, h1 = min(h0 + DELTA_HEADS, heads);
    const long long t = w / parts * 4 + (lane >> 3);
    const bool in = t < rows;
    const uint4 none = make_uint4(0, 0, 0, 0);
    // this lane's row and columns of head 0
    const int col0 = (lane & 7) * 8;
    uint4 xs[DELTA_HEADS], gs[DELTA_HEADS], os[DELTA_HEADS];
#pragma unroll
    for (int i = 0; i < DELTA_HEADS; ++i) {
        const int col = (h0 + i) * DH + col0;
        const bool here = in && h0 + i < h1;
        xs[i] = here ? *reinterpret_cast<const uint4*>((key ? p.K + t * p.ld_k : p.Q + t * p.ld_q) + col) : none;
        gs[i] = here && !key ? *reinterpret_cast<const uint4*>(p.dOut + t * p.ld_do + col) : none;
        os[i] = here && !key ? *reinterpret_cast<const uint4*>(p.Out + t * p.ld_out + col) : none;
    }
    if (key) {
#pragma unroll
        for (int i = 0; i < DELTA_HEADS; ++i) {
            const int h = h0 + i;
            if (h >= h1) break;
            const uint4 x = xs[i];
            const uint32_t odd = __ballot_sync(0xffffffffu, odd_values(x)) >> (lane & 24) & 0xffu;   // of the row's eight lanes
            if (in && (lane & 7) == 0) p.key_odd[(long long)h * p.Tk + t] = odd ? 1 : 0;
        }
        return;
    }
    int k0 = 0, lo = 0, sk = 0, n = 0;
    if (in) {
        const int s = cq.find((int)t), q0 = cq.begin(s), q1 = cq.begin(s + 1);
        if (t >= q0 && t < q1) {
            k0 = ck.begin(s);
            const int nk = max(ck.begin(s + 1) - k0, 0);
            const RowKeys r(p, nk - (q1 - q0) + (int)t - q0, nk);
            lo = r.lo;
            n = r.n;
            sk = r.sk;
        }
    }
    const int most = __reduce_max_sync(0xffffffffu, sk + n <= FEW ? sk + n : 0);
#pragma unroll
    for (int e = 0; e < DELTA_HEADS; ++e) {
        const int h = h0 + e;
        if (h >= h1) break;
        const uint4 x = xs[e], g = gs[e], o = os[e];
        const uint32_t odd = __ballot_sync(0xffffffffu, odd_values(x)) >> (lane & 24) & 0xffu;
        float delta = sum8(dot8(g, o));
        if (most > 0) {
            const bool few = sk + n <= FEW && sk + n > 0;
            const float lse = few ? p.Lse[(long long)h * p.Tq + t] : 0.f;
            const int kcol = h / (p.Hq / p.Hk) * DH + col0;
            const float whole = delta;
            float sum = 0.f, pk[8] = {}, pdk[8] = {};
            for (int i = 0; i < most; ++i) {
                uint4 k = none, v = none;
                const bool seen = few && i < sk + n;
                if (seen) {
                    const long long u = k0 + (i < sk ? i : lo + i - sk);
                    k = *reinterpret_cast<const uint4*>(p.K + u * p.ld_k + kcol);
                    v = *reinterpret_cast<const uint4*>(p.V + u * p.ld_v + kcol);
                }
                const float score = sum8(dot8(x, k)), dp = sum8(dot8(g, v));
                if (!seen) continue;
                const float w = ex2(fmaf(score, p.scale * kLog2e, -kLog2e * lse)), wd = w * dp;
                sum += wd;
                const uint32_t kw[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float kc = __uint_as_float(c % 2 ? kw[c / 2] & 0xffff0000u : kw[c / 2] << 16);
                    pk[c] = fmaf(w, kc, pk[c]);
                    pdk[c] = fmaf(wd, kc, pdk[c]);
                }
            }
            if (few) {
                // a product of dO and Out that is not finite spoils the row; one key's weight is 1 whatever its score
                if (isfinite(whole)) delta = sum;
                const float scale = sk + n == 1 ? 0.f : p.grad_scale;
                float d[8];
                bool fine = true;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    d[c] = odd || !isfinite(whole) ? NAN : scale * fmaf(-delta, pk[c], pdk[c]);
                    fine &= isfinite(d[c]);
                }
                if (!fine) atomicOr(p.status, kStatusNonFinite);
                *reinterpret_cast<uint4*>(p.dQ + t * p.ld_dq + h * DH + col0) =
                    make_uint4(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7]));
            }
        }
        if (odd) delta = NAN;
        if (in && (lane & 7) == 0) p.delta[(long long)h * p.Tq + t] = delta;
    }
}

// after_dkv: the launch before is the one of dK and dV, whose end need not be waited for
cudaError_t launch_dq(const WindowArgs& a, int sms, bool after_dkv, cudaStream_t s) {
    QArgs p{};
    p.w = a;
    const bool k = a.Tk > 0;   // without keys the tiles are never loaded; any valid array serves the maps
    if (!make_map(&p.mapQ, a.Q, a.Tq, a.Hq * DH, a.ld_q) || !make_map(&p.mapDO, a.dOut, a.Tq, a.Hq * DH, a.ld_do) ||
        !make_map(&p.mapK, k ? a.K : a.Q, k ? a.Tk : a.Tq, (k ? a.Hk : a.Hq) * DH, k ? a.ld_k : a.ld_q) ||
        !make_map(&p.mapV, k ? a.V : a.Q, k ? a.Tk : a.Tq, (k ? a.Hk : a.Hq) * DH, k ? a.ld_v : a.ld_q))
        return cudaErrorInvalidValue;
    p.c = a.scale * kLog2e;
    p.n_items = win::block_numbers<ROWS>(a.Tq, a.n_seq) * a.Hq;
    p.sorted = win::ordered(a, p.n_items / a.Hq, sms);
    cudaError_t e = cudaFuncSetAttribute(window_dq_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.n_items < sms ? p.n_items : sms));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = after_dkv ? 1 : 0;
    LaunchScope scope("window_dq", s);
    return cudaLaunchKernelEx(&cfg, window_dq_kernel, p);
}

}  // namespace

cudaError_t launch_window_attention_backward(const WindowArgs& a, cudaStream_t s) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    {
        LaunchScope scope("window_delta", s);
        const auto parts = [](int heads) { return (heads + DELTA_HEADS - 1) / DELTA_HEADS; };
        const long long q = ((long long)a.Tq + 3) / 4 * parts(a.Hq), warps = q + ((long long)a.Tk + 3) / 4 * parts(a.Hk);
        window_delta_kernel<<<(unsigned)((warps + 7) / 8 ? (warps + 7) / 8 : 1), 256, 0, s>>>(a, q, warps);
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.Tk) e = launch_window_dkv(a, sms, s);
    if (e == cudaSuccess && a.Tq) e = launch_dq(a, sms, a.Tk > 0, s);
    if (e == cudaSuccess && a.Tk) e = launch_window_sink_sum(a, s);
    return e;
}

}  // namespace ttt
