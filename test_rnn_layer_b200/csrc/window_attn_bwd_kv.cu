// Window attention, backward: dK and dV on the tcgen05 tensor cores (head dim 64, bf16, fp32 accumulation).
//   P = exp(scale q.k - lse), dS = P (dO.v - delta), dV_u = sum_i P_iu dO_i, dK_u = scale sum_i dS_iu q_i
// over the queries i that see key u, of every query head that shares the key head.
//
// Work: an item is 128 keys of a sequence of one key head; it walks the query tiles of 128 rows that see them,
// head after head, so that each sum has one owner and one order (no atomics).  The transposed scores are
// computed, S^T = K Q^T and dP^T = V dO^T with a key per tensor-memory lane, so that P^T and dS^T are the A
// operands of dV += P^T dO and dK += dS^T Q straight from tensor memory.  Four softmax groups take 32 queries of
// a tile each: a thread holds 32 scores and 32 products of its key.  The rows' lse and delta lie in shared
// memory beside the tile.
//
// Roles (608 threads): warps 0-7 queries 0..63 of a tile, 8-15 queries 64..127, warp 16 the TMA producer, warp 17
// the MMA issuer (one, so that the sums' order is fixed), warp 18 loads lse and delta and zeroes rows that are not
// finite.
// Tensor memory (512 columns), half X: S 192 X, dP 192 X + 64, P 192 X + 128, dS 192 X + 160; dV 384, dK 448.
// Per tile of 128 x 128 scores the tensor cores have 4 products of 2.1 MFLOP and the exponential unit 14,336
// results (1,024 and 896 cycles).  Every wait is bounded, as in the forward kernel.
#include "window_bwd.cuh"

namespace ttt {
namespace {

using namespace winb;

constexpr int NST = 4;
constexpr int OFF_KV = 0;                             // item n: K at (n & 1) 2 TILE, V after it
constexpr int OFF_Q = 4 * TILE;                       // stage s: Q at OFF_Q + 2 s TILE, dO after it
constexpr int OFF_STAT = OFF_Q + NST * 2 * TILE;      // stage s: 128 x -lse2, 128 x -delta
constexpr int OFF_BAR = OFF_STAT + NST * 1024;
constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
constexpr int KV_THREADS = THREADS - 32;
constexpr uint32_t TM_X = 192, TM_S = 0, TM_DP = 64, TM_P = 128, TM_DS = 160, TM_DV = 384, TM_DK = 448;

enum : int {
    B_KVF = 0,             // [2] the item's K and V landed
    B_KVE = 2,             // [2] its S and dP products are done
    B_QF = 4,              // [NST] Q and dO landed
    B_ST = 4 + NST,        // [NST] lse and delta written, rows that must not take part zeroed
    B_QE = 4 + 2 * NST,    // [NST] stage free (a commit and 16 warps)
    B_SF = 4 + 3 * NST,    // [2] S_X and dP_X in tensor memory
    B_SR = B_SF + 2,       // [2] the group has read them (8 warps)
    B_PF = B_SR + 2,       // [2] P_X and dS_X written (8 warps)
    B_PV = B_PF + 2,       // [2] their products are done
    B_AF = B_PV + 2,       // the item's dV and dK are complete
    B_AE = B_AF + 1,       // and read (16 warps)
    B_SLOT = B_AE + 1,
    B_BAD = 36,            // [NST] 16 bytes: bits of the stage's query rows that are not finite
    B_IF = B_BAD + 2 * NST,  // [4] the CTA's items: handed out, taken; their numbers (4 ints)
    B_IE = B_IF + win::kItemSlots,
    B_ITEM = B_IE + win::kItemSlots
};
static_assert(B_SLOT < B_BAD && B_BAD % 2 == 0 && B_ITEM * 8 + 16 <= 512, "barrier area");
constexpr int kTicket = 1;   // the item counter's place behind the status word (cleared with it)
static_assert(SMEM_BYTES <= 232448, "shared memory");

struct KvArgs {
    CUtensorMap mapQ, mapK, mapV, mapDO;
    WindowArgs w;
    long long n_window, n_chunk, n_items;   // window items and chunks of the sinks' further queries
    int blocks;                    // key blocks with sinks
    int chunks_first;              // the longer kind of item goes first
    float c;
    int cut;                       // whether sinks are cut up (partial sums in w.partial)
};

struct Item {
    int k_lo, keys, u0, nk, hk;    // first key row, number of keys, its index in the sequence
    int q0, nq, first;             // the sequence's first query row, number of queries, position of query 0
    int i0, i1, h0, heads;         // query range, heads h0 .. h0 + heads - 1
    long long slot;                // partial sums go here (-1: the item's sums are dK and dV)

    __device__ __forceinline__ bool load(const KvArgs& a, long long w) {
        const WindowArgs& p = a.w;
        const SeqOffsets cq{p.cu_q, p.n_seq, p.Tq}, ck{p.cu_k, p.n_seq, p.Tk};
        const int G = p.Hq / p.Hk;
        const bool window = a.chunks_first ? w >= a.n_chunk : w < a.n_window;
        if (window && a.chunks_first) w -= a.n_chunk;
        if (!window && !a.chunks_first) w -= a.n_window;
        int s, c0 = 0, c1 = 0;
        long long number = 0;
        if (window) {
            hk = (int)(w % p.Hk);
            h0 = hk * G;
            heads = G;
            s = win::block_of<BT>(ck, (int)(w / p.Hk), k_lo, keys);
        } else {
            h0 = (int)(w % p.Hq);
            hk = h0 / G;
            heads = 1;
            number = w / p.Hq / a.blocks;
            s = win::block_of<CHUNK>(cq, (int)number, c0, c1);
            u0 = (int)(w / p.Hq % a.blocks) * BT;
        }
        if (s < 0) return false;
        q0 = cq.begin(s);
        nq = max(cq.begin(s + 1) - q0, 0);
        const int kb = ck.begin(s);
        nk = max(ck.begin(s + 1) - kb, 0);
        first = nk - nq;
        if (window) {
            u0 = k_lo - kb;
        } else {
            if (u0 >= min(p.sinks, nk)) return false;
            k_lo = kb + u0;
            keys = min(BT, nk - u0);
        }
        const QueryRange r = queries_of(u0, u0 + keys, first, nq, p.left, p.right);
        i0 = r.ia;
        i1 = r.ib;
        slot = -1;
        if (u0 < p.sinks && i1 < nq) {
            if (!a.cut) {
                i1 = nq;
            } else if (window) {
                slot = chunk_slots(p) + ((long long)s * p.Hk + hk) * SINK_BLOCKS + u0 / BT;
            }
        }
        if (!window) {
            i0 = max(i1, c0 - q0);
            i1 = min(nq, c0 - q0 + c1);
            if (i1 <= i0) return false;
            slot = (number * SINK_BLOCKS + u0 / BT) * p.Hq + h0;
        }
        return true;
    }
    __device__ __forceinline__ int tiles() const { return (i1 - i0 + BT - 1) / BT; }
};

__global__ void __launch_bounds__(KV_THREADS, 1) window_dkv_kernel(const __grid_constant__ KvArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);   // (an offset: the pointer stays known as shared)
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_SLOT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint4* bad_rows = reinterpret_cast<uint4*>(bars + B_BAD);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // dQ needs nothing of this kernel: its CTAs may take the SMs that this kernel's last items leave
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const win::ItemQueue items{bars + B_IF, bars + B_IE, reinterpret_cast<volatile int*>(bars + B_ITEM), abort_flag};

    if (tid == 0) {
        items.init(1 + 1 + SOFT);   // MMA issuers, side warps, softmax warps
        for (int x = 0; x < 2; ++x) {
            tc::mbar_init(bars + B_KVF + x, 1);
            tc::mbar_init(bars + B_KVE + x, 1);
            tc::mbar_init(bars + B_SF + x, 1);
            tc::mbar_init(bars + B_SR + x, SOFT / 2);
            tc::mbar_init(bars + B_PF + x, SOFT / 2);
            tc::mbar_init(bars + B_PV + x, 1);
        }
        for (int s = 0; s < NST; ++s) {
            tc::mbar_init(bars + B_QF + s, 1);
            tc::mbar_init(bars + B_ST + s, 1);
            tc::mbar_init(bars + B_QE + s, 1 + SOFT);
        }
        tc::mbar_init(bars + B_AF, 1);
        tc::mbar_init(bars + B_AE, SOFT);
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&p.mapQ);
        tc::tma_prefetch_desc(&p.mapK);
        tc::tma_prefetch_desc(&p.mapV);
        tc::tma_prefetch_desc(&p.mapDO);
    }
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
            for (int w = blockIdx.x, next, k = 0; ok && !*abort_flag; w = next) {
                if (w >= p.n_items) {
                    ok = items.put(k, -1);
                    break;
                }
                next = gridDim.x + atomicAdd(p.w.status + kTicket, 1);
                if (!it.load(p, w)) continue;
                if (!items.put(k++, w)) { ok = false; break; }
                if (it.tiles() == 0) continue;
                const int kv = n & 1, xk = it.hk * DH, tiles = it.tiles();
                if (n >= 2 && !tc::mbar_wait(bars + B_KVE + kv, ((n >> 1) - 1) & 1, abort_flag, win::kItemWait)) { ok = false; break; }
                uint8_t* kt = sm + OFF_KV + kv * 2 * TILE;
                tc::mbar_arrive_expect_tx(bars + B_KVF + kv, 2 * TILE);
                tc::tma_load_2d(kt, &p.mapK, xk, it.k_lo, bars + B_KVF + kv);
                tc::tma_load_2d(kt + TILE, &p.mapV, xk, it.k_lo, bars + B_KVF + kv);
                ++n;
                for (int t = 0; t < it.heads * tiles; ++t, ++g) {
                    const int s = g % NST, use = g / NST, x = (it.h0 + t / tiles) * DH;
                    const int row = it.q0 + it.i0 + (t % tiles) * BT;
                    if (use > 0 && !tc::mbar_wait(bars + B_QE + s, (use - 1) & 1, abort_flag)) { ok = false; break; }
                    uint8_t* qt = sm + OFF_Q + s * 2 * TILE;
                    tc::mbar_arrive_expect_tx(bars + B_QF + s, 2 * TILE);
                    tc::tma_load_2d(qt, &p.mapQ, x, row, bars + B_QF + s);
                    tc::tma_load_2d(qt + TILE, &p.mapDO, x, row, bars + B_QF + s);
                }
            }
            if (!ok) give_up();
        }
    } else if (warp == SOFT + 1) {
        // ---------------- MMA issuer.  In turn: the scores of half 0 of the next tile, the products of half 1 of the
        // tile before, the scores of half 1, the products of half 0: the order in which the two halves' softmax
        // reaches them, half a tile apart, so that scores are always there and neither waits for products.
        if (tc::elect_one()) {
            constexpr uint32_t ID_S = tc::instr_desc(1, BT, HALF, 0, 0);   // both K-major
            constexpr uint32_t ID_A = tc::instr_desc(1, BT, DH, 0, 1);     // A in tensor memory, B MN-major
            int g = 0, n = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int w = items.take(k);
                if (w < 0) {
                    ok = w == -1;
                    break;
                }
                it.load(p, w);
                if (it.tiles() == 0) continue;
                const int kv = n & 1, steps = it.heads * it.tiles();
                if (!tc::mbar_wait(bars + B_KVF + kv, (n >> 1) & 1, abort_flag, win::kItemWait)) { ok = false; break; }
                const uint64_t dK = kmajor_desc(sm + OFF_KV + kv * 2 * TILE), dV = kmajor_desc(sm + OFF_KV + kv * 2 * TILE + TILE);
                auto scores = [&](int X, int t) {
                    const int gt = g + t, s = gt % NST;
                    if (X == 0 && !tc::mbar_wait(bars + B_QF + s, (gt / NST) & 1, abort_flag)) return false;
                    if (gt > 0 && !tc::mbar_wait(bars + B_SR + X, (gt - 1) & 1, abort_flag)) return false;
                    tc::tc_fence_after();
                    const uint8_t* qt = sm + OFF_Q + s * 2 * TILE + X * (TILE / 2);
                    const uint64_t dQ = kmajor_desc(qt), dO = kmajor_desc(qt + TILE);
#pragma unroll
                    for (int kk = 0; kk < DH / 16; ++kk) tc::mma_f16_ss(tm + TM_X * X + TM_S, dK + 2 * kk, dQ + 2 * kk, ID_S, kk > 0);
#pragma unroll
                    for (int kk = 0; kk < DH / 16; ++kk) tc::mma_f16_ss(tm + TM_X * X + TM_DP, dV + 2 * kk, dO + 2 * kk, ID_S, kk > 0);
                    tc::mma_commit(bars + B_SF + X);
                    if (X == 1 && t == steps - 1) tc::mma_commit(bars + B_KVE + kv);
                    return true;
                };
                auto products = [&](int X, int t) {
                    const int gt = g + t, s = gt % NST;
                    if (!tc::mbar_wait(bars + B_PF + X, gt & 1, abort_flag)) return false;
                    tc::tc_fence_after();
                    const uint8_t* qt = sm + OFF_Q + s * 2 * TILE + X * (TILE / 2);
                    const uint64_t mQ = mnmajor_desc(qt), mO = mnmajor_desc(qt + TILE);
                    const uint32_t more = t > 0 || X > 0;
#pragma unroll
                    for (int kk = 0; kk < HALF / 16; ++kk)
                        tc::mma_f16_ts(tm + TM_DV, tm + TM_X * X + TM_P + 8 * kk, mO + (uint64_t)(kk * 128), ID_A, more | (kk > 0));
#pragma unroll
                    for (int kk = 0; kk < HALF / 16; ++kk)
                        tc::mma_f16_ts(tm + TM_DK, tm + TM_X * X + TM_DS + 8 * kk, mQ + (uint64_t)(kk * 128), ID_A, more | (kk > 0));
                    tc::mma_commit(bars + B_PV + X);
                    if (X == 1) tc::mma_commit(bars + B_QE + s);
                    return true;
                };
                ok = scores(0, 0) && scores(1, 0);
                // the item before has left the sums
                if (ok && n > 0) ok = tc::mbar_wait(bars + B_AE, (n - 1) & 1, abort_flag);
                for (int t = 0; t < steps && ok; ++t)
                    ok = (t + 1 == steps || scores(0, t + 1)) && (t == 0 || products(1, t - 1)) &&
                         (t + 1 == steps || scores(1, t + 1)) && products(0, t);
                ok = ok && products(1, steps - 1);
                if (ok) tc::mma_commit(bars + B_AF);
                g += steps;
                ++n;
            }
            if (!ok) give_up();
        }
    } else if (warp == SOFT + 2) {
        // ---------------- lse and delta of the tile's rows; rows of Q and dO that are not finite (delta says so), or
        // behind the sequence's last query, are zeroed
        int g = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int w = items.take_warp(k);
            if (w < 0) {
                ok = w == -1;
                break;
            }
            it.load(p, w);
            const int tiles = it.tiles();
            for (int t = 0; t < it.heads * tiles; ++t, ++g) {
                const int s = g % NST, use = g / NST;
                const int i0 = it.i0 + (t % tiles) * BT;
                const long long at = (long long)(it.h0 + t / tiles) * p.w.Tq + it.q0;
                float l[4], d[4];
                uint32_t bad[4], out[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + 32 * e + lane;
                    const bool in = i < it.nq;
                    l[e] = in ? p.w.Lse[at + i] : 0.f;
                    d[e] = in ? p.w.delta[at + i] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    bad[e] = __ballot_sync(0xffffffffu, !isfinite(d[e]));
                    out[e] = bad[e] | ~win::low_bits(it.nq - i0 - 32 * e);
                }
                if (use > 0 && !wait_all(bars + B_QE + s, (use - 1) & 1)) { ok = false; break; }
                float* st = reinterpret_cast<float*>(sm + OFF_STAT + s * 1024);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    st[32 * e + lane] = -l[e] * kLog2e;
                    st[BT + 32 * e + lane] = -d[e];
                }
                if (out[0] | out[1] | out[2] | out[3]) {
                    if (!wait_all(bars + B_QF + s, use & 1)) { ok = false; break; }
                    zero_rows(sm + OFF_Q + s * 2 * TILE, lane, out);
                    zero_rows(sm + OFF_Q + s * 2 * TILE + TILE, lane, out);
                    tc::fence_proxy_async_smem();
                }
                if (lane == 0) bad_rows[s] = make_uint4(bad[0], bad[1], bad[2], bad[3]);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + B_ST + s);
            }
        }
        if (!ok && lane == 0) give_up();
    } else if (warp < SOFT) {
        // ---------------- softmax groups: thread = key r of the block, queries 64 X + 32 y ... + 31 of each tile
        const int X = warp / (SOFT / 2), y = (warp >> 2) & 1, qd = warp & 3, r = 32 * qd + lane;
        const uint32_t lanes = (uint32_t)(32 * qd) << 16, tX = tm + lanes + TM_X * X;
        const float c = p.c;
        int g = 0, n = 0, nonfinite = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int w = items.take_warp(k);
            if (w < 0) {
                ok = w == -1;
                break;
            }
            it.load(p, w);
            const int tiles = it.tiles(), steps = it.heads * tiles, u = it.u0 + r;
            // queries (as indices) that see key u, cut to the item's
            const int lo_i = max(u - p.w.right - it.first, it.i0), hi_i = u < p.w.sinks ? it.i1 : min(u + p.w.left + 1 - it.first, it.i1);
            int lo = 0, hi = 0;   // of the part's first query
            for (int t = 0, ti = 0; t < steps; ++t, ++g) {
                const int s = g % NST, use = g / NST;
                if (ti == 0) {
                    lo = lo_i - it.i0 - HALF * X - COLS * y;
                    hi = hi_i - it.i0 - HALF * X - COLS * y;
                } else {
                    lo -= BT;
                    hi -= BT;
                }
                if (++ti == tiles) ti = 0;
                const bool whole = __all_sync(0xffffffffu, lo <= 0 && hi >= COLS);
                const uint32_t vis = win::low_bits(hi) & ~win::low_bits(lo);
                if (!wait_all(bars + B_ST + s, use & 1) || !wait_all(bars + B_SF + X, g & 1)) { ok = false; break; }
                tc::tc_fence_after();
                const uint32_t bad = reinterpret_cast<const uint32_t*>(bad_rows + s)[2 * X + y] & vis;
                uint32_t sc[COLS], dp[COLS];
                tc::tmem_ld_32x32b_x32(tX + TM_S + COLS * y, sc);
                tc::tmem_ld_32x32b_x32(tX + TM_DP + COLS * y, dp);
                tc::tmem_wait_ld();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + B_SR + X);
                const ulonglong2* nl = reinterpret_cast<const ulonglong2*>(sm + OFF_STAT + s * 1024) + HALF / 4 * X + COLS / 4 * y;
                auto neg = [&](int k4, uint64_t& l0, uint64_t& l1, uint64_t& d0, uint64_t& d1) {
                    const ulonglong2 l = nl[k4], d = nl[BT / 4 + k4];
                    l0 = l.x;
                    l1 = l.y;
                    d0 = d.x;
                    d1 = d.y;
                };
                if (whole) grad_scores<true, true>(sc, dp, c, vis, bad, neg);
                else grad_scores<false, true>(sc, dp, c, vis, bad, neg);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + B_QE + s);   // the statistics have been read
                if (g > 0) {
                    if (!wait_all(bars + B_PV + X, (g - 1) & 1)) { ok = false; break; }
                    tc::tc_fence_after();
                }
                tc::tmem_st_32x32b_x16(tX + TM_P + COLS / 2 * y, *reinterpret_cast<uint32_t(*)[16]>(sc));
                tc::tmem_st_32x32b_x16(tX + TM_DS + COLS / 2 * y, *reinterpret_cast<uint32_t(*)[16]>(dp));
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + B_PF + X);
            }
            if (!ok) break;
            // ---- epilogue: groups X = 0 take dV, X = 1 dK, 32 columns a thread
            if (steps > 0) {
                if (!wait_all(bars + B_AF, n & 1)) { ok = false; break; }
                tc::tc_fence_after();
                ++n;
            }
            uint32_t o[COLS];
            tc::tmem_ld_32x32b_x32(tm + lanes + (X ? TM_DK : TM_DV) + COLS * y, o);
            tc::tmem_wait_ld();
            if (steps > 0) {
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + B_AE);
            } else {
#pragma unroll
                for (int e = 0; e < COLS; ++e) o[e] = 0;
            }
            if (r < it.keys) {
                const float f = X ? p.w.grad_scale : 1.f;
                if (it.slot >= 0) {
                    float4* dst = reinterpret_cast<float4*>(p.w.partial + it.slot * SLOT + (X * BT + r) * DH + COLS * y);
#pragma unroll
                    for (int e = 0; e < COLS / 4; ++e)
                        dst[e] = make_float4(f * __uint_as_float(o[4 * e]), f * __uint_as_float(o[4 * e + 1]),
                                             f * __uint_as_float(o[4 * e + 2]), f * __uint_as_float(o[4 * e + 3]));
                } else {
                    const long long t = it.k_lo + r;
                    const int col = it.hk * DH + COLS * y;
                    nonfinite |= X ? store_row(p.w.dK + t * p.w.ld_dk + col, o, f) : store_row(p.w.dV + t * p.w.ld_dv + col, o, f);
                }
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
}

// dK and dV of the key blocks with sinks that were cut up: the window's sums, then the chunks' head by head.
// One block per sequence, key block and key head; a thread per four columns of a key.
__global__ void window_sink_sum_kernel(const WindowArgs p) {
    const SeqOffsets cq{p.cu_q, p.n_seq, p.Tq}, ck{p.cu_k, p.n_seq, p.Tk};
    const int G = p.Hq / p.Hk, hk = blockIdx.x % p.Hk, s = blockIdx.x / p.Hk, u0 = blockIdx.y * BT;
    const int q0 = cq.begin(s), nq = max(cq.begin(s + 1) - q0, 0), k0 = ck.begin(s), nk = max(ck.begin(s + 1) - k0, 0);
    if (u0 >= min(p.sinks, nk)) return;
    const int keys = min(BT, nk - u0);
    const QueryRange r = queries_of(u0, u0 + keys, nk - nq, nq, p.left, p.right);
    if (r.ib >= nq) return;
    const int unit = blockIdx.z * blockDim.x + threadIdx.x;   // (dV or dK, key, four columns)
    const int X = unit / (BT * DH / 4), key = unit / (DH / 4) % BT, col = unit % (DH / 4) * 4;
    if (key >= keys) return;
    const long long off = (X * BT + key) * DH + col;
    float4 sum = *reinterpret_cast<const float4*>(p.partial + (chunk_slots(p) + ((long long)s * p.Hk + hk) * SINK_BLOCKS + blockIdx.y) * SLOT + off);
    const long long b0 = q0 / CHUNK + s;
    if (u0 + key < p.sinks)
        for (int h = hk * G; h < hk * G + G; ++h)
            for (int b = r.ib / CHUNK; b * CHUNK < nq; ++b) {
                const long long slot = ((b0 + b) * SINK_BLOCKS + blockIdx.y) * p.Hq + h;
                const float4 v = *reinterpret_cast<const float4*>(p.partial + slot * SLOT + off);
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
    if (!(isfinite(sum.x) && isfinite(sum.y) && isfinite(sum.z) && isfinite(sum.w))) atomicOr(p.status, kStatusNonFinite);
    __nv_bfloat16* dst = X ? p.dK + (k0 + u0 + key) * p.ld_dk : p.dV + (k0 + u0 + key) * p.ld_dv;
    *reinterpret_cast<uint2*>(dst + hk * DH + col) = make_uint2(pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w));
}

}  // namespace

cudaError_t launch_window_dkv(const WindowArgs& a, int sms, cudaStream_t s) {
    KvArgs p{};
    p.w = a;
    const bool q = a.Tq > 0;   // without queries the tiles are never loaded; any valid array serves the maps
    if (!make_map(&p.mapK, a.K, a.Tk, a.Hk * DH, a.ld_k) || !make_map(&p.mapV, a.V, a.Tk, a.Hk * DH, a.ld_v) ||
        !make_map(&p.mapQ, q ? a.Q : a.K, q ? a.Tq : a.Tk, (q ? a.Hq : a.Hk) * DH, q ? a.ld_q : a.ld_k) ||
        !make_map(&p.mapDO, q ? a.dOut : a.K, q ? a.Tq : a.Tk, (q ? a.Hq : a.Hk) * DH, q ? a.ld_do : a.ld_k))
        return cudaErrorInvalidValue;
    p.c = a.scale * kLog2e;
    p.cut = cuts_sinks(a);
    p.n_window = win::block_numbers<BT>(a.Tk, a.n_seq) * a.Hk;
    p.blocks = (a.sinks + BT - 1) / BT;
    p.n_chunk = p.cut ? win::block_numbers<CHUNK>(a.Tq, a.n_seq) * a.Hq * p.blocks : 0;
    p.n_items = p.n_window + p.n_chunk;
    p.chunks_first = (long long)CHUNK > (a.Hq / a.Hk) * ((long long)a.left + a.right + BT);
    cudaError_t e = cudaFuncSetAttribute(window_dkv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    {
        LaunchScope scope("window_dkv", s);
        window_dkv_kernel<<<(unsigned)(p.n_items < sms ? p.n_items : sms), KV_THREADS, SMEM_BYTES, s>>>(p);
    }
    return cudaGetLastError();
}

// The sums of the key blocks that were cut up, if there are any.
cudaError_t launch_window_sink_sum(const WindowArgs& a, cudaStream_t s) {
    if (!cuts_sinks(a)) return cudaSuccess;
    LaunchScope scope("window_sink_sum", s);
    window_sink_sum_kernel<<<dim3((unsigned)(a.n_seq * a.Hk), (a.sinks + BT - 1) / BT, SLOT / 4 / 256), 256, 0, s>>>(a);
    return cudaGetLastError();
}

long long window_partial_floats(const WindowArgs& a) { return all_slots(a) * SLOT; }

}  // namespace ttt
