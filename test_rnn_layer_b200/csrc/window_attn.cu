// Window attention with sinks, forward, on the tcgen05 tensor cores (head dim 64, bf16, fp32 accumulation):
//   Out[i, h] = Xres[i, h] + sum_u softmax_u(scale q_i . k_u) v_u over the keys u that row i sees:
//   u <= p + right and (u >= p - left or u < sinks), p = nk - nq + i.
//
// Work: an item is 256 query rows of a sequence (tiles A and B of 128) of one head; a persistent grid walks the
// items, heads fastest, so that the CTAs running at a time share the keys and values of few windows in L2.  An
// item's key tiles are those of its sinks (one of 32 keys where they are that few) and those of the window of
// its rows; a tile that only one of A and B sees is skipped by the other.  Per key tile, as in the
// segment-local kernel: S_X = Q_X K^T (tensor memory), P_X = exp2(c S_X - m_X) with a lazily raised maximum,
// O_X += P_X V.  Masks are four 32-bit words per row, applied only where the tile is not seen whole.
//
// A weight of zero times a non-finite value is NaN, and a tile's rows behind the sequence's end may hold
// anything: warp 11 looks through each value tile in shared memory (one product by zero per pair of elements,
// well below a tenth of the tile's softmax), zeroes the rows that are not finite and leaves their bits for the
// softmax, which spoils exactly the query rows that see them.
//
// Roles (384 threads): warps 0-3 the softmax of tile A, 4-7 that of tile B (a thread per query row), warp 8 the
// TMA producer, warps 9 and 10 the MMA issuers of A and B, warp 11 the value screen.
// Tensor memory (512 columns): S_A 0, S_B 128; O_A 256, O_B 320; P_A 384, P_B 448.
// Every wait is bounded; on a timeout the CTA sets the status word, lets its copies and products in flight
// land and returns.
#include <type_traits>

#include "attn_prims.cuh"
#include "internal.h"
#include "window_items.cuh"

namespace ttt {
namespace {

using namespace attn;

constexpr int DH = 64, BQ = 128, BKV = 128, ROWS = 2 * BQ, NARROW = 32, NST = 4, THREADS = 384;
constexpr int TILE = BQ * DH * 2;                 // 16 KB: a 128 x 64 bf16 tile
constexpr int OFF_Q = 0;                          // Q_A, Q_B
constexpr int OFF_KV = 2 * TILE;                  // stage s: K at OFF_KV + 2 s TILE, V after it
constexpr int OFF_BAR = OFF_KV + NST * 2 * TILE;
constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
constexpr uint32_t TM_S = 0, TM_O = 256, TM_P = 384;   // + 128 X (S), + 64 X (O, P) for tile X
constexpr float kLazy = 8.0f;                     // log2 of the largest unscaled exponential
constexpr int EMU = 1;                            // pairs of every 8 whose 2^x runs on the FMA pipe

// Barrier slots (8 bytes each) from OFF_BAR.
enum : int {
    B_QF = 0,              // Q_A, Q_B landed (TMA bytes)
    B_QE = 1,              // the item's last S products of both tiles are done (2 arrivals)
    B_KF = 2,              // [NST] K tile landed
    B_VF = 2 + NST,        // [NST] V tile landed
    B_VS = 2 + 2 * NST,    // [NST] V tile screened
    B_KVE = 2 + 3 * NST,   // [NST] both tiles are done with the stage (2 arrivals)
    B_SF = 2 + 4 * NST,    // [2] S_X is in tensor memory (MMA commit)
    B_SR = B_SF + 2,       // [2] the softmax group has read S_X (4 warp arrivals)
    B_PF = B_SR + 2,       // [2] P_X written, O_X rescaled (4 warp arrivals)
    B_PV = B_PF + 2,       // [2] O_X += P_X V done (MMA commit)
    B_SLOT = B_PV + 2,     // tensor memory address (u32) and the abort flag (int)
    B_BAD = 32,            // [NST] 16 bytes: bits of the stage's V rows that are not finite
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
    float c;                        // scale * log2(e)
};

struct Item {
    int q_lo, rows, pos0, k0, nk, h, hk;
    int ns, nt;                     // sink tiles, all tiles
    bool narrow;                    // the one sink tile has NARROW keys
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
        narrow = r.sk > 0 && r.sk <= NARROW;
        ns = (r.sk + BKV - 1) / BKV;
        nt = ns + (r.hi - r.lo + BKV - 1) / BKV;
        return true;
    }
    __device__ __forceinline__ int start(int j) const { return j < ns ? BKV * j : r.lo + BKV * (j - ns); }
    // tile X's window tiles [a, b), counted from the item's first tile (sinks that reach into the window begin it)
    __device__ __forceinline__ void range(const WindowArgs& p, int X, int& a, int& b) const {
        const int n = min(rows - BQ * X, BQ), q = pos0 + BQ * X;
        const int lo = p.sinks > r.lo ? r.lo : max(q - p.left, r.lo), hi = min(q + n + p.right, r.hi);
        if (n <= 0 || hi <= lo) {
            a = b = ns;
            return;
        }
        a = ns + (lo - r.lo) / BKV;
        b = ns + (hi - r.lo + BKV - 1) / BKV;
    }
    // sinks lie in front of the item's window, so every row of the item sees them
    __device__ __forceinline__ bool sees(int X, int j, int a, int b) const { return j < ns ? rows > BQ * X : j >= a && j < b; }
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
    // nothing seen so far: any finite reference serves, as every weight is zero (or 2^-125 on the FMA pipe,
    // which the factor 0 of the first raise removes)
    const float ref = st.m == -INFINITY ? 0.f : st.m;
    const uint64_t c2 = f2(c, c), nm2 = f2(-ref, -ref);
    uint64_t ls[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k2 = 0; k2 < NC / 2; ++k2) {
        const uint64_t x = f2_fma(f2(__uint_as_float(s[2 * k2]), __uint_as_float(s[2 * k2 + 1])), c2, nm2);
        float p0, p1;
        if ((k2 & 7) >= 8 - EMU) {
            ex2_poly2(x, p0, p1);
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
        items.init(2 + 1 + 8);   // MMA issuers, side warps, softmax warps
        tc::mbar_init(bars + B_QF, 1);
        tc::mbar_init(bars + B_QE, 2);
        for (int s = 0; s < NST; ++s) {
            tc::mbar_init(bars + B_KF + s, 1);
            tc::mbar_init(bars + B_VF + s, 1);
            tc::mbar_init(bars + B_VS + s, 1);
            tc::mbar_init(bars + B_KVE + s, 2);
        }
        for (int x = 0; x < 2; ++x) {
            tc::mbar_init(bars + B_SF + x, 1);
            tc::mbar_init(bars + B_SR + x, 4);
            tc::mbar_init(bars + B_PF + x, 4);
            tc::mbar_init(bars + B_PV + x, 1);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
        tc::tma_prefetch_desc(&p.mapQ);
        tc::tma_prefetch_desc(&p.mapK);
        tc::tma_prefetch_desc(&p.mapV);
    }
    if (warp == 9) {
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

    if (warp == 8) {
        // ---------------- TMA producer: the item's Q tiles, then its K and V tiles through the ring
        if (tc::elect_one()) {
            int gkv = 0, n = 0;
            bool ok = true;
            for (int w = blockIdx.x, next, k = 0; ok && !*abort_flag; w = next) {
                if (w >= p.n_items) {
                    ok = items.put(k, -1);
                    break;
                }
                next = gridDim.x + atomicAdd(p.w.status + kTicket, 1);
                if (!it.load(p.w, w)) continue;
                if (!items.put(k++, w)) { ok = false; break; }
                if (n > 0 && !tc::mbar_wait(bars + B_QE, (n - 1) & 1, abort_flag)) { ok = false; break; }
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
    } else if (warp == 11) {
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
    } else if (warp >= 9) {
        // ---------------- MMA issuers, one per tile.  Step n = the tile's n-th key tile; the issuer of X issues
        // S_X of step n (once its group has read S_X of the step before), then P_X V of step n - 1.
        const int X = warp - 9;
        if (tc::elect_one()) {
            constexpr uint32_t ID_S = tc::instr_desc(1, BQ, BKV, 0, 0);      // bf16, both K-major
            constexpr uint32_t ID_SN = tc::instr_desc(1, BQ, NARROW, 0, 0);
            constexpr uint32_t ID_PV = tc::instr_desc(1, BQ, DH, 0, 1);      // bf16, A in tensor memory, V MN-major
            const uint64_t dQ = kmajor_desc(sm + OFF_Q + X * TILE);
            int gkv = 0, gs = 0, n = 0;
            bool ok = true;
            // P_X V of step gs - 1, whose values lie in stage s
            auto pv = [&](int s, bool accumulate, bool narrow) {
                if (!tc::mbar_wait(bars + B_PF + X, (gs - 1) & 1, abort_flag)) return false;
                tc::tc_fence_after();
                const uint64_t dV = mnmajor_desc(sm + OFF_KV + s * 2 * TILE + TILE);
                const int steps = narrow ? NARROW / 16 : BKV / 16;
                for (int kk = 0; kk < steps; ++kk)
                    tc::mma_f16_ts(tm + TM_O + 64 * X, tm + TM_P + 64 * X + 8 * kk, dV + (uint64_t)(kk * 128), ID_PV,
                                   (accumulate || kk > 0) ? 1u : 0u);
                tc::mma_commit(bars + B_PV + X);
                tc::mma_commit(bars + B_KVE + s);
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
                const int steps = (it.rows > BQ * X ? it.ns : 0) + b - a;
                if (!tc::mbar_wait(bars + B_QF, n & 1, abort_flag)) { ok = false; break; }
                ++n;
                tc::tc_fence_after();
                if (steps == 0) tc::mbar_arrive(bars + B_QE);
                int done = 0, prev = -1;
                bool prev_narrow = false;
                for (int j = 0; j < it.nt && ok; ++j, ++gkv) {
                    const int s = gkv % NST, use = gkv / NST;
                    if (!tc::mbar_wait(bars + B_KF + s, use & 1, abort_flag)) { ok = false; break; }
                    if (!it.sees(X, j, a, b)) {
                        tc::mbar_arrive(bars + B_KVE + s);
                        continue;
                    }
                    if (gs > 0 && !tc::mbar_wait(bars + B_SR + X, (gs - 1) & 1, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
                    const bool narrow = it.narrow && j == 0;
                    const uint64_t dK = kmajor_desc(sm + OFF_KV + s * 2 * TILE);
                    const uint32_t id = narrow ? ID_SN : ID_S;
#pragma unroll
                    for (int kk = 0; kk < DH / 16; ++kk)
                        tc::mma_f16_ss(tm + TM_S + 128 * X, dQ + 2 * kk, dK + 2 * kk, id, kk > 0);
                    tc::mma_commit(bars + B_SF + X);
                    if (done == steps - 1) tc::mma_commit(bars + B_QE);
                    if (prev >= 0 && !pv(prev, done > 1, prev_narrow)) { ok = false; break; }
                    ++gs;
                    ++done;
                    prev = s;
                    prev_narrow = narrow;
                }
                if (ok && prev >= 0 && !pv(prev, done > 1, prev_narrow)) ok = false;
            }
            if (!ok) give_up();
        }
    } else {
        // ---------------- softmax groups: warps 0-3 tile A, 4-7 tile B; thread = query row r of its tile
        const int X = warp >> 2, qd = warp & 3, r = 32 * qd + lane;
        const uint32_t lanes = (uint32_t)(32 * qd) << 16;
        const uint32_t tS = tm + lanes + TM_S + 128 * X, tO = tm + lanes + TM_O + 64 * X, tP = tm + lanes + TM_P + 64 * X;
        const float c = p.c;
        int gs = 0, gkv = 0, nonfinite = 0;
        bool ok = true;
        // every branch below is uniform over the warp (the item, the key tile, the waits' outcome)
        auto wait_all = [&](uint64_t* bar, uint32_t parity) {
            const bool got = tc::mbar_wait(bar, parity, abort_flag);
            return __all_sync(0xffffffffu, got);
        };
        for (int k = 0; ok; ++k) {
            const int w = items.take_warp(k);
            if (w < 0) {
                ok = w == -1;
                break;
            }
            it.load(p.w, w);
            int a, b;
            it.range(p.w, X, a, b);
            const int pos = it.pos0 + BQ * X + r;
            RowState st{-INFINITY, 0.f, true};
            // one key tile of NC keys: softmax, the screen's verdict, O's rescaling, P to tensor memory
            auto step = [&](auto width, int j) {
                constexpr int NC = decltype(width)::value;
                // the keys of this tile that the row sees, as bits
                const int t0 = it.start(j);
                int lo = 0, hi = it.r.sk - t0, sk = 0;
                if (j >= it.ns) {
                    lo = pos - p.w.left - t0;
                    hi = min(pos + p.w.right + 1, it.nk) - t0;
                    sk = p.w.sinks - t0;
                }
                const bool whole = __all_sync(0xffffffffu, hi >= NC && lo <= 0);
                if (!wait_all(bars + B_SF + X, gs & 1)) return false;
                tc::tc_fence_after();
                uint32_t s[NC];
#pragma unroll
                for (int k = 0; k < NC; k += 32) tc::tmem_ld_32x32b_x32(tS + k, *reinterpret_cast<uint32_t(*)[32]>(s + k));
                tc::tmem_wait_ld();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + B_SR + X);   // S_X may be overwritten
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < NC / 32; ++i) {
                        const uint32_t vis = visible(lo, hi, sk, i);
#pragma unroll
                        for (int k = 0; k < 32; ++k) s[32 * i + k] = (vis >> k) & 1u ? s[32 * i + k] : 0xff800000u;   // -inf
                    }
                }
                const float f = softmax_tile<NC>(s, c, st);
                // the screened values: a row that sees one that is not finite becomes NaN
                const int stage = gkv % NST;
                if (!wait_all(bars + B_VS + stage, (gkv / NST) & 1)) return false;
                const uint4 bad = bad_rows[stage];
                if (bad.x | bad.y | bad.z | bad.w) {
                    if ((bad.x & visible(lo, hi, sk, 0)) | (bad.y & visible(lo, hi, sk, 1)) | (bad.z & visible(lo, hi, sk, 2)) |
                        (bad.w & visible(lo, hi, sk, 3)))
                        st.l = NAN;
                }
                // the previous step's P V is done: P_X may be rewritten and O_X is stable
                if (gs > 0) {
                    if (!wait_all(bars + B_PV + X, (gs - 1) & 1)) return false;
                    tc::tc_fence_after();
                }
                if (__any_sync(0xffffffffu, f != 1.f && !st.first)) {
                    uint32_t o[32];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        tc::tmem_ld_32x32b_x32(tO + 32 * half, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc::tmem_st_32x32b_x32(tO + 32 * half, o);
                    }
                }
                st.first = false;
                if constexpr (NC == NARROW) {
                    tc::tmem_st_32x32b_x16(tP, *reinterpret_cast<uint32_t(*)[16]>(s));
                } else {
                    tc::tmem_st_32x32b_x32(tP + 0, *reinterpret_cast<uint32_t(*)[32]>(s + 0));
                    tc::tmem_st_32x32b_x32(tP + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(bars + B_PF + X);
                ++gs;
                return true;
            };
            for (int j = 0; j < it.nt && ok; ++j, ++gkv) {
                if (!it.sees(X, j, a, b)) continue;
                ok = it.narrow && j == 0 ? step(std::integral_constant<int, NARROW>{}, j)
                                               : step(std::integral_constant<int, BKV>{}, j);
            }
            if (!ok) break;
            // ---- epilogue: O_X / l (+ residual) as bf16, the row's log-sum-exp
            if (!st.first) {
                if (!wait_all(bars + B_PV + X, (gs - 1) & 1)) { ok = false; break; }
                tc::tc_fence_after();
            }
            uint32_t o[64];   // without a key tile what was there before: not used
            tc::tmem_ld_32x32b_x32(tO + 0, *reinterpret_cast<uint32_t(*)[32]>(o + 0));
            tc::tmem_ld_32x32b_x32(tO + 32, *reinterpret_cast<uint32_t(*)[32]>(o + 32));
            tc::tmem_wait_ld();
            if (BQ * X + r < it.rows) {
                const bool empty = st.first || (st.m == -INFINITY && st.l == st.l);
                const float inv = 1.0f / st.l;
                const long long t = it.q_lo + BQ * X + r, col = (long long)it.h * DH;
                const uint4* xr = p.w.Xres ? reinterpret_cast<const uint4*>(p.w.Xres + t * p.w.ld_out + col) : nullptr;
                uint4* dst = reinterpret_cast<uint4*>(p.w.Out + t * p.w.ld_out + col);
#pragma unroll
                for (int c8 = 0; c8 < DH / 8; ++c8) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = empty ? 0.f : __uint_as_float(o[8 * c8 + e]) * inv;
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
                if (p.w.Lse)
                    p.w.Lse[(long long)it.h * p.w.Tq + t] =
                        empty ? -INFINITY : (st.m == -INFINITY ? 0.f : st.m) * 0.69314718055994531f + logf(st.l);
            }
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
    if (warp == 9) {
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
    cudaError_t e = cudaFuncSetAttribute(window_fwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    LaunchScope scope("window_attn", s);
    window_fwd_kernel<<<(unsigned)(p.n_items < sms ? p.n_items : sms), THREADS, SMEM_BYTES, s>>>(p);
    return cudaGetLastError();
}

}  // namespace ttt
