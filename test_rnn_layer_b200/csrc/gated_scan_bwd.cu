// Gated linear recurrence, backward: rows in the order of lambda's walk, against the forward walk
// (gated_scan.cuh says how).
//   l_t = dy_t + a_{t+1} l_{t+1},  df_t = l_t dh_t/df_t,  dx_t = l_t s(a_t)
#include "gated_scan.cuh"

namespace ttt {
namespace {

using namespace scan;

template <bool BF, int FORM, int LC>
__global__ void __launch_bounds__(kThreads, 2) gated_bwd_kernel(const __grid_constant__ GatedScanArgs p, const __grid_constant__ Maps m) {
    constexpr int R = kRowsB, V = Elem<BF>::V, TILE = kThreads / LC * R, ARRAY = TILE * LC * 4;
    constexpr int STAGE = 3 * ARRAY + TILE / kKeep * LC * V * 4;
    __shared__ Shared<LC, V> sh;
    extern __shared__ __align__(128) uint8_t stages[];
    const SeqOffsets c{p.cu, p.n_seq, p.T};
    const int cs = cluster_size(), rank = tc::cluster_ctarank(), chunks = (p.T + TILE - 1) / TILE, steps = (chunks + cs - 1) / cs;
    const int col = threadIdx.x % LC, group = threadIdx.x / LC, dir = p.reverse ? 1 : -1;
    const int strip = blockIdx.x / cs * LC * V, ch = strip + col * V;
    const bool on = ch < p.D;
    empty_sequences(c, p.D, p.dH_T, p.dH_0, p.status);

    // stage s: TILE rows of the strip of F, X and dY, then the kept states of the tile's segments
    auto issue = [&](int step) {
        const int chunk = step * cs + rank, s = step % kStages;
        if (step >= steps || chunk >= chunks) return;
        const int row = (p.reverse ? chunk : chunks - 1 - chunk) * TILE;
        uint8_t* to = stages + s * STAGE;
        tc::mbar_arrive_expect_tx(sh.full + s, STAGE);
        static_assert(TILE <= 256, "a box has at most 256 rows");
        tc::tma_load_2d(to, &m.f, strip, row, sh.full + s);
        tc::tma_load_2d(to + ARRAY, &m.x, strip, row, sh.full + s);
        tc::tma_load_2d(to + 2 * ARRAY, &m.dy, strip, row, sh.full + s);
        tc::tma_load_2d(to + 3 * ARRAY, &m.h, strip, row / kKeep, sh.full + s);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) tc::mbar_init(sh.full + s, 1);
        for (int s = 0; s < 2; ++s) tc::mbar_init(sh.sent + s, 1);
        tc::fence_mbar_init();
    }
    tc::cluster_sync();   // every CTA runs and has its barriers: its shared memory may be written
    if (threadIdx.x == 32)
        for (int s = 0; s < kStages - 1; ++s) issue(s);

    Vec<V> state = all<V>(0.f);
    bool bad = false, ok = true;
    int seq_b = 0, seq_e = 0;
    Cursor at_row;
    using T = typename Elem<BF>::type;
    for (int step = 0; step < steps; ++step) {
        // the group's first row in lambda's order; past the last chunk outside [0, T)
        const int chunk = step * cs + rank;
        const int t0 = p.reverse ? chunk * TILE + group * R : (chunks - chunk) * TILE - 1 - group * R;
        const bool plain = plain_rows<R>(c, t0, dir, seq_b, seq_e);
        if (chunk < chunks) ok = tc::mbar_wait(sh.full + step % kStages, (step / kStages) & 1, nullptr);
        const uint8_t* st = stages + step % kStages * STAGE;
        const int seg = p.reverse ? group : kThreads / LC - 1 - group;   // in the tile
        const Vec<V> kept = *reinterpret_cast<const Vec<V>*>(st + 3 * ARRAY + (seg * LC + col) * V * 4);
        // row k = 0 in lambda's order; the forward walk begins at k = R - 1
        const uint8_t* in = st + ((seg * R + (p.reverse ? 0 : R - 1)) * LC + col) * 4;
        const int pitch_in = dir * LC * 4;
        auto word = [&](int array, int k) { return *reinterpret_cast<const uint32_t*>(in + array * ARRAY + k * pitch_in); };
        Vec<V> a[R], sc[R], sl[R], dy[R], lam;
        Run<V> run{all<V>(1.f), all<V>(0.f)};
        if (plain) {
            Vec<V> h = kept;
#pragma unroll
            for (int k = R - 1; k >= 0; --k) {
                const Vec<V> x = Elem<BF>::get(word(1, k));
                Vec<V> rest;
                gates<V>(Elem<BF>::get(word(0, k)), a[k], rest);
                slopes<FORM, V>(a[k], rest, h, x, sc[k], sl[k]);
                h = fma(a[k], h, mul(sc[k], x));
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                dy[k] = Elem<BF>::get(word(2, k));
                run.b = mul(a[k], add(run.b, dy[k]));
                run.a = mul(run.a, a[k]);
            }
        } else {
#pragma unroll 1
            for (int k = 0; k < R; ++k) {
                const Row q = row_of(c, at_row, t0 + dir * k, p.reverse);
                if (q.s < 0) continue;
                Vec<V> ak, rest;
                gates<V>(Elem<BF>::get(word(0, k)), ak, rest);
                const Vec<V> g = Elem<BF>::get(word(2, k));
                if (q.end) {   // lambda starts anew, with the final state's gradient
                    run = Run<V>{all<V>(kReset), mul(ak, add(state_of<V>(p.dH_T, q.s, p.D, ch, on), g))};
                } else {
                    run.b = mul(ak, add(run.b, g));
                    run.a = mul(run.a, ak);   // -0 stays -0
                }
            }
        }
        if (!exchange<LC, V>(sh, step, cs, rank, run, state, lam, ok, [&]() { issue(step + kStages - 1); })) break;
        T* df = static_cast<T*>(p.dF) + (long long)t0 * p.ld_df + ch;
        T* dx = static_cast<T*>(p.dX) + (long long)t0 * p.ld_dx + ch;
        const long long pitch_f = dir * p.ld_df, pitch_x = dir * p.ld_dx;
        Vec<V> seen = all<V>(0.f);   // 0 times what is stored: NaN where it is not finite
        if (plain) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const Vec<V> l = add(lam, dy[k]), d = mul(l, sl[k]);
                seen = fma(all<V>(0.f), d, seen);
                lam = mul(a[k], l);
                if (on) {
                    __stcs(reinterpret_cast<uint32_t*>(df), Elem<BF>::put(d));
                    __stcs(reinterpret_cast<uint32_t*>(dx), Elem<BF>::put(mul(l, sc[k])));
                }
                df += pitch_f;
                dx += pitch_x;
            }
            seen = fma(all<V>(0.f), lam, seen);   // inside a sequence what is not finite stays so
        } else {
            Vec<V> before[R];   // h before each row (a short array in local memory)
            Vec<V> h = kept;
#pragma unroll 1
            for (int k = R - 1; k >= 0; --k) {
                const Row q = row_of(c, at_row, t0 + dir * k, p.reverse);
                if (q.s < 0) continue;
                if (q.start) h = state_of<V>(p.H_0, q.s, p.D, ch, on);
                before[k] = h;
                Vec<V> ak, rest;
                gates<V>(Elem<BF>::get(word(0, k)), ak, rest);
                h = fma(ak, h, input<FORM, V>(ak, rest, Elem<BF>::get(word(1, k))));
            }
#pragma unroll 1
            for (int k = 0; k < R; ++k) {
                const Row q = row_of(c, at_row, t0 + dir * k, p.reverse);
                if (q.s < 0) continue;
                Vec<V> ak, rest, s, slope;
                gates<V>(Elem<BF>::get(word(0, k)), ak, rest);
                slopes<FORM, V>(ak, rest, before[k], Elem<BF>::get(word(1, k)), s, slope);
                if (q.end) lam = state_of<V>(p.dH_T, q.s, p.D, ch, on);
                const Vec<V> l = add(lam, Elem<BF>::get(word(2, k))), d = mul(l, slope);
                lam = mul(ak, l);
                seen = fma(all<V>(0.f), d, seen);
                seen = fma(all<V>(0.f), lam, seen);
                if (on) {
                    *reinterpret_cast<uint32_t*>(df + k * pitch_f) = Elem<BF>::put(d);
                    *reinterpret_cast<uint32_t*>(dx + k * pitch_x) = Elem<BF>::put(mul(l, s));
                }
                if (q.start) put_state<V>(p.dH_0, q.s, p.D, ch, on, lam);
            }
        }
        bad |= on && wild<V>(seen);
    }
    if (bad) atomicOr(p.status, kStatusNonFinite);
    if (!ok) {
        atomicOr(p.status, kStatusTimeout);
        settle();
    }
    tc::cluster_sync();   // nobody leaves while another may still write to its shared memory
}

template <bool BF, int FORM>
cudaError_t backward(const GatedScanArgs& a, cudaStream_t s) {
    const Shape q = shape_of(a, kRowsB);
    if (q.lanes == 32) return launch<BF, 32, kRowsB>(gated_bwd_kernel<BF, FORM, 32>, a, true, q.cs, s);
    if (q.lanes == 16) return launch<BF, 16, kRowsB>(gated_bwd_kernel<BF, FORM, 16>, a, true, q.cs, s);
    return launch<BF, 8, kRowsB>(gated_bwd_kernel<BF, FORM, 8>, a, true, q.cs, s);
}

}  // namespace

cudaError_t launch_gated_scan_backward(const GatedScanArgs& a, cudaStream_t s) {
    const cudaError_t e = cudaMemsetAsync(a.status, 0, 16, s);
    if (e != cudaSuccess) return e;
    LaunchScope scope("gated_scan_backward", s);
    if (a.bf16) return a.form == 0 ? backward<true, 0>(a, s) : a.form == 1 ? backward<true, 1>(a, s) : backward<true, 2>(a, s);
    return a.form == 0 ? backward<false, 0>(a, s) : a.form == 1 ? backward<false, 1>(a, s) : backward<false, 2>(a, s);
}

}  // namespace ttt
