// Gated linear recurrence, backward: rows in the order of lambda's walk, against the forward walk
// (gated_scan.cuh says how).
//   l_t = dy_t + a_{t+1} l_{t+1},  df_t = l_t dh_t/df_t,  dx_t = l_t s(a_t)
#include "gated_scan.cuh"

namespace ttt {
namespace {

using namespace scan;

template <bool BF, int FORM, int LC>
__global__ void __launch_bounds__(32 * (kWarpsB + 1), kPerSmB)
    gated_bwd_kernel(const __grid_constant__ GatedScanArgs p, const __grid_constant__ Maps m) {
    constexpr int R = kRows, W = kWarpsB, V = Elem<BF>::V, GROUPS = 32 / LC * W, TILE = GROUPS * R, ARRAY = TILE * LC * 4;
    constexpr int STAGE = (3 * ARRAY + GROUPS * LC * V * 4 + 127) / 128 * 128;
    __shared__ Shared<LC, V, W> sh;
    extern __shared__ __align__(128) uint8_t stages[];
    const SeqOffsets c{p.cu, p.n_seq, p.T};
    const int cs = cluster_size(), rank = tc::cluster_ctarank(), chunks = (p.T + TILE - 1) / TILE, steps = (chunks + cs - 1) / cs;
    const int strip = blockIdx.x / cs * LC * V, cols = min(LC, (p.D - strip) / V);
    empty_sequences(c, p.D, p.dH_T, p.dH_0, p.status);
    init_barriers(sh);
    bool ok = true;
    if (threadIdx.x >= 32 * W) {
        // stage s: TILE rows of the strip of F, X and dY, then the kept states of the tile's segments
        ok = exchange<LC, V, W>(sh, steps, cs, rank, cols, [&](int step) {
            const int chunk = step * cs + rank, s = step % kStages;
            if (step >= steps || chunk >= chunks) return;
            const int row = (p.reverse ? chunk : chunks - 1 - chunk) * TILE;
            uint8_t* to = stages + s * STAGE;
            tc::mbar_arrive_expect_tx(sh.full + s, 3 * ARRAY + GROUPS * LC * V * 4);
            for (int i = 0; i < TILE; i += box_rows(TILE)) {
                tc::tma_load_2d(to + i * LC * 4, &m.f, strip, row + i, sh.full + s);
                tc::tma_load_2d(to + ARRAY + i * LC * 4, &m.x, strip, row + i, sh.full + s);
                tc::tma_load_2d(to + 2 * ARRAY + i * LC * 4, &m.dy, strip, row + i, sh.full + s);
            }
            tc::tma_load_2d(to + 3 * ARRAY, &m.h, strip, row / kKeep, sh.full + s);
        });
    } else {
        const int col = min((int)threadIdx.x % LC, cols - 1), group = threadIdx.x / LC, dir = p.reverse ? 1 : -1, ch = strip + col * V;
        using T = typename Elem<BF>::type;
        bool bad = false;
        int seq_b = 0, seq_e = 0;
        const int seg = p.reverse ? group : GROUPS - 1 - group;   // in the tile
        const int pitch_in = dir * LC * 4;
        const long long pitch_f = dir * p.ld_df, pitch_x = dir * p.ld_dx;
        // the group's first row in lambda's order; past the last chunk outside [0, T)
        auto first_row = [&](int step) {
            const int chunk = step * cs + rank;
            return p.reverse ? chunk * TILE + group * R : (chunks - chunk) * TILE - 1 - group * R;
        };
        // row k = 0 in lambda's order; the forward walk begins at k = R - 1
        auto input_of = [&](int step) { return stages + step % kStages * STAGE + ((seg * R + (p.reverse ? 0 : R - 1)) * LC + col) * 4; };
        auto kept_of = [&](int step) {
            return *reinterpret_cast<const Vec<V>*>(stages + step % kStages * STAGE + 3 * ARRAY + (seg * LC + col) * V * 4);
        };
        struct Set {
            Vec<V> a[R], sc[R], sl[R];
            uint32_t dy[R];
            Run<V> before;
            bool plain;
            uint32_t marks;   // where not plain
        };
        auto first_half = [&](Set& q, int step) {
            const int t0 = first_row(step);
            q.plain = plain_rows<R>(c, t0, dir, seq_b, seq_e);
            if (step * cs + rank < chunks) ok = ok && tc::mbar_wait(sh.full + step % kStages, (step / kStages) & 1, &sh.abort);
            const uint8_t* in = input_of(step);
            auto word = [&](int array, int k) { return *reinterpret_cast<const uint32_t*>(in + array * ARRAY + k * pitch_in); };
            Run<V> run{all<V>(1.f), all<V>(0.f)};
            if (q.plain) {
                Vec<V> h = kept_of(step);
#pragma unroll
                for (int k = R - 1; k >= 0; --k) {
                    const Vec<V> x = Elem<BF>::get(word(1, k));
                    Vec<V> rest;
                    gates<V>(Elem<BF>::get(word(0, k)), q.a[k], rest);
                    slopes<FORM, V>(q.a[k], rest, h, x, q.sc[k], q.sl[k]);
                    h = fma(q.a[k], h, mul(q.sc[k], x));
                }
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    q.dy[k] = word(2, k);
                    run.b = mul(q.a[k], add(run.b, Elem<BF>::get(q.dy[k])));
                    run.a = mul(run.a, q.a[k]);
                }
            } else {
                q.marks = marks_of(c, t0, dir, p.reverse);
                in = apart(in);
                Vec<V> anew[R];   // the states that sequences begin with, then the gradients of their final ones
                states_at<V>(anew, q.marks >> 8 & 0xffu, c, t0, dir, p.H_0, p.D, ch);
                Vec<V> h = kept_of(step);
#pragma unroll
                for (int k = R - 1; k >= 0; --k) {
                    const Vec<V> x = Elem<BF>::get(word(1, k));
                    Vec<V> rest;
                    gates<V>(Elem<BF>::get(word(0, k)), q.a[k], rest);
                    if (first_of(q.marks, k)) h = anew[k];
                    slopes<FORM, V>(q.a[k], rest, h, x, q.sc[k], q.sl[k]);
                    h = fma(q.a[k], h, mul(q.sc[k], x));
                }
                states_at<V>(anew, q.marks >> 16 & 0xffu, c, t0, dir, p.dH_T, p.D, ch);
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    q.dy[k] = word(2, k);
                    const Vec<V> g = Elem<BF>::get(q.dy[k]);
                    if (last_of(q.marks, k)) {   // lambda starts anew
                        run = Run<V>{all<V>(kReset), mul(q.a[k], add(anew[k], g))};
                    } else if (in_sequence(q.marks, k)) {
                        run.b = mul(q.a[k], add(run.b, g));
                        run.a = mul(run.a, q.a[k]);   // -0 stays -0
                    } else {   // a row of no sequence leaves lambda as it is
                        q.a[k] = all<V>(1.f);
                        q.dy[k] = 0;
                    }
                }
            }
            q.before = hand_over<LC, V, W>(sh, step, col, run);
        };
        auto second_half = [&](Set& q, int step) {
            const int t0 = first_row(step);
            Vec<V> lam;
            if (!ok || !take_over<LC, V, W>(sh, step, col, q.before, lam)) {
                ok = false;
                return;
            }
            T* df = static_cast<T*>(p.dF) + (long long)t0 * p.ld_df + ch;
            T* dx = static_cast<T*>(p.dX) + (long long)t0 * p.ld_dx + ch;
            Vec<V> seen = all<V>(0.f);   // 0 times what is stored: NaN where it is not finite
            if (q.plain) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const Vec<V> l = add(lam, Elem<BF>::get(q.dy[k])), d = mul(l, q.sl[k]);
                    seen = fma(all<V>(0.f), d, seen);
                    lam = mul(q.a[k], l);
                    __stcs(reinterpret_cast<uint32_t*>(df), Elem<BF>::put(d));
                    __stcs(reinterpret_cast<uint32_t*>(dx), Elem<BF>::put(mul(l, q.sc[k])));
                    df += pitch_f;
                    dx += pitch_x;
                }
                seen = fma(all<V>(0.f), lam, seen);   // inside a sequence what is not finite stays so
            } else {
                df = apart(df);
                dx = apart(dx);
                Vec<V> anew[R], at[R];
                states_at<V>(anew, q.marks >> 16 & 0xffu, c, t0, dir, p.dH_T, p.D, ch);
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    if (last_of(q.marks, k)) lam = anew[k];
                    const Vec<V> l = add(lam, Elem<BF>::get(q.dy[k])), d = mul(l, q.sl[k]);
                    lam = mul(q.a[k], l);
                    at[k] = lam;
                    if (in_sequence(q.marks, k)) {
                        seen = fma(all<V>(0.f), d, seen);
                        seen = fma(all<V>(0.f), lam, seen);
                        __stcs(reinterpret_cast<uint32_t*>(df), Elem<BF>::put(d));
                        __stcs(reinterpret_cast<uint32_t*>(dx), Elem<BF>::put(mul(l, q.sc[k])));
                    }
                    df += pitch_f;
                    dx += pitch_x;
                }
                if (p.dH_0)
                    for (uint32_t bits = q.marks >> 8 & 0xffu; bits; bits &= bits - 1) {
                        const int k = __ffs(bits) - 1;
                        put_state<V>(p.dH_0, c.find(t0 + dir * k), p.D, ch, at[k]);
                    }
            }
            bad |= wild<V>(seen);
        };
        Set q0, q1;
        if (steps > 0) first_half(q0, 0);
        for (int step = 0; step < steps && __all_sync(0xffffffffu, ok); step += 2) {
            if (step + 1 < steps) first_half(q1, step + 1);
            second_half(q0, step);
            if (step + 1 >= steps) break;
            if (step + 2 < steps) first_half(q0, step + 2);
            second_half(q1, step + 1);
        }
        if (bad) atomicOr(p.status, kStatusNonFinite);
    }
    if (!ok) {
        sh.abort = 1;
        atomicOr(p.status, kStatusTimeout);
        settle();
    }
    tc::cluster_sync();   // nobody leaves while another may still write to its shared memory
}

template <bool BF, int FORM>
cudaError_t backward(const GatedScanArgs& a, cudaStream_t s) {
    const Shape q = shape_of(a, true);
    if (q.lanes == 32) return launch<BF, 32>(gated_bwd_kernel<BF, FORM, 32>, a, true, q.cs, s);
    if (q.lanes == 16) return launch<BF, 16>(gated_bwd_kernel<BF, FORM, 16>, a, true, q.cs, s);
    return launch<BF, 8>(gated_bwd_kernel<BF, FORM, 8>, a, true, q.cs, s);
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
