// Gated linear recurrence: the forward walk and the single token (gated_scan.cuh says how).
#include "gated_scan.cuh"

namespace ttt {
namespace {

using namespace scan;

template <bool BF, int FORM, int LC>
__global__ void __launch_bounds__(32 * (kWarpsF + 1), kPerSmF)
    gated_fwd_kernel(const __grid_constant__ GatedScanArgs p, const __grid_constant__ Maps m) {
    constexpr int R = kRows, W = kWarpsF, V = Elem<BF>::V, TILE = 32 / LC * W * R, ARRAY = TILE * LC * 4, STAGE = 2 * ARRAY;
    __shared__ Shared<LC, V, W> sh;
    extern __shared__ __align__(128) uint8_t stages[];
    const SeqOffsets c{p.cu, p.n_seq, p.T};
    const int cs = cluster_size(), rank = tc::cluster_ctarank(), chunks = (p.T + TILE - 1) / TILE, steps = (chunks + cs - 1) / cs;
    const int strip = blockIdx.x / cs * LC * V, cols = min(LC, (p.D - strip) / V);
    empty_sequences(c, p.D, p.H_0, p.H_T, p.status);
    init_barriers(sh);
    bool ok = true;
    if (threadIdx.x >= 32 * W) {
        // stage s: TILE rows of the strip of F, then of X
        ok = exchange<LC, V, W>(sh, steps, cs, rank, cols, [&](int step) {
            const int chunk = step * cs + rank, s = step % kStages;
            if (step >= steps || chunk >= chunks) return;
            const int row = (p.reverse ? chunks - 1 - chunk : chunk) * TILE;
            uint8_t* to = stages + s * STAGE;
            tc::mbar_arrive_expect_tx(sh.full + s, STAGE);
            for (int i = 0; i < TILE; i += box_rows(TILE)) {
                tc::tma_load_2d(to + i * LC * 4, &m.f, strip, row + i, sh.full + s);
                tc::tma_load_2d(to + ARRAY + i * LC * 4, &m.x, strip, row + i, sh.full + s);
            }
        });
    } else {
        const int col = min((int)threadIdx.x % LC, cols - 1), group = threadIdx.x / LC, dir = p.reverse ? -1 : 1, ch = strip + col * V;
        using T = typename Elem<BF>::type;
        bool bad = false;
        int seq_b = 0, seq_e = 0;
        const int pitch_in = dir * LC * 4;
        const long long pitch = dir * p.ld_y;
        // the group's first row in walking order; past the last chunk outside [0, T)
        auto first_row = [&](int step) {
            const int chunk = step * cs + rank;
            return p.reverse ? (chunks - chunk) * TILE - 1 - group * R : chunk * TILE + group * R;
        };
        auto input_of = [&](int step) {
            return stages + step % kStages * STAGE + ((p.reverse ? TILE - 1 - group * R : group * R) * LC + col) * 4;
        };
        auto load = [&](const uint8_t* at, Vec<V>& a, Vec<V>& b) {
            const Vec<V> f = Elem<BF>::get(*reinterpret_cast<const uint32_t*>(at));
            const Vec<V> x = Elem<BF>::get(*reinterpret_cast<const uint32_t*>(at + ARRAY));
            Vec<V> rest;
            gates<V>(f, a, rest);
            b = input<FORM, V>(a, rest, x);
        };
        struct Set {
            Vec<V> a[R], b[R];
            Run<V> before;
            bool plain;
            uint32_t marks;   // where not plain
        };
        auto first_half = [&](Set& q, int step) {
            const int t0 = first_row(step);
            q.plain = plain_rows<R>(c, t0, dir, seq_b, seq_e);
            if (step * cs + rank < chunks) ok = ok && tc::mbar_wait(sh.full + step % kStages, (step / kStages) & 1, &sh.abort);
            const uint8_t* in = input_of(step);
            Run<V> run{all<V>(1.f), all<V>(0.f)};
            if (q.plain) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    load(in, q.a[k], q.b[k]);
                    in += pitch_in;
                    run.b = fma(q.a[k], run.b, q.b[k]);
                    run.a = mul(run.a, q.a[k]);
                }
            } else {   // rows that begin a sequence take its first state, rows of none leave the state as it is
                q.marks = marks_of(c, t0, dir, p.reverse);
                in = apart(in);
                Vec<V> h0[R];
                states_at<V>(h0, q.marks >> 8 & 0xffu, c, t0, dir, p.H_0, p.D, ch);
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    load(in, q.a[k], q.b[k]);
                    in += pitch_in;
                    if (first_of(q.marks, k)) {
                        q.b[k] = fma(q.a[k], h0[k], q.b[k]);
                        run = Run<V>{all<V>(kReset), q.b[k]};
                    } else if (in_sequence(q.marks, k)) {
                        run.b = fma(q.a[k], run.b, q.b[k]);
                        run.a = mul(run.a, q.a[k]);   // -0 stays -0
                    } else {
                        q.a[k] = all<V>(1.f);
                        q.b[k] = all<V>(0.f);
                    }
                }
            }
            q.before = hand_over<LC, V, W>(sh, step, col, run);
        };
        auto second_half = [&](Set& q, int step) {
            const int t0 = first_row(step);
            Vec<V> h;
            if (!ok || !take_over<LC, V, W>(sh, step, col, q.before, h)) {
                ok = false;
                return;
            }
            // the state that enters the rows
            if (p.chunk_states && t0 >= 0 && t0 / kKeep * kKeep < p.T) {
                const long long at = (long long)(t0 / kKeep) * p.D + ch;
                *reinterpret_cast<Vec<V>*>(p.chunk_states + at) = h;
            }
            T* y = static_cast<T*>(p.Y) + (long long)t0 * p.ld_y + ch;
            if (q.plain) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    h = fma(q.a[k], h, q.b[k]);
                    __stcs(reinterpret_cast<uint32_t*>(y), Elem<BF>::put(h));
                    y += pitch;
                }
                bad |= wild<V>(h);   // inside a sequence a state that is not finite stays so
            } else {
                y = apart(y);
                Vec<V> at[R];
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    h = first_of(q.marks, k) ? q.b[k] : fma(q.a[k], h, q.b[k]);
                    at[k] = h;
                    if (in_sequence(q.marks, k)) {
                        bad |= wild<V>(h);
                        __stcs(reinterpret_cast<uint32_t*>(y), Elem<BF>::put(h));
                    }
                    y += pitch;
                }
                if (p.H_T)
                    for (uint32_t bits = q.marks >> 16 & 0xffu; bits; bits &= bits - 1) {
                        const int k = __ffs(bits) - 1;
                        put_state<V>(p.H_T, c.find(t0 + dir * k), p.D, ch, at[k]);
                    }
            }
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

// One token of each row: a thread takes eight channels, 16 or 32 bytes at a time.
template <bool BF, int FORM>
__global__ void __launch_bounds__(128) gated_step_kernel(int D, long long units, const void* F, long long ld_f, const void* X,
                                                         long long ld_x, const float* H, float* H_out, void* Y, long long ld_y) {
    constexpr int V = Elem<BF>::V, N = 8 / V;   // 32-bit words of eight elements
    const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= units) return;
    const int per = D / 8;
    const long long b = u / per, ch = u % per * 8;
    uint4 fw[N / 4], xw[N / 4], yw[N / 4];
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
    Vec<V>* hv = reinterpret_cast<Vec<V>*>(h);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        Vec<V> a, rest;
        gates<V>(Elem<BF>::get(reinterpret_cast<const uint32_t*>(fw)[i]), a, rest);
        hv[i] = fma(a, hv[i], input<FORM, V>(a, rest, Elem<BF>::get(reinterpret_cast<const uint32_t*>(xw)[i])));
        reinterpret_cast<uint32_t*>(yw)[i] = Elem<BF>::put(hv[i]);
    }
    float4* ho = reinterpret_cast<float4*>(H_out + b * D + ch);
    ho[0] = h[0];
    ho[1] = h[1];
    if (!Y) return;
    uint4* y = reinterpret_cast<uint4*>(static_cast<typename Elem<BF>::type*>(Y) + b * ld_y + ch);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) y[i] = yw[i];
}

template <bool BF, int FORM>
cudaError_t forward(const GatedScanArgs& a, cudaStream_t s) {
    const Shape q = shape_of(a, false);
    if (q.lanes == 32) return launch<BF, 32>(gated_fwd_kernel<BF, FORM, 32>, a, false, q.cs, s);
    if (q.lanes == 16) return launch<BF, 16>(gated_fwd_kernel<BF, FORM, 16>, a, false, q.cs, s);
    return launch<BF, 8>(gated_fwd_kernel<BF, FORM, 8>, a, false, q.cs, s);
}

}  // namespace

long long gated_scan_chunk_state_floats(int T, int D) { return ((long long)T + kKeep - 1) / kKeep * D; }

cudaError_t launch_gated_scan(const GatedScanArgs& a, cudaStream_t s) {
    const cudaError_t e = cudaMemsetAsync(a.status, 0, 16, s);
    if (e != cudaSuccess) return e;
    LaunchScope scope("gated_scan", s);
    if (a.bf16) return a.form == 0 ? forward<true, 0>(a, s) : a.form == 1 ? forward<true, 1>(a, s) : forward<true, 2>(a, s);
    return a.form == 0 ? forward<false, 0>(a, s) : a.form == 1 ? forward<false, 1>(a, s) : forward<false, 2>(a, s);
}

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
