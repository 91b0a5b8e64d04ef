// Gated linear recurrence: one thread per sequence and channel walks the rows.
#include "common.cuh"
#include "seq_offsets.cuh"

namespace ttt {
namespace {

constexpr int kChunk = 64;   // rows between two kept states

// a = sigmoid(f), 1 - a as sigmoid(-f), the input's scale s(a) and ds/df
struct Gate {
    float a, rest, s, ds;
};
__device__ __forceinline__ Gate gate(float f, int form) {
    Gate g;
    g.a = 1.f / (1.f + expf(-f));
    g.rest = 1.f / (1.f + expf(f));
    if (form == 0) {
        g.s = 1.f;
        g.ds = 0.f;
    } else if (form == 1) {
        g.s = g.rest;
        g.ds = -g.a * g.rest;
    } else {
        g.s = sqrtf(g.rest * (1.f + g.a));
        g.ds = -g.a * g.a * sqrtf(g.rest / (1.f + g.a));
    }
    return g;
}

__global__ void gated_fwd_kernel(const GatedScanArgs p) {
    const SeqOffsets c{p.cu, p.n_seq, p.T};
    const int s = blockIdx.y, ch = blockIdx.x * blockDim.x + threadIdx.x;
    if (threadIdx.x == 0 && blockIdx.x == 0 && (c.bad(s) || c.bad(s + 1))) atomicOr(p.status, kStatusBadOffsets);
    if (ch >= p.D) return;
    const int t0 = c.begin(s), t1 = c.begin(s + 1);
    float h = p.H_0 ? p.H_0[(long long)s * p.D + ch] : 0.f;
    bool bad = false;
    for (int i = t0; i < t1; ++i) {
        const int t = p.reverse ? t1 - 1 - (i - t0) : i;
        const bool first = p.reverse ? (t % kChunk == kChunk - 1 || t == t1 - 1) : (t % kChunk == 0 || t == t0);
        // the state that enters a chunk; a later sequence's first row in a chunk does not overwrite it
        if (p.chunk_states && first && (p.reverse ? t % kChunk == kChunk - 1 : t % kChunk == 0))
            p.chunk_states[(long long)(t / kChunk) * p.D + ch] = h;
        const Gate g = gate(load_elem(p.F, t * p.ld_f + ch, p.bf16), p.form);
        h = g.a * h + g.s * load_elem(p.X, t * p.ld_x + ch, p.bf16);
        store_elem(p.Y, t * p.ld_y + ch, p.bf16, h);
        bad |= !isfinite(h);
    }
    if (p.H_T) p.H_T[(long long)s * p.D + ch] = h;
    if (bad) atomicOr(p.status, kStatusNonFinite);
}

__global__ void gated_bwd_kernel(const GatedScanArgs p) {
    const SeqOffsets c{p.cu, p.n_seq, p.T};
    const int s = blockIdx.y, ch = blockIdx.x * blockDim.x + threadIdx.x;
    if (threadIdx.x == 0 && blockIdx.x == 0 && (c.bad(s) || c.bad(s + 1))) atomicOr(p.status, kStatusBadOffsets);
    if (ch >= p.D) return;
    const int t0 = c.begin(s), t1 = c.begin(s + 1);
    float lam = p.dH_T ? p.dH_T[(long long)s * p.D + ch] : 0.f;
    bool bad = false;
    float hp[kChunk];
    // chunks of the walk's end first; hp[k]: the state before walk step k of the chunk
    const int step = p.reverse ? -1 : 1;
    int c0 = p.reverse ? t0 / kChunk : (t1 - 1) / kChunk;
    for (; t1 > t0; c0 -= step) {
        const int a0 = max(c0 * kChunk, t0), a1 = min((c0 + 1) * kChunk, t1), n = a1 - a0;
        if (n <= 0) break;
        const int first = p.reverse ? a1 - 1 : a0;
        const bool start = p.reverse ? first == t1 - 1 : first == t0;
        float h = start ? (p.H_0 ? p.H_0[(long long)s * p.D + ch] : 0.f) : p.chunk_states[(long long)c0 * p.D + ch];
        for (int k = 0; k < n; ++k) {
            const int t = first + step * k;
            hp[k] = h;
            const Gate g = gate(load_elem(p.F, t * p.ld_f + ch, p.bf16), p.form);
            h = g.a * h + g.s * load_elem(p.X, t * p.ld_x + ch, p.bf16);
        }
        for (int k = n - 1; k >= 0; --k) {
            const int t = first + step * k;
            const Gate g = gate(load_elem(p.F, t * p.ld_f + ch, p.bf16), p.form);
            const float l = lam + load_elem(p.dY, t * p.ld_dy + ch, p.bf16);
            const float df = l * (hp[k] * g.a * g.rest + load_elem(p.X, t * p.ld_x + ch, p.bf16) * g.ds);
            store_elem(p.dF, t * p.ld_df + ch, p.bf16, df);
            store_elem(p.dX, t * p.ld_dx + ch, p.bf16, l * g.s);
            bad |= !isfinite(df) || !isfinite(l);
            lam = g.a * l;
        }
    }
    if (p.dH_0) p.dH_0[(long long)s * p.D + ch] = lam;
    if (bad) atomicOr(p.status, kStatusNonFinite);
}

__global__ void gated_step_kernel(int B, int D, int form, int bf16, const void* F, long long ld_f, const void* X,
                                  long long ld_x, const float* H, float* H_out, void* Y, long long ld_y) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)B * D) return;
    const int b = (int)(i / D), c = (int)(i - (long long)b * D);
    const Gate g = gate(load_elem(F, b * ld_f + c, bf16), form);
    const float h = g.a * H[i] + g.s * load_elem(X, b * ld_x + c, bf16);
    H_out[i] = h;
    if (Y) store_elem(Y, b * ld_y + c, bf16, h);
}

}  // namespace

long long gated_scan_workspace_bytes(int, int) { return 0; }
long long gated_scan_chunk_state_floats(int T, int D) { return (long long)((T + kChunk - 1) / kChunk) * D; }

cudaError_t launch_gated_scan(const GatedScanArgs& a, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(a.status, 0, 16, s);
    if (e != cudaSuccess) return e;
    LaunchScope scope("gated_scan", s);
    gated_fwd_kernel<<<dim3((a.D + 63) / 64, a.n_seq), 64, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_gated_scan_backward(const GatedScanArgs& a, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(a.status, 0, 16, s);
    if (e != cudaSuccess) return e;
    LaunchScope scope("gated_scan_backward", s);
    gated_bwd_kernel<<<dim3((a.D + 63) / 64, a.n_seq), 64, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_gated_scan_step(int B, int D, int form, int bf16, const void* F, long long ld_f, const void* X,
                                   long long ld_x, const float* H, float* H_out, void* Y, long long ld_y,
                                   cudaStream_t s) {
    LaunchScope scope("gated_scan_step", s);
    gated_step_kernel<<<(unsigned)(((long long)B * D + 255) / 256), 256, 0, s>>>(B, D, form, bf16, F, ld_f, X, ld_x, H,
                                                                               H_out, Y, ld_y);
    return cudaGetLastError();
}

}  // namespace ttt
