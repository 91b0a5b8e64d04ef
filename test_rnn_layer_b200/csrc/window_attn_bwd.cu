// Window attention with sinks, backward: one warp per query row (dQ), one per key row (dK, dV).
#include "common.cuh"
#include "window_mask.cuh"

namespace ttt {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct Pair {
    float x, y;
};
__device__ __forceinline__ Pair load2(const __nv_bfloat16* base, long long ld, int row, int h, int lane) {
    const __nv_bfloat16* q = base + row * ld + h * 64 + 2 * lane;
    return {__bfloat162float(q[0]), __bfloat162float(q[1])};
}
__device__ __forceinline__ void store2(__nv_bfloat16* base, long long ld, int row, int h, int lane, Pair v) {
    __nv_bfloat16* q = base + row * ld + h * 64 + 2 * lane;
    q[0] = __float2bfloat16_rn(v.x);
    q[1] = __float2bfloat16_rn(v.y);
}

__global__ void window_dq_kernel(const WindowArgs p) {
    const SeqOffsets cq{p.cu_q, p.n_seq, p.Tq}, ck{p.cu_k, p.n_seq, p.Tk};
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s <= p.n_seq; s += blockDim.x)
            if (cq.bad(s) || ck.bad(s)) atomicOr(p.status, kStatusBadOffsets);
    if (w >= (long long)p.Tq * p.Hq) return;
    const int t = (int)(w / p.Hq), h = (int)(w % p.Hq), hk = h / (p.Hq / p.Hk);
    const int s = cq.find(t);
    if (t < cq.begin(s) || t >= cq.begin(s + 1)) return;
    const int k0 = ck.begin(s), nk = max(ck.begin(s + 1) - k0, 0);
    const int pos = nk - (cq.begin(s + 1) - cq.begin(s)) + t - cq.begin(s);
    const Pair q = load2(p.Q, p.ld_q, t, h, lane), g = load2(p.dOut, p.ld_do, t, h, lane), o = load2(p.Out, p.ld_out, t, h, lane);
    const float lse = p.Lse[(long long)h * p.Tq + t], delta = warp_sum(g.x * o.x + g.y * o.y);
    if (lane == 0) p.delta[(long long)h * p.Tq + t] = delta;
    Pair d = {0.f, 0.f};
    const int lo = max(pos - p.left, 0), hi = min(pos + p.right, nk - 1);
    for (int u = p.sinks > 0 ? 0 : lo; u <= hi; ++u) {
        if (!window_sees(pos, u, p.left, p.right, p.sinks)) continue;
        const Pair k = load2(p.K, p.ld_k, k0 + u, hk, lane), v = load2(p.V, p.ld_v, k0 + u, hk, lane);
        const float x = p.scale * warp_sum(q.x * k.x + q.y * k.y), dp = warp_sum(g.x * v.x + g.y * v.y);
        const float ds = p.scale * expf(x - lse) * (dp - delta);
        d.x += ds * k.x;
        d.y += ds * k.y;
    }
    if (!(isfinite(d.x) && isfinite(d.y))) atomicOr(p.status, kStatusNonFinite);
    store2(p.dQ, p.ld_dq, t, h, lane, d);
}

__global__ void window_dkv_kernel(const WindowArgs p) {
    const SeqOffsets cq{p.cu_q, p.n_seq, p.Tq}, ck{p.cu_k, p.n_seq, p.Tk};
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (w >= (long long)p.Tk * p.Hk) return;
    const int t = (int)(w / p.Hk), hk = (int)(w % p.Hk), G = p.Hq / p.Hk;
    const int s = ck.find(t);
    if (t < ck.begin(s) || t >= ck.begin(s + 1)) return;
    const int u = t - ck.begin(s), q0 = cq.begin(s), nq = max(cq.begin(s + 1) - q0, 0);
    const int shift = ck.begin(s + 1) - ck.begin(s) - nq;
    const Pair k = load2(p.K, p.ld_k, t, hk, lane), v = load2(p.V, p.ld_v, t, hk, lane);
    Pair dk = {0.f, 0.f}, dv = {0.f, 0.f};
    for (int h = hk * G; h < hk * G + G; ++h)
        for (int i = 0; i < nq; ++i) {
            if (!window_sees(shift + i, u, p.left, p.right, p.sinks)) continue;
            const Pair q = load2(p.Q, p.ld_q, q0 + i, h, lane), g = load2(p.dOut, p.ld_do, q0 + i, h, lane);
            const float x = p.scale * warp_sum(q.x * k.x + q.y * k.y), dp = warp_sum(g.x * v.x + g.y * v.y);
            const long long at = (long long)h * p.Tq + q0 + i;
            const float e = expf(x - p.Lse[at]), ds = p.scale * e * (dp - p.delta[at]);
            dv.x += e * g.x;
            dv.y += e * g.y;
            dk.x += ds * q.x;
            dk.y += ds * q.y;
        }
    if (!(isfinite(dk.x) && isfinite(dk.y) && isfinite(dv.x) && isfinite(dv.y))) atomicOr(p.status, kStatusNonFinite);
    store2(p.dK, p.ld_dk, t, hk, lane, dk);
    store2(p.dV, p.ld_dv, t, hk, lane, dv);
}

}  // namespace

cudaError_t launch_window_attention_backward(const WindowArgs& a, cudaStream_t s) {
    if (a.Tq) {
        LaunchScope scope("window_dq", s);
        window_dq_kernel<<<(unsigned)(((long long)a.Tq * a.Hq + 7) / 8), 256, 0, s>>>(a);
    }
    if (a.Tk) {
        LaunchScope scope("window_dkv", s);
        window_dkv_kernel<<<(unsigned)(((long long)a.Tk * a.Hk + 7) / 8), 256, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace ttt
