// Window attention with sinks, forward: one warp per query row and head.
#include "common.cuh"
#include "window_mask.cuh"

namespace ttt {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__global__ void window_fwd_kernel(const WindowArgs p) {
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
    const __nv_bfloat16* q = p.Q + t * p.ld_q + h * 64 + 2 * lane;
    const float q0 = __bfloat162float(q[0]), q1 = __bfloat162float(q[1]);
    float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
    const int lo = max(pos - p.left, 0), hi = min(pos + p.right, nk - 1);
    for (int u = min(p.sinks, lo) > 0 ? 0 : lo; u <= hi; ++u) {
        if (u == p.sinks && u < lo) u = lo;
        if (u > hi) break;
        const __nv_bfloat16* k = p.K + (k0 + u) * p.ld_k + hk * 64 + 2 * lane;
        const __nv_bfloat16* v = p.V + (k0 + u) * p.ld_v + hk * 64 + 2 * lane;
        const float x = p.scale * warp_sum(q0 * __bfloat162float(k[0]) + q1 * __bfloat162float(k[1]));
        const float m2 = x > m || x != x ? x : m, f = m2 == -INFINITY ? 1.f : expf(m - m2), e = m2 == -INFINITY ? 0.f : expf(x - m2);
        l = l * f + e;
        o0 = o0 * f + e * __bfloat162float(v[0]);
        o1 = o1 * f + e * __bfloat162float(v[1]);
        m = m2;
    }
    o0 = l > 0.f ? o0 / l : l;   // an empty row is 0, a NaN sum stays
    o1 = l > 0.f ? o1 / l : l;
    if (!(isfinite(o0) && isfinite(o1))) atomicOr(p.status, kStatusNonFinite);
    const long long at = t * p.ld_out + h * 64 + 2 * lane;
    if (p.Xres) {
        o0 += __bfloat162float(p.Xres[at]);
        o1 += __bfloat162float(p.Xres[at + 1]);
    }
    p.Out[at] = __float2bfloat16_rn(o0);
    p.Out[at + 1] = __float2bfloat16_rn(o1);
    if (p.Lse && lane == 0) p.Lse[(long long)h * p.Tq + t] = m == -INFINITY ? m : m + logf(l);
}

}  // namespace

cudaError_t launch_window_attention(const WindowArgs& a, cudaStream_t s) {
    LaunchScope scope("window_attn", s);
    const long long warps = (long long)a.Tq * a.Hq;
    window_fwd_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ttt
