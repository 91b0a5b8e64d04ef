// Window attention, one token per request: one warp per request and query head.
#include "common.cuh"

namespace ttt {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__global__ void window_decode_kernel(const WindowDecodeArgs p) {
    const int b = blockIdx.x, h = blockIdx.y, lane = threadIdx.x, G = p.Hq / p.Hk, hk = h / G;
    const int ring = p.slots - p.sinks;
    int n = p.lens[b];
    if (n < 0 || (n > p.slots && ring < 1)) {
        if (lane == 0) atomicOr(p.status, kStatusBadOffsets);
        n = 0;
    }
    auto slot = [&](int u) { return u < p.slots ? u : p.sinks + (u - p.sinks) % ring; };
    const long long base = b * p.ld_request + hk * p.ld_head + 2 * lane;
    const __nv_bfloat16* q = p.Q + b * p.ld_q + h * 64 + 2 * lane;
    const float q0 = __bfloat162float(q[0]), q1 = __bfloat162float(q[1]);
    float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
    const int lo = max(max(n - 1 - p.left, 0), n > p.slots ? n - ring : 0);
    for (int u = min(p.sinks, lo) > 0 ? 0 : lo; u < n; ++u) {
        if (u == p.sinks && u < lo) u = lo;
        if (u >= n) break;
        const long long at = base + slot(u) * p.ld_slot;
        __nv_bfloat162 k, v;
        if (u == n - 1 && p.K_new) {
            const long long nw = b * p.ld_new + hk * 64 + 2 * lane;
            k = *reinterpret_cast<const __nv_bfloat162*>(p.K_new + nw);
            v = *reinterpret_cast<const __nv_bfloat162*>(p.V_new + nw);
            if (h == hk * G) {
                *reinterpret_cast<__nv_bfloat162*>(p.K_cache + at) = k;
                *reinterpret_cast<__nv_bfloat162*>(p.V_cache + at) = v;
            }
        } else {
            k = *reinterpret_cast<const __nv_bfloat162*>(p.K_cache + at);
            v = *reinterpret_cast<const __nv_bfloat162*>(p.V_cache + at);
        }
        const float x = p.scale * warp_sum(q0 * __low2float(k) + q1 * __high2float(k));
        const float m2 = x > m || x != x ? x : m, f = m2 == -INFINITY ? 1.f : expf(m - m2), e = m2 == -INFINITY ? 0.f : expf(x - m2);
        l = l * f + e;
        o0 = o0 * f + e * __low2float(v);
        o1 = o1 * f + e * __high2float(v);
        m = m2;
    }
    o0 = l > 0.f ? o0 / l : l;
    o1 = l > 0.f ? o1 / l : l;
    if (!(isfinite(o0) && isfinite(o1))) atomicOr(p.status, kStatusNonFinite);
    __nv_bfloat16* out = p.Out + b * p.ld_out + h * 64 + 2 * lane;
    out[0] = __float2bfloat16_rn(o0);
    out[1] = __float2bfloat16_rn(o1);
}

}  // namespace

cudaError_t launch_window_decode(const WindowDecodeArgs& a, cudaStream_t s) {
    LaunchScope scope("window_decode", s);
    window_decode_kernel<<<dim3(a.B, a.Hq), 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace ttt
