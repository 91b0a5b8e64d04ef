// Window attention, one token per request, on its cache (head dim 64, bf16).
//
// Every visible key and value is read once: the bytes of the cache bound it.  A cluster of up to eight CTAs takes
// one request and key head (and sixteen of the query heads that share it, padded to the matrix instruction's 16
// rows); its warps take tiles of 32 visible keys in turn, each through a ring of its own (cp.async, 16 bytes a
// lane, rows in a 128-byte swizzle; no barrier between warps; two stages, so that three CTAs share an SM: 64 requests
// x 16,388 keys in 377 us, 5.7 TB/s, against 427 us with three stages and two CTAs).  S = Q K^T and O += P V run on mma.sync with the
// softmax's statistics in registers: one token gives far too few rows for tcgen05's 128, and the tensor time is
// a few percent of the loads'.  The warps' partial results join in shared memory, the CTAs' in the first CTA's
// (distributed shared memory), in a fixed order: no workspace, no second launch.
//
// Keys that are not visible are never loaded (a tile's rest is zero-filled and masked), so whatever the cache
// holds there does not matter.
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_prims.cuh"
#include "common.cuh"

namespace ttt {
namespace {

constexpr int kWarps = 4, kTile = 32, kStages = 2, kHeads = 16, DH = 64, kMaxCluster = 8;
constexpr int kStageBytes = 2 * kTile * DH * 2;   // K and V rows of a tile

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct Partial {      // of sixteen query heads: unnormalised outputs, reference maxima (log2 units) and sums
    float o[kHeads][DH], m[kHeads], l[kHeads];
};

__global__ void __launch_bounds__(32 * kWarps) window_decode_kernel(const WindowDecodeArgs p, float c, int cs) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % cs, item = blockIdx.x / cs, G = p.Hq / p.Hk, per = (G + kHeads - 1) / kHeads;
    const int part = item % per, hk = item / per % p.Hk, b = item / per / p.Hk;
    const int h0 = hk * G + part * kHeads, heads = min(kHeads, G - part * kHeads);
    const int ring = p.slots - p.sinks;
    int n = p.lens[b];
    if (n < 0 || (n > p.slots && ring < 1)) {
        if (rank == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBadOffsets);
        n = 0;
    }
    // visible: the first `ns` positions, then [lo, n)
    const int lo = max(max(n - 1 - min(p.left, n), 0), n > p.slots ? n - ring : 0), ns = min(p.sinks, lo), total = ns + n - lo;
    // position n - d, past the sinks, lies in the ring's place (n - sinks - d) mod ring
    const int turn = ring > 0 && n > p.sinks ? (n - p.sinks) % ring : 0;
    auto slot_of = [&](int u) {
        if (u < p.sinks) return u;
        const int r = turn - (n - u);
        return p.sinks + (r < 0 ? r + ring : r);
    };
    const long long head_at = b * p.ld_request + hk * p.ld_head;
    const bool fresh = p.K_new != nullptr && n > 0;
    const long long new_at = b * p.ld_new + (long long)hk * DH;
    if (fresh && rank == 0 && part == 0 && threadIdx.x < 16) {   // the token's key and value go to their slot
        const int ch = threadIdx.x % 8 * 8;
        const long long at = head_at + slot_of(n - 1) * p.ld_slot + ch;
        if (threadIdx.x < 8) *reinterpret_cast<uint4*>(p.K_cache + at) = *reinterpret_cast<const uint4*>(p.K_new + new_at + ch);
        else *reinterpret_cast<uint4*>(p.V_cache + at) = *reinterpret_cast<const uint4*>(p.V_new + new_at + ch);
    }

    // the warp's tiles: first, first + step, ...
    const int tiles = (total + kTile - 1) / kTile, first = rank * kWarps + warp, step = cs * kWarps;
    uint8_t* ringbuf = smem + warp * kStages * kStageBytes;
    const uint32_t ring_at = tc::smem_u32(ringbuf);
    auto fetch = [&](int tile, int stage) {
        const uint32_t to = ring_at + stage * kStageBytes;
#pragma unroll
        for (int i = 0; i < kTile / 4; ++i) {   // four keys a pass, eight 16-byte chunks each
            const int key = 4 * i + lane / 8, ch = lane % 8, j = tile * kTile + key;
            const bool in = tile < tiles && j < total;
            const int u = j < ns ? j : lo + (j - ns);
            const __nv_bfloat16 *k = p.K_cache, *v = p.V_cache;
            if (in) {
                const bool use_new = fresh && u == n - 1;
                const long long at = use_new ? new_at : head_at + slot_of(u) * p.ld_slot;
                k = (use_new ? p.K_new : p.K_cache) + at + ch * 8;
                v = (use_new ? p.V_new : p.V_cache) + at + ch * 8;
            }
            const uint32_t dst = to + key * 128 + ((ch ^ (key & 7)) << 4);
            cp_async16(dst, k, in);
            cp_async16(dst + kTile * 128, v, in);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(first + s * step, s);

    // Q as A operand: rows are heads (g and g + 8), zero beyond the last
    const int g = lane >> 2, q4 = lane & 3;
    uint32_t qa[DH / 16][4];
    {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p.Q + b * p.ld_q + (long long)h0 * DH) + q4;
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = g + 8 * (r & 1);
                qa[kk][r] = row < heads ? q[row * (DH / 2) + kk * 8 + 4 * (r >> 1)] : 0u;
            }
    }
    float o[DH / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int stage = 0;
    for (int t = first; t < tiles; t += step) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncwarp();
        fetch(t + (kStages - 1) * step, (stage + kStages - 1) % kStages);   // into the stage read a turn ago
        const uint32_t ks = ring_at + stage * kStageBytes, vs = ks + kTile * 128;
        float s[kTile / 8][4] = {};
#pragma unroll
        for (int nt = 0; nt < kTile / 8; ++nt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {   // 32 of the 64 columns
                uint32_t kb[4];
                const int key = nt * 8 + (lane & 7), ch = half * 4 + (lane >> 3);
                ldmatrix_x4(ks + key * 128 + ((ch ^ (key & 7)) << 4), kb);
                mma_bf16(s[nt], qa[2 * half], kb[0], kb[1]);
                mma_bf16(s[nt], qa[2 * half + 1], kb[2], kb[3]);
            }
        const int left = total - t * kTile;
        if (left < kTile) {
#pragma unroll
            for (int nt = 0; nt < kTile / 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (nt * 8 + 2 * q4 + (e & 1) >= left) s[nt][e] = -INFINITY;
        }
        uint32_t pa[kTile / 16][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {   // rows g and g + 8
            float mt = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < kTile / 8; ++nt) mt = fmaxf(mt, fmaxf(s[nt][2 * r], s[nt][2 * r + 1]));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
            const float m2 = fmaxf(m[r], mt * c), ref = m2 == -INFINITY ? 0.f : m2, f = attn::ex2(m[r] - ref);
            m[r] = m2;
            float sum = 0.f;
#pragma unroll
            for (int nt = 0; nt < kTile / 8; ++nt) {
                const float p0 = attn::ex2(fmaf(s[nt][2 * r], c, -ref)), p1 = attn::ex2(fmaf(s[nt][2 * r + 1], c, -ref));
                sum += p0 + p1;
                pa[nt / 2][(nt & 1) * 2 + r] = attn::pack_bf16(p0, p1);   // the weights enter the product as bf16
            }
            l[r] = l[r] * f + sum;
#pragma unroll
            for (int d = 0; d < DH / 8; ++d) {
                o[d][2 * r] *= f;
                o[d][2 * r + 1] *= f;
            }
        }
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
#pragma unroll
            for (int d2 = 0; d2 < DH / 16; ++d2) {   // sixteen columns: matrices (keys 0-7, 8-15) x (columns 0-7, 8-15)
                uint32_t vb[4];
                const int key = kk * 16 + (lane & 15), ch = d2 * 2 + (lane >> 4);
                ldmatrix_x4_trans(vs + key * 128 + ((ch ^ (key & 7)) << 4), vb);
                mma_bf16(o[2 * d2], pa[kk], vb[0], vb[1]);
                mma_bf16(o[2 * d2 + 1], pa[kk], vb[2], vb[3]);
            }
        stage = (stage + 1) % kStages;
        __syncwarp();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    // this CTA's tiles are no longer needed: the others may write where they were
    if (cs > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    // ---- join: the warps' results, then the CTAs' in the cluster's first one
    Partial* warps = reinterpret_cast<Partial*>(smem);
    Partial* ctas = warps + kWarps;          // [kMaxCluster], used in the first CTA
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        const int row = g + 8 * r;
#pragma unroll
        for (int d = 0; d < DH / 8; ++d)
            *reinterpret_cast<float2*>(&warps[warp].o[row][d * 8 + 2 * q4]) = make_float2(o[d][2 * r], o[d][2 * r + 1]);
        if (q4 == 0) {
            warps[warp].m[row] = m[r];
            warps[warp].l[row] = l[r];
        }
    }
    __syncthreads();
    const int row = threadIdx.x / 8, col = threadIdx.x % 8 * 8;
    float mj, lj, oj[8];
    auto join = [&](const Partial* q, int count) {
        mj = -INFINITY;
        lj = 0.f;
        for (int i = 0; i < count; ++i) mj = fmaxf(mj, q[i].m[row]);
        const float ref = mj == -INFINITY ? 0.f : mj;
#pragma unroll
        for (int e = 0; e < 8; ++e) oj[e] = 0.f;
        for (int i = 0; i < count; ++i) {
            const float f = attn::ex2(q[i].m[row] - ref);
            lj = fmaf(f, q[i].l[row], lj);
#pragma unroll
            for (int e = 0; e < 8; ++e) oj[e] = fmaf(f, q[i].o[row][col + e], oj[e]);
        }
    };
    join(warps, kWarps);
    if (cs > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        Partial* mine = &ctas[rank];
        const uint32_t to = tc::mapa_shared(tc::smem_u32(&mine->o[row][col]), 0);
        tc::st_cluster_v4(to, oj[0], oj[1], oj[2], oj[3]);
        tc::st_cluster_v4(to + 16, oj[4], oj[5], oj[6], oj[7]);
        if (col == 0) {
            tc::st_cluster_f32(tc::mapa_shared(tc::smem_u32(&mine->m[row]), 0), mj);
            tc::st_cluster_f32(tc::mapa_shared(tc::smem_u32(&mine->l[row]), 0), lj);
        }
        tc::cluster_sync();
        if (rank != 0) return;
        join(ctas, cs);
    }
    if (row >= heads) return;
    float v[8];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // an idle request is 0; a sum that is NaN, or 0 because every score is -infinity, makes NaN as in the formula
        v[e] = total == 0 ? 0.f : lj > 0.f ? oj[e] / lj : NAN;
        bad |= !isfinite(v[e]);
    }
    if (bad) atomicOr(p.status, kStatusNonFinite);
    *reinterpret_cast<uint4*>(p.Out + b * p.ld_out + (long long)(h0 + row) * DH + col) =
        make_uint4(attn::pack_bf16(v[0], v[1]), attn::pack_bf16(v[2], v[3]), attn::pack_bf16(v[4], v[5]), attn::pack_bf16(v[6], v[7]));
}

constexpr int kSmem = kWarps * kStages * kStageBytes;
static_assert(kSmem >= (int)sizeof(Partial) * (kWarps + kMaxCluster), "the partial results fit where the tiles were");

}  // namespace

cudaError_t launch_window_decode(const WindowDecodeArgs& a, cudaStream_t s) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaError_t e = cudaFuncSetAttribute(window_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int G = a.Hq / a.Hk;
    const long long items = (long long)a.B * a.Hk * ((G + kHeads - 1) / kHeads);
    const long long keys = std::min<long long>(a.slots, (long long)a.left + 1 + a.sinks);   // at most, per request
    // split the keys while the card has room (four waves of three CTAs per SM, for requests of unequal lengths: the
    // 377 us above are 405 with half as many, 491 with a quarter) and every warp keeps a tile
    int cs = 1;
    while (cs < kMaxCluster && items * cs < 12LL * sms && keys > (long long)cs * kWarps * kTile) cs *= 2;
    if (items * cs > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(items * cs));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    LaunchScope scope("window_decode", s);
    return cudaLaunchKernelEx(&cfg, window_decode_kernel, a, (float)(a.scale * 1.4426950408889634), cs);
}

}  // namespace ttt
