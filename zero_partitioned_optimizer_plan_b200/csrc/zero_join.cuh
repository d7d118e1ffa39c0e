// What the block boundary's forward and gradient kernels share: sums over a row by a team of
// warps. Internal; everything in an anonymous namespace.
#pragma once

#include "zero_act.cuh"

namespace zk {
namespace {

constexpr int kMaxWarps = 16;          // warps of a CTA
constexpr int kMaxCluster = 8;

uint32_t chunks_of(uint64_t cols) { return (uint32_t)((cols + kWarpCols - 1) / kWarpCols); }

// ---------------------------------------------------------------------------------------------
// sums over a row
// ---------------------------------------------------------------------------------------------
// The warps that share a row: `warps` of this CTA, from warp `first`, times `ctas` of a cluster.
// Entries of `part` alternate between two slots, so that one barrier per sum is enough.
struct Team {
    float (*part)[kMaxWarps * kMaxCluster][4];
    uint32_t lane, warp, first, warps, ctas, rank, bar;
    uint32_t slot;
};

__device__ __forceinline__ void team_barrier(const Team& t) {
    if (t.ctas > 1) {
        asm volatile(
            "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                : "memory");
    } else {
        asm volatile("bar.sync %0, %1;" ::"r"(t.bar), "r"(t.warps * 32u) : "memory");
    }
}

// Sums of N = 2 or 4 values over the team, the same in every lane, in a fixed order. The first
// steps halve the values a lane carries: lane l ends with the sum of value l / (32/N).
template <int N>
__device__ __forceinline__ void team_sum(Team& t, float (&v)[N]) {
    constexpr uint32_t kLanes = 32 / N;
    float s;
    const bool hi = t.lane & 16u;
    if constexpr (N == 4) {
        const float a = __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
        const float b = __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
        const float c = __fadd_rn(hi ? v[2] : v[0], a), d = __fadd_rn(hi ? v[3] : v[1], b);
        const bool odd = t.lane & 8u;
        s = __fadd_rn(odd ? d : c, __shfl_xor_sync(0xffffffffu, odd ? c : d, 8));
    } else {
        s = __fadd_rn(hi ? v[1] : v[0], __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[1], 16));
    }
#pragma unroll
    for (uint32_t d = kLanes / 2; d > 0; d >>= 1)
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
    const uint32_t total = t.warps * t.ctas;
    if (total > 1) {
        float(*part)[4] = t.part[t.slot];
        t.slot ^= 1u;
        const uint32_t k = t.lane / kLanes, e0 = t.lane % kLanes;
        if (e0 == 0) {
            const uint32_t e = t.first + t.rank * t.warps + t.warp;
            if (t.ctas > 1) {
                const uint32_t at = smem_addr(&part[e][k]);
                for (uint32_t r = 0; r < t.ctas; ++r) {
                    uint32_t to;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(r));
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(s) : "memory");
                }
            } else {
                part[e][k] = s;
            }
        }
        team_barrier(t);
        s = 0.0f;
        for (uint32_t e = e0; e < total; e += kLanes) s = __fadd_rn(s, part[t.first + e][k]);
#pragma unroll
        for (uint32_t d = kLanes / 2; d > 0; d >>= 1)
            s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(0xffffffffu, s, k * kLanes);
}

__device__ __forceinline__ uint64_t row_over(uint64_t r, uint64_t d) {
    return ((r | d) >> 32) == 0 ? (uint64_t)((uint32_t)r / (uint32_t)d) : r / d;
}

__device__ __forceinline__ uint64_t both(float a) { return f2_pack(a, a); }

// launch_act in clusters of `ctas` CTAs.
template <typename K, typename... A>
cudaError_t launch_clusters(K kernel, unsigned clusters, unsigned ctas, unsigned threads,
                            cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * ctas);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    count_launch();
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

// Whether every operand moves in 16-byte accesses.
template <typename T>
bool all_aligned(const JoinArgs& a) {
    for (const Mat* m : {&a.gate, &a.x, &a.h, &a.y, &a.u, &a.dy, &a.du, &a.dx, &a.dh, &a.dgate})
        if (m->p && !rows_aligned<T>(*m)) return false;
    for (const void* v : {a.post_w, a.post_b, a.pre_w, a.pre_b})
        if (!aligned16(v)) return false;
    return true;
}

}  // namespace
}  // namespace zk
