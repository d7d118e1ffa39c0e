// What the block boundary's forward and gradient kernels share: sums over a row by a team of
// warps. Internal; everything in an anonymous namespace.
#pragma once

#include "zero_act.cuh"

namespace zk {
namespace {

constexpr int kMaxWarps = 16;          // warps of a CTA
constexpr int kMaxCluster = 8;         // CTAs that share a row

uint32_t chunks_of(uint64_t cols) { return (uint32_t)((cols + kWarpCols - 1) / kWarpCols); }

// The warps that share a row: `warps` of this CTA, from warp `first`, times `ctas` of a cluster.
// Entries of `part` alternate between two slots, so that one barrier per sum is enough.
struct Team {
    float (*part)[kMaxWarps * kMaxCluster][4];
    uint32_t lane, warp, first, warps, ctas, rank, bar;
    uint32_t slot;
};

__device__ __forceinline__ void cluster_barrier() {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
            : "memory");
}

// Sums of N = 2 or 4 values over the team, the same in every lane, in a fixed order. The first
// steps halve the values a lane carries: lane l ends with the sum of value l / (32/N). Up to 16
// warps of one CTA meet in shared memory; the CTAs of a cluster store into each other's.
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
    if (t.warps * t.ctas > 1) {
        float(*part)[4] = t.part[t.slot];
        t.slot ^= 1u;
        const uint32_t k = t.lane / kLanes, e = t.lane % kLanes;
        if (t.ctas == 1) {
            if (e == 0) part[t.first + t.warp][k] = s;
            asm volatile("bar.sync %0, %1;" ::"r"(t.bar), "r"(t.warps * 32u) : "memory");
            s = e < t.warps ? part[t.first + e][k] : 0.0f;
            if (N == 4 && e + 8 < t.warps) s = __fadd_rn(s, part[t.first + e + 8][k]);
        } else {
            if (e == 0) {
                const uint32_t at = smem_addr(&part[t.rank * t.warps + t.warp][k]);
                for (uint32_t r = 0; r < t.ctas; ++r) {
                    uint32_t to;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(r));
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(s) : "memory");
                }
            }
            cluster_barrier();
            s = 0.0f;
            for (uint32_t i = e; i < t.warps * t.ctas; i += kLanes) s = __fadd_rn(s, part[i][k]);
        }
#pragma unroll
        for (uint32_t d = kLanes / 2; d > 0; d >>= 1)
            s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(0xffffffffu, s, k * kLanes);
}

__device__ __forceinline__ uint64_t both(float a) { return f2_pack(a, a); }

// ---------------------------------------------------------------------------------------------
// Rows on their way to a thread. A thread copies its own columns of the next rows into slots of
// shared memory that only it reads (cp.async: no register holds a load in flight, and nothing
// else the thread loads waits for them), kDepth rows ahead.
// ---------------------------------------------------------------------------------------------
// Copies of 16 bytes bypass L1, unless the neighbouring half of a 32-byte sector is another copy
// of the same warp's (32-bit values: through L1 it is fetched once).
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int bytes,
                                           bool halves = false) {
    if (bytes == 16 && halves)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else if (bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else if (bytes == 8)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// All but the last N groups of this thread's copies have landed.
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Slot n of this thread: 8 * sizeof(T) bytes as 16-byte words `threads` apart (no bank conflicts).
template <typename T>
struct Slots {
    uint32_t base, threads;   // this thread's first word; threads of the CTA
    static constexpr uint32_t kWords = sizeof(T) / 2;
    __device__ __forceinline__ uint32_t word(uint32_t n, uint32_t k) const {
        return base + (n * kWords + k) * threads * 16u;
    }
    __device__ __forceinline__ void clear(uint32_t n) const {
#pragma unroll
        for (uint32_t k = 0; k < kWords; ++k)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(word(n, k)), "r"(0)
                         : "memory");
    }
    __device__ __forceinline__ Raw<T> get(uint32_t n) const {
        Raw<T> r;
#pragma unroll
        for (uint32_t k = 0; k < kWords; ++k)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.w[4 * k]), "=r"(r.w[4 * k + 1]), "=r"(r.w[4 * k + 2]),
                           "=r"(r.w[4 * k + 3])
                         : "r"(word(n, k))
                         : "memory");
        return r;
    }
    __device__ __forceinline__ void put(uint32_t n, const Raw<T>& r) const {
#pragma unroll
        for (uint32_t k = 0; k < kWords; ++k)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(word(n, k)),
                         "r"(r.w[4 * k]), "r"(r.w[4 * k + 1]), "r"(r.w[4 * k + 2]),
                         "r"(r.w[4 * k + 3])
                         : "memory");
    }
    // a lane's columns of a row of a matrix (kNarrow: 32-bit values), or the codes and scale of a
    // checkpoint's (kWide)
    template <int kA>
    __device__ __forceinline__ void copy(uint32_t n, const T* row, const Cols<kA>& c) const {
        if constexpr (kA == kWide) {
            if (!c.any()) return;
#pragma unroll
            for (uint32_t k = 0; k < kWords; ++k)
                copy_async(word(n, k), row + c.c0 + k * 16 / sizeof(T), 16, kWords > 1);
        } else {
            static_assert(sizeof(T) == 4, "cp.async moves 4 bytes at least");
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c.mask >> j & 1u) copy_async(word(n, j / 4) + 4 * (j % 4), row + c.at(j), 4);
        }
    }
    __device__ __forceinline__ void copy_codes(uint32_t n, const uint8_t* row, const CkptShape& s,
                                               const Cols<kWide>& c) const {
        if (!c.any()) return;
        copy_async(word(n, 0), row + c.c0, 8);
        copy_async(word(n, 0) + 8, ckpt_scales(row, s) + (c.c0 >> 7), 4);
    }
    // (kNarrow leaves a checkpoint's row to get_row: its single bytes cannot be copied)
    template <int kA>
    __device__ __forceinline__ void copy_row(uint32_t n, const Rows& m, bool codes,
                                             const CkptShape& s, uint32_t r,
                                             const Cols<kA>& c) const {
        if (!codes)
            copy<kA>(n, row_of<T>(m, r), c);
        else if constexpr (kA == kWide)
            copy_codes(n, row_of<uint8_t>(m, r), s, c);
    }
    // values of row r, from the slot that copy_row filled
    template <int kA>
    __device__ __forceinline__ Raw<T> get_row(uint32_t n, const Rows& m, bool codes,
                                              const CkptShape& s, uint32_t r,
                                              const Cols<kA>& c) const {
        if (kA == kNarrow && codes) return load_codes<T, kA>(row_of<uint8_t>(m, r), s, c);
        Raw<T> v = get(n);
        if (codes) v.w[3] = v.w[2];
        return v;
    }
};

// Whether rows travel through slots: 16-bit values that cannot move as 16 bytes go through
// registers, one row ahead.
template <typename T, int kA>
constexpr bool piped() { return kA == kWide || sizeof(T) == 4; }

// Let a kernel use up to `most` bytes of dynamic shared memory on device `dev`, and tell how many
// of its CTAs (threads, smem) an SM holds at once. Asked once per host thread and shape.
template <typename K>
cudaError_t resident(K kernel, int dev, unsigned threads, size_t smem, size_t most, int* ctas) {
    constexpr int kSlots = 64;
    thread_local struct {
        const void* kernel;
        int dev;
        unsigned threads;
        int ctas;
    } known[kSlots];
    thread_local int used = 0;
    const void* kp = reinterpret_cast<const void*>(kernel);
    for (int i = 0; i < used; ++i)
        if (known[i].kernel == kp && known[i].dev == dev && known[i].threads == threads) {
            *ctas = known[i].ctas;
            return cudaSuccess;
        }
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)most);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, kernel, (int)threads, smem);
    if (e != cudaSuccess) return e;
    if (*ctas < 1) return cudaErrorInvalidConfiguration;
    if (used < kSlots) known[used++] = {kp, dev, threads, *ctas};
    return cudaSuccess;
}

// launch_act in clusters of `ctas` CTAs.
template <typename K, typename... A>
cudaError_t launch_clusters(K kernel, unsigned clusters, unsigned ctas, unsigned threads,
                            size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
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

// kWide where every operand moves in 16-byte accesses, else kNarrow.
template <typename T>
Access all_access(const JoinArgs& a) {
    if (a.cols % 8 != 0) return kNarrow;
    for (const Rows* m : {&a.gate, &a.x, &a.h, &a.y, &a.u, &a.dy, &a.du, &a.dx, &a.dh, &a.dgate})
        if (m->p && (!aligned16(m->p) || m->pitch % 16 != 0)) return kNarrow;
    for (const void* v : {a.post_w, a.post_b, a.pre_w, a.pre_b})
        if (!aligned16(v)) return kNarrow;
    return kWide;
}

}  // namespace
}  // namespace zk
