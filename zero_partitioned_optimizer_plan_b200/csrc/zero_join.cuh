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
// kNarrow 16-bit rows use one more 4-byte word per warp and slot, lane 0's, at `extra`.
template <typename T>
struct Slots {
    uint32_t base, threads;   // this thread's first word; threads of the CTA
    uint32_t extra;           // this warp's first extra word; the next slot's is threads/8 away
    __device__ __forceinline__ Slots(uint32_t smem, uint32_t count)
        : base(smem + threadIdx.x * 16u), threads(blockDim.x),
          extra(smem + count * kWords * blockDim.x * 16u + (threadIdx.x >> 5) * 4u) {}
    // bytes of shared memory of `count` slots
    static size_t bytes(uint32_t count, unsigned threads) {
        return (size_t)count * (kWords * threads * 16u + threads / 8);
    }
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
    // a lane's columns of a row of a matrix
    template <int kA>
    __device__ __forceinline__ void copy(uint32_t n, const T* row, const Cols<kA>& c) const {
        if constexpr (kA == kWide) {
            if (!c.any()) return;
#pragma unroll
            for (uint32_t k = 0; k < kWords; ++k)
                copy_async(word(n, k), row + c.c0 + k * 16 / sizeof(T), 16, kWords > 1);
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c.mask >> j & 1u) copy_async(word(n, j / 4) + 4 * (j % 4), row + c.at(j), 4);
        } else {
            // the words that hold the pairs, or, where the row starts inside a word, those of
            // each pair's first value and the one before it; lane 0 also the word behind the
            // warp's columns. (A word at a row's end may hold two bytes of its neighbour.)
            const uint32_t inside = (uint32_t)reinterpret_cast<uintptr_t>(row) & 2u;
            const char* p = reinterpret_cast<const char*>(row) - inside;
            const uint32_t last = c.cols + (inside ? 1u : 0u);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c.at(2 * k) < last) copy_async(word(n, 0) + 4 * k, p + 2 * c.at(2 * k), 4);
            if ((threadIdx.x & 31u) == 0 && c.c0 + kWarpCols < last)
                copy_async(extra + n * (threads / 8), p + 2 * (c.c0 + kWarpCols), 4);
        }
    }
    // the same of a matrix or of a checkpoint: codes and scales (kNarrow: the warp's 256 codes as
    // words l and l + 32, to be exchanged by get_row)
    template <int kA>
    __device__ __forceinline__ void copy_row(uint32_t n, const Rows& m, bool codes,
                                             const CkptShape& s, uint32_t r,
                                             const Cols<kA>& c) const {
        if (!codes) {
            copy<kA>(n, row_of<T>(m, r), c);
            return;
        }
        const uint8_t* row = row_of<uint8_t>(m, r);
        const uint32_t block = c.c0 >> 7;
        if constexpr (kA == kWide) {
            if (!c.any()) return;
            copy_async(word(n, 0), row + c.c0, 8);
            copy_async(word(n, 0) + 8, ckpt_scales(row, s) + block, 4);
        } else {
            const uint32_t at = (c.c0 & ~(kWarpCols - 1)) + 4u * (threadIdx.x & 31u);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (at + 128u * k < s.code_bytes)
                    copy_async(word(n, 0) + 4 * k, row + at + 128u * k, 4);
                if (block + k < s.blocks)
                    copy_async(word(n, 0) + 8 + 4 * k, ckpt_scales(row, s) + block + k, 4);
            }
        }
    }
    // values of row r, from the slot that copy filled; every lane of the warp calls it
    template <int kA>
    __device__ __forceinline__ Raw<T> get(uint32_t n, const Rows& m, uint32_t r,
                                          const Cols<kA>& c) const {
        Raw<T> v = get(n);
        if constexpr (kA == kNarrow && sizeof(T) == 2) {
            if (reinterpret_cast<uintptr_t>(row_of<T>(m, r)) & 2u) {   // halves of two words
                const uint32_t lane = threadIdx.x & 31u;
                uint32_t behind = 0;
                if (lane == 0)
                    asm volatile("ld.shared.b32 %0, [%1];"
                                 : "=r"(behind)
                                 : "r"(extra + n * (threads / 8))
                                 : "memory");
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t give = lane == 0 ? (k < 3 ? v.w[k < 3 ? k + 1 : 3] : behind) : v.w[k];
                    const uint32_t next = __shfl_sync(0xffffffffu, give, (lane + 1u) & 31u);
                    w[k] = v.w[k] >> 16 | next << 16;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) v.w[k] = w[k];
            }
            if (c.mask != 0xffu) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v.w[k] &= (c.mask >> (2 * k) & 1u ? 0xffffu : 0u) |
                              (c.mask >> (2 * k + 1) & 1u ? 0xffff0000u : 0u);
            }
        }
        return v;
    }
    template <int kA>
    __device__ __forceinline__ Raw<T> get_row(uint32_t n, const Rows& m, bool codes, uint32_t r,
                                              const Cols<kA>& c) const {
        if (!codes) return get<kA>(n, m, r, c);
        Raw<T> v = get(n);
        if constexpr (kA == kWide) {
            v.w[3] = v.w[2];
        } else {
            const uint32_t lane = threadIdx.x & 31u;
            uint32_t pair[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t word = __shfl_sync(0xffffffffu, v.w[k / 2], (16 * k + (lane >> 1)) & 31u);
                pair[k] = word >> 16 * (lane & 1u) & 0xffffu;
                // missing columns: q = 0 (the second of a pair is padding then)
                if (!(c.mask >> (2 * k) & 1u)) pair[k] = 0x8080u;
            }
            v.w[0] = pair[0] | pair[1] << 16;
            v.w[1] = pair[2] | pair[3] << 16;
        }
        return v;
    }
};

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
