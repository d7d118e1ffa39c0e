// The block boundary for sm_100a: y = rs*x + bs*gate*post(h), u = pre(y), and the 8-bit
// checkpoints of y and h.
//
// Bound by HBM: every matrix is read or written once. Eight columns per lane and 256 per warp
// stay in registers from the load to the last use; the sums over a row go through warp shuffles
// and, where several warps share a row (a "team"), one exchange through shared memory each.
//
// A norm's statistics need one sum for RMS (of z^2) and two in turn for LayerNorm (of z, then of
// (z - mean)^2: the difference of large squares would lose the variance of a row with a mean).
#pragma once

#include "zero_join.cuh"

namespace zk {
namespace {

// ---------------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------------
// z - mean (LayerNorm; missing columns stay 0) and 1/deviation of the team's row.
template <int kA, int G>
__device__ __forceinline__ float centre(Team& t, int kind, float eps, float inv_cols,
                                        const Cols<kA> (&c)[G], F8 (&z)[G]) {
    float s[2];
    if (kind == ZERO_NORM_LAYER) {
        s[0] = s[1] = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) s[0] = __fadd_rn(s[0], sum8(z[g]));
        team_sum<2>(t, s);
        const uint64_t m = both(__fmul_rn(s[0], -inv_cols));
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int k = 0; k < 4; ++k) z[g][k] = f2_add(z[g][k], m);
            clear_missing<kA>(c[g], z[g]);
        }
    }
    s[0] = s[1] = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) s[0] = __fadd_rn(s[0], dot8(z[g], z[g]));
    team_sum<2>(t, s);
    return __frsqrt_rn(__fadd_rn(__fmul_rn(s[0], inv_cols), eps));
}

// z*r*w + b; slots n and n + G hold w and b, where there is room (see ForwardShape).
template <typename T, int kA, int G>
__device__ __forceinline__ void scale_shift(const Slots<T>& slots, uint32_t n, const Cols<kA>& c,
                                            float r, const void* w, const void* b, F8& z) {
    constexpr bool kSlots = sizeof(T) * G <= 4;
    F8 wv;
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = f2_mul(z[k], both(r));
    if (w) {
        if (kSlots)
            widen<T>(slots.get(n), wv);
        else
            load_vec<T, kA>(w, 1.0f, c, wv);
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = f2_mul(z[k], wv[k]);
    }
    if (b) {
        if (kSlots)
            widen<T>(slots.get(n + G), wv);
        else
            load_vec<T, kA>(b, 0.0f, c, wv);
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = f2_add(z[k], wv[k]);
    }
}

// Checkpoint of a warp's chunks; 32-bit values one chunk after the other (registers).
template <typename T, int kA, int G>
__device__ __forceinline__ void save_all(uint8_t* row, const CkptShape& s, uint32_t at,
                                         uint32_t stride, uint32_t lane, const Raw<T> (&raw)[G]) {
    if constexpr (sizeof(T) == 2) {
        save_chunks<T, kA, G>(row, s, at, stride, lane, raw);
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const Raw<T> one[1] = {raw[g]};
            save_chunks<T, kA, 1>(row, s, at + g * stride, stride, lane, one);
        }
    }
}

// A CTA has kW warps at most, 8 or 16 (rows of more than 4096 columns; of more than 2048 where
// 32-bit values move singly, one chunk per lane); still wider rows are shared by the CTAs of a
// cluster.

// Rows on the way: many for one chunk per lane. Two 16-bit chunks per lane take one row ahead,
// which with their registers held down (forward_ctas) lets three CTAs fit an SM: 8192 x 4096 bf16 with
// both checkpoints 127 us, 16384 x 2048 fp16 101; with three rows ahead and two CTAs 149 and 107.
// Where two CTAs fit either way, or one (wider rows, rows of any alignment, norms of two kinds, rows
// from checkpoints, a norm alone), one row is as good or better: us with one and with three,
//   4096 x 8192 fp16 51, 53      8192 x 1001 fp16 29, 31       16384 x 2048 mixed norms 76, 77
//   16384 x 2048 from checkpoints 76, 80     norm alone 47, 50    4096 x 8192 with checkpoints 143, 142
template <typename T, int kA, int G>
struct ForwardShape {
    // post_w, post_b, pre_w, pre_b; two 32-bit chunks leave no room for them
    static constexpr uint32_t kVectors = sizeof(T) * G <= 4 ? 4 : 0;
    static constexpr uint32_t kOps = 3;       // x, h, gate
    static constexpr uint32_t kDepth = sizeof(T) == 2 ? (G == 1 ? 4 : 1) : (G == 1 ? 3 : 2);
    static constexpr uint32_t kSlots = (kVectors + kDepth * kOps) * G;
};

// kUse: kAny, or what of a call is known beforehand (without the questions in its rows the kernel
// takes an eighth less time). kUsual: x and h are matrices, y and u are asked for. kNorms: the
// norms are RMS or LayerNorms (kLayer), with one after the block (kPost) or none.
enum Known { kAny = 0, kUsual = 1, kPost = 2, kLayer = 4, kNorms = 8 };

// CTAs an SM holds at least.
template <typename T, int kA, int G, int kW, int kUse>
constexpr int forward_ctas() {
    if (kW == 16) return 1;
    return sizeof(T) == 2 && kA == kWide && (G == 1 || kUse != kAny) ? 3 : 2;
}

template <typename T, int kA, int G, int kW, int kUse>
__global__ void __launch_bounds__(32 * kW, forward_ctas<T, kA, G, kW, kUse>())
    join_kernel(const __grid_constant__ JoinArgs p, uint32_t warps, uint32_t ctas, float inv_cols) {
    using S = ForwardShape<T, kA, G>;
    constexpr bool kAll = kUse != kAny;
    const bool x_codes = !kAll && p.x_codes, h_codes = !kAll && p.h_codes;
    const bool branch = kAll || p.has_branch, has_y = kAll || p.y.p, has_u = kAll || p.u.p;
    constexpr int kind = kUse & kLayer ? ZERO_NORM_LAYER : ZERO_NORM_RMS;
    const int post = !(kUse & kNorms) ? p.post : kUse & kPost ? kind : ZERO_NORM_NONE;
    const int pre = kUse & kNorms ? kind : p.pre;
    __shared__ float part[2][kMaxWarps * kMaxCluster][4];
    const uint32_t warp = threadIdx.x >> 5, team = warp / warps, teams = (blockDim.x >> 5) / warps;
    uint32_t rank = 0;
    if (ctas > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    Team t{part, threadIdx.x & 31u, warp - team * warps, team * warps, warps, ctas, rank, team + 1,
           0};
    const uint32_t first = rank * warps + t.warp, step = warps * ctas;   // this warp's chunks
    const uint32_t cluster = blockIdx.x / ctas, stride = gridDim.x / ctas * teams;
    Cols<kA> c[G];
#pragma unroll
    for (int g = 0; g < G; ++g) c[g] = Cols<kA>(g * step + first, t.lane, p.cols);
    grid_wait();
    if (ctas > 1) cluster_barrier();   // every CTA is there before the first remote store

    extern __shared__ uint4 dynamic[];
    const Slots<T> slots(smem_addr(dynamic), S::kSlots);
    auto fetch = [&](uint32_t r, uint32_t stage) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const uint32_t n = (S::kVectors + stage * S::kOps) * G + g;
            slots.template copy_row<kA>(n, p.x, x_codes, p.ck, r, c[g]);
            if (branch) slots.template copy_row<kA>(n + G, p.h, h_codes, p.ck, r, c[g]);
            if (p.gate_rows)
                slots.template copy<kA>(n + 2 * G, row_of<T>(p.gate, r / p.gate_rows), c[g]);
        }
    };
    // vectors into their slots; columns that do not exist are zeros in every slot
    const void* const vectors[4] = {p.post_w, p.post_b, p.pre_w, p.pre_b};
#pragma unroll
    for (int g = 0; g < G; ++g) {
        if (!c[g].whole())
            for (uint32_t n = g; n < S::kSlots; n += G) slots.clear(n);
#pragma unroll
        for (int n = 0; n < (int)S::kVectors; ++n)
            if (vectors[n]) slots.put(n * G + g, load_raw<T, kA>((const T*)vectors[n], c[g]));
    }
    uint32_t r = cluster * teams + team, ahead = r, stage = 0;
#pragma unroll
    for (uint32_t k = 0; k < S::kDepth; ++k) {
        if (ahead < p.rows) fetch(ahead, k);
        ahead = stride < p.rows - min(ahead, p.rows) ? ahead + stride : p.rows;
        copy_commit();
    }
    for (; r < p.rows; r = stride < p.rows - r ? r + stride : p.rows) {
        Raw<T> rx[G], rh[G], rg[G];
        copy_wait<S::kDepth - 1>();
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const uint32_t n = (S::kVectors + stage * S::kOps) * G + g;
            rx[g] = slots.template get_row<kA>(n, p.x, x_codes, r, c[g]);
            if (branch) rh[g] = slots.template get_row<kA>(n + G, p.h, h_codes, r, c[g]);
            if (p.gate_rows)
                rg[g] = slots.template get<kA>(n + 2 * G, p.gate, r / p.gate_rows, c[g]);
        }
        if (ahead < p.rows) fetch(ahead, stage);   // the next row, into the slots just read
        ahead = stride < p.rows - min(ahead, p.rows) ? ahead + stride : p.rows;
        copy_commit();
        stage = stage + 1 == S::kDepth ? 0 : stage + 1;
        if (p.save_h.p) {
            uint8_t* row = row_of<uint8_t>(p.save_h, r);
            save_all<T, kA, G>(row, p.ck, first, step, t.lane, rh);
            if (first == 0) save_pad(row, p.ck, t.lane);
        }
        F8 y[G];
        if (branch) {
            F8 h[G];
#pragma unroll
            for (int g = 0; g < G; ++g) widen_row<T>(rh[g], h_codes, h[g]);
            if (post != ZERO_NORM_NONE) {
                const float hr = centre<kA, G>(t, post, p.post_eps, inv_cols, c, h);
#pragma unroll
                for (int g = 0; g < G; ++g)
                    scale_shift<T, kA, G>(slots, g, c[g], hr, p.post_w, p.post_b, h[g]);
            }
            if (p.gate_rows) {
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    F8 gv;
                    widen<T>(rg[g], gv);
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[g][k] = f2_mul(h[g][k], gv[k]);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                widen_row<T>(rx[g], x_codes, y[g]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[g][k] = f2_fma(both(p.bs), h[g][k], f2_mul(both(p.rs), y[g][k]));
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                widen_row<T>(rx[g], x_codes, y[g]);
#pragma unroll
                for (int k = 0; k < 4; ++k) y[g][k] = f2_mul(both(p.rs), y[g][k]);
            }
        }
        if (has_y || p.save_y.p) {
            Raw<T> ry[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                ry[g] = narrow<T>(y[g]);
                if (has_y) store_raw<T, kA>(row_of<T>(p.y, r), c[g], ry[g]);
            }
            if (p.save_y.p) {
                uint8_t* row = row_of<uint8_t>(p.save_y, r);
                save_all<T, kA, G>(row, p.ck, first, step, t.lane, ry);
                if (first == 0) save_pad(row, p.ck, t.lane);
            }
        }
        if (has_u) {
            const float yr = centre<kA, G>(t, pre, p.pre_eps, inv_cols, c, y);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                scale_shift<T, kA, G>(slots, 2 * G + g, c[g], yr, p.pre_w, p.pre_b, y[g]);
                store_raw<T, kA>(row_of<T>(p.u, r), c[g], narrow<T>(y[g]));
            }
        }
    }
    if (ctas > 1) cluster_barrier();   // no CTA leaves while another may still store into it
}

template <typename T, int kA, int G, int kW>
cudaError_t run_forward(const JoinArgs& a, const DevInfo& di, cudaStream_t stream) {
    uint32_t warps = (chunks_of(a.cols) + G - 1) / G, ctas = 1;
    while ((warps + ctas - 1) / ctas > (uint32_t)kW) ctas *= 2;
    warps = (warps + ctas - 1) / ctas;
    const uint32_t teams = ctas == 1 ? kW / warps : 1;
    const unsigned threads = 32 * warps * teams;
    auto kernel = join_kernel<T, kA, G, kW, kAny>;
    const bool usual = !a.x_codes && !a.h_codes && a.has_branch && a.y.p && a.u.p;
    if constexpr (kA == kWide) {
        if (usual && (a.post == ZERO_NORM_NONE || a.post == a.pre)) {
            constexpr int kU = kUsual | kNorms;
            const bool layer = a.pre == ZERO_NORM_LAYER;
            if (a.post == ZERO_NORM_NONE)
                kernel = layer ? join_kernel<T, kA, G, kW, kU | kLayer>
                               : join_kernel<T, kA, G, kW, kU>;
            else
                kernel = layer ? join_kernel<T, kA, G, kW, kU | kPost | kLayer>
                               : join_kernel<T, kA, G, kW, kU | kPost>;
        }
    } else if (usual) {
        kernel = join_kernel<T, kA, G, kW, kUsual>;
    }
    constexpr uint32_t kSlots = ForwardShape<T, kA, G>::kSlots;
    const size_t smem = Slots<T>::bytes(kSlots, threads);
    int per_sm = 1;
    const cudaError_t e = resident(kernel, di.dev, threads, smem,
                                   Slots<T>::bytes(kSlots, 32 * kW),
                                   &per_sm);
    if (e != cudaSuccess) return e;
    const uint64_t clusters = ((uint64_t)a.rows + teams - 1) / teams;
    const uint64_t cap = (uint64_t)di.sms * per_sm / ctas;
    return launch_clusters(kernel, (unsigned)(clusters < cap ? clusters : cap), ctas, threads, smem,
                           stream, a, warps, ctas, 1.0f / (float)a.cols);
}

// Chunks per lane: two, so that the work per row that does not grow with the columns is shared by
// more of them (16384 x 2048 fp16 with both checkpoints: 101 us, with one 131); one where a row
// has three or fewer, where it has 32-bit values that move singly, or where there are too few rows
// to fill the device anyway.
template <typename T, int kA>
cudaError_t run_forward_any(const JoinArgs& a, cudaStream_t stream) {
    DevInfo di;
    const cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    const uint32_t chunks = chunks_of(a.cols);
    constexpr bool kOne = sizeof(T) == 4 && kA == kNarrow;
    if (chunks <= 3 || (chunks <= 8 && (kOne || a.rows <= (uint32_t)di.sms)))
        return run_forward<T, kA, 1, 8>(a, di, stream);
    if constexpr (kOne) {
        return run_forward<T, kA, 1, 16>(a, di, stream);
    } else {
        if (chunks <= 16) return run_forward<T, kA, 2, 8>(a, di, stream);
        return run_forward<T, kA, 2, 16>(a, di, stream);
    }
}

template <typename T>
cudaError_t run_join(const JoinArgs& a, cudaStream_t stream) {
    return all_access<T>(a) == kWide ? run_forward_any<T, kWide>(a, stream)
                                     : run_forward_any<T, kNarrow>(a, stream);
}

}  // namespace
}  // namespace zk
