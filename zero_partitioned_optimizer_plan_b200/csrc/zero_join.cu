// The block boundary for sm_100a: y = rs*x + bs*gate*post(h), u = pre(y), and the 8-bit
// checkpoints of y and h.
//
// Bound by HBM: every matrix is read or written once. Eight columns per lane and 256 per warp
// stay in registers from the load to the last use; the sums over a row go through warp shuffles
// and, where several warps share a row (a "team"), one exchange through shared memory each.
//
// A norm's statistics need one sum for RMS (of z^2) and two in turn for LayerNorm (of z, then of
// (z - mean)^2: the difference of large squares would lose the variance of a row with a mean).
#include "zero_join.cuh"

namespace zk {
namespace {

// ---------------------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------------------
// z - mean (LayerNorm; missing columns stay 0) and 1/deviation of the team's row.
template <bool kVec, int G>
__device__ __forceinline__ float centre(Team& t, int kind, float eps, float inv_cols,
                                        const Cols<kVec> (&c)[G], F8 (&z)[G]) {
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
            clear_missing<kVec>(c[g], z[g]);
        }
    }
    s[0] = s[1] = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) s[0] = __fadd_rn(s[0], dot8(z[g], z[g]));
    team_sum<2>(t, s);
    return __frsqrt_rn(__fadd_rn(__fmul_rn(s[0], inv_cols), eps));
}

// z*r*w + b.
template <typename T, bool kVec>
__device__ __forceinline__ void scale_shift(const Cols<kVec>& c, float r, const void* w,
                                            const void* b, F8& z) {
    F8 wv;
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = f2_mul(z[k], both(r));
    if (w) {
        load_vec<T, kVec>(w, 1.0f, c, wv);
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = f2_mul(z[k], wv[k]);
    }
    if (b) {
        load_vec<T, kVec>(b, 0.0f, c, wv);
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = f2_add(z[k], wv[k]);
    }
}

// Checkpoint of a warp's chunks; many or 32-bit values one chunk after the other (registers).
template <typename T, bool kVec, int G>
__device__ __forceinline__ void save_all(uint8_t* row, const CkptShape& s, uint32_t at,
                                         uint32_t stride, uint32_t lane, const Raw<T> (&raw)[G]) {
    if constexpr (sizeof(T) == 2 && G <= 2) {
        save_chunks<T, kVec, G>(row, s, at, stride, lane, raw);
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const Raw<T> one[1] = {raw[g]};
            save_chunks<T, kVec, 1>(row, s, at + g * stride, stride, lane, one);
        }
    }
}

// Warps of a CTA at most. Four chunks of 32-bit values per lane need 255 registers; rows beyond
// eight such warps are shared by the CTAs of a cluster.
template <typename T, int G>
constexpr int forward_warps() { return sizeof(T) * G == 16 ? 8 : kMaxWarps; }

template <typename T, bool kVec, int G>
__global__ void __launch_bounds__(32 * forward_warps<T, G>(), 1)
    join_kernel(const __grid_constant__ JoinArgs p, uint32_t warps, uint32_t ctas, float inv_cols) {
    __shared__ float part[2][kMaxWarps * kMaxCluster][4];
    const uint32_t warp = threadIdx.x >> 5, team = warp / warps, teams = (blockDim.x >> 5) / warps;
    uint32_t rank = 0;
    if (ctas > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    Team t{part, threadIdx.x & 31u, warp - team * warps, team * warps, warps, ctas, rank, team + 1,
           0};
    const uint32_t first = rank * warps + t.warp, step = warps * ctas;   // this warp's chunks
    const uint64_t cluster = blockIdx.x / ctas, clusters = gridDim.x / ctas;
    Cols<kVec> c[G];
#pragma unroll
    for (int g = 0; g < G; ++g) c[g] = Cols<kVec>(g * step + first, t.lane, p.cols);
    grid_wait();
    if (ctas > 1) team_barrier(t);   // every CTA is there before the first remote store
    for (uint64_t r = cluster * teams + team; r < p.rows; r += clusters * teams) {
        Raw<T> rx[G], rh[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            rx[g] = load_row<T, kVec>(p.x, p.x_ckpt, p.ck, r, c[g]);
            if (p.has_branch) rh[g] = load_row<T, kVec>(p.h, p.h_ckpt, p.ck, r, c[g]);
        }
        if (p.save_h) {
            uint8_t* row = p.save_h + r * p.ck.row_bytes;
            save_all<T, kVec, G>(row, p.ck, first, step, t.lane, rh);
            if (first == 0) save_pad(row, p.ck, t.lane);
        }
        F8 y[G];
        if (p.has_branch) {
            F8 h[G];
#pragma unroll
            for (int g = 0; g < G; ++g) widen_row<T>(rh[g], p.h_ckpt != nullptr, h[g]);
            if (p.post != ZERO_NORM_NONE) {
                const float hr = centre<kVec, G>(t, p.post, p.post_eps, inv_cols, c, h);
#pragma unroll
                for (int g = 0; g < G; ++g)
                    scale_shift<T, kVec>(c[g], hr, p.post_w, p.post_b, h[g]);
            }
            if (p.gate_rows) {
                const T* gate = (const T*)p.gate.p + row_over(r, p.gate_rows) * p.gate.ld;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    F8 gv;
                    widen<T>(load_raw<T, kVec>(gate, c[g]), gv);
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[g][k] = f2_mul(h[g][k], gv[k]);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                widen_row<T>(rx[g], p.x_ckpt != nullptr, y[g]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[g][k] = f2_fma(both(p.bs), h[g][k], f2_mul(both(p.rs), y[g][k]));
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                widen_row<T>(rx[g], p.x_ckpt != nullptr, y[g]);
#pragma unroll
                for (int k = 0; k < 4; ++k) y[g][k] = f2_mul(both(p.rs), y[g][k]);
            }
        }
        if (p.y.p || p.save_y) {
            Raw<T> ry[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                ry[g] = narrow<T>(y[g]);
                if (p.y.p) store_raw<T, kVec>((T*)p.y.p + r * p.y.ld, c[g], ry[g]);
            }
            if (p.save_y) {
                uint8_t* row = p.save_y + r * p.ck.row_bytes;
#pragma unroll
                for (int g = 0; g < G; ++g)   // a post bias may have filled missing columns
                    if (c[g].mask != 0xffu) {
                        F8 z;
                        widen<T>(ry[g], z);
                        clear_missing<kVec>(c[g], z);
                        ry[g] = narrow<T>(z);
                    }
                save_all<T, kVec, G>(row, p.ck, first, step, t.lane, ry);
                if (first == 0) save_pad(row, p.ck, t.lane);
            }
        }
        if (p.u.p) {
            const float yr = centre<kVec, G>(t, p.pre, p.pre_eps, inv_cols, c, y);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                scale_shift<T, kVec>(c[g], yr, p.pre_w, p.pre_b, y[g]);
                store_raw<T, kVec>((T*)p.u.p + r * p.u.ld, c[g], narrow<T>(y[g]));
            }
        }
    }
    if (ctas > 1) team_barrier(t);   // no CTA leaves while another may still store into it
}

template <typename T, bool kVec, int G>
cudaError_t run_forward(const JoinArgs& a, uint32_t warps, int sms, cudaStream_t stream) {
    uint32_t ctas = 1;
    while ((warps + ctas - 1) / ctas > (uint32_t)forward_warps<T, G>()) ctas *= 2;
    warps = (warps + ctas - 1) / ctas;
    const uint32_t teams = ctas == 1 && warps < 4 ? 4 / warps : 1;
    const uint64_t clusters = (a.rows + teams - 1) / teams, cap = (uint64_t)sms * 32 / ctas;
    return launch_clusters(join_kernel<T, kVec, G>,
                           (unsigned)(clusters < cap ? clusters : cap), ctas, 32 * warps * teams,
                           stream, a, warps, ctas, 1.0f / (float)a.cols);
}

// Warps and chunks per lane of a row: as few warps as registers allow (one up to 1024 columns:
// no exchange between warps), but one chunk per warp where there are too few rows to fill the
// device anyway.
template <typename T, bool kVec>
cudaError_t run_forward_any(const JoinArgs& a, cudaStream_t stream) {
    DevInfo di;
    const cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    const uint32_t chunks = chunks_of(a.cols);
    if (chunks <= kMaxWarps && a.rows <= (uint64_t)di.sms)
        return run_forward<T, kVec, 1>(a, chunks, di.sms, stream);
    if (chunks == 1) return run_forward<T, kVec, 1>(a, 1, di.sms, stream);
    if (chunks == 2) return run_forward<T, kVec, 2>(a, 1, di.sms, stream);
    if (chunks <= 4) return run_forward<T, kVec, 4>(a, 1, di.sms, stream);
    if (chunks <= 16) return run_forward<T, kVec, 2>(a, (chunks + 1) / 2, di.sms, stream);
    return run_forward<T, kVec, 4>(a, (chunks + 3) / 4, di.sms, stream);
}

template <typename T>
cudaError_t run_join(const JoinArgs& a, cudaStream_t stream) {
    return all_aligned<T>(a) ? run_forward_any<T, true>(a, stream)
                             : run_forward_any<T, false>(a, stream);
}

}  // namespace

cudaError_t launch_join(const JoinArgs& a, int dtype, cudaStream_t stream) {
    return dtype == ZERO_F16    ? run_join<__half>(a, stream)
           : dtype == ZERO_BF16 ? run_join<bf16>(a, stream)
                                : run_join<float>(a, stream);
}

}  // namespace zk
