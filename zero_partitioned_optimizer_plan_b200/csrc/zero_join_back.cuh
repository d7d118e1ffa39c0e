// Gradient of the block boundary for sm_100a (zero_join_forward.cuh: the forward pass).
//
// Bound by HBM: dy, du and the saved y and h (bytes, where they are checkpoints) are read once,
// dx and dh written once. Persistent teams of warps walk their rows with the next row's loads in
// flight and keep the column sums (of the weights', biases' and gate's gradients) in registers;
// the teams of a CTA are added through shared memory, the CTAs by a second kernel, always in the
// same order. Rows wider than a CTA's warps are shared by the CTAs of a cluster, whose sums meet
// in distributed shared memory.
//
// The statistics are computed again from the saved rows. The sums of g and g*(z - mean) that a
// norm's gradient needs ride along with its second statistic, so a LayerNorm before the next
// block costs two exchanges per row (RMS: one) and a norm after the block one more.
#pragma once

#include "zero_join.cuh"

namespace zk {
namespace {

constexpr int kMaxParts = 148;         // clusters that leave partial column sums

// ---------------------------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------------------------
// How a call's rows and columns are dealt out. A unit is a run of rows within one gate row (all
// rows where no gate gradient is asked for): `parts` units of part_rows rows per gate row.
struct BackGeom {
    uint32_t warps, ctas, teams;   // warps of a CTA per row, CTAs per row, rows a CTA has in hand
    uint32_t clusters;
    uint32_t group_rows, parts, part_rows, units;
    float inv_cols;
};

// lanes_of: chunks of 256 columns per lane (G); most_warps: warps of a CTA.
BackGeom back_geom(uint32_t rows, uint64_t cols, uint32_t group_rows, uint32_t lane_chunks,
                   uint32_t most_warps, uint32_t sms) {
    BackGeom g = {};
    const uint32_t pieces = (chunks_of(cols) + lane_chunks - 1) / lane_chunks;
    g.ctas = 1;
    while ((pieces + g.ctas - 1) / g.ctas > most_warps) g.ctas *= 2;
    g.warps = (pieces + g.ctas - 1) / g.ctas;
    g.teams = g.ctas > 1 ? 1 : most_warps / g.warps;
    uint32_t clusters = sms / g.ctas;
    if (clusters > (uint32_t)kMaxParts) clusters = kMaxParts;
    const uint32_t useful = (rows + g.teams - 1) / g.teams;
    if (clusters > useful) clusters = useful;
    if (clusters < 1) clusters = 1;
    g.clusters = clusters;
    g.group_rows = group_rows && group_rows < rows ? group_rows : rows;
    if (g.group_rows) {
        const uint32_t groups = (rows + g.group_rows - 1) / g.group_rows;
        uint32_t parts = g.clusters * g.teams / groups;
        if (parts < 1) parts = 1;
        g.part_rows = (g.group_rows + parts - 1) / parts;
        g.parts = (g.group_rows + g.part_rows - 1) / g.part_rows;
        g.units = groups * g.parts;
    }
    g.inv_cols = 1.0f / (float)cols;
    return g;
}

// The shape of one instantiation. A lane holds G chunks (256 columns per warp) of each matrix and
// the column sums of up to four vectors in registers: one 16-bit chunk takes 128 of them (16 warps
// per SM), two without a norm after the block, or a 32-bit one, 168 (12 warps).
template <typename T, int kA, bool kPost, bool kGate, int G>
struct BackShape {
    static constexpr bool kHeavy = kPost || kGate;
    static constexpr int kWarps = sizeof(T) == 4 || G == 2 ? 12 : 16;
    static constexpr uint32_t kOps = kHeavy ? 5 : 4;       // y, du, dy, gate, h
    static constexpr uint32_t kVectors = kHeavy ? 3 : 1;   // pre_w, post_w, post_b
    static constexpr uint32_t kDepth = sizeof(T) == 4 ? 2 : G == 2 ? 3 : 4;   // rows on the way
    static constexpr uint32_t kSlots = (kVectors + kDepth * kOps) * G;
    static constexpr size_t kBytes = (size_t)kSlots * (8 * sizeof(T) * 32 + 4) * kWarps +
                                     (size_t)(kPost && kGate ? 2 * G : 1) * kWarps * 1024 + 4096;
    static_assert(kBytes <= 227 * 1024, "shared memory of one CTA");
};

// A team's place in its rows; row == end: no more.
struct Walk {
    uint32_t unit, row, end;
    __device__ __forceinline__ explicit Walk(uint32_t first) : unit(first), row(0), end(0) {}
    __device__ __forceinline__ void open(const BackGeom& g, uint32_t rows) {
        for (; unit < g.units; unit += g.clusters * g.teams) {
            const uint32_t group = unit / g.parts, first = group * g.group_rows;
            const uint32_t last = first + min(g.group_rows, rows - first);
            row = first + (unit - group * g.parts) * g.part_rows;
            end = row + g.part_rows < last ? row + g.part_rows : last;
            if (row < end) return;
        }
        row = end = 0;
    }
    // to the next row; true if it is another unit's (or none)
    __device__ __forceinline__ bool next(const BackGeom& g, uint32_t rows) {
        if (++row < end) return false;
        unit += g.clusters * g.teams;
        open(g, rows);
        return true;
    }
};

template <typename T>
__device__ __forceinline__ void put_sum(void* p, uint64_t at, float s, bool add) {
    T* d = (T*)p + at;
    *d = from_f<T>(add ? __fadd_rn(to_f(*d), s) : s);
}

// The partial sums of the vector gradients in the workspace: [cluster][4][cols], then the parts
// of the gate's gradient: [unit][cols].
__host__ __device__ __forceinline__ uint64_t vector_partials(uint32_t cols) {
    return (uint64_t)kMaxParts * 4 * cols;
}

// kUse: kAny, or what of a call is known beforehand. kUsual: every gradient matrix (dy, du in, dx,
// dh out) is there, the saved rows are all checkpoints (kCodes) or all matrices. kNorms: the norms
// are all LayerNorms (kLayer) or all RMS, and there is a gate exactly if its gradient is asked
// for. Without the questions in its rows the kernel takes a fifth less time (16384 x 2048 fp16:
// 113 us with them, 95 without the first, 89 without both).
enum Use { kAny = 0, kUsual = 1, kCodes = 2, kLayer = 4, kNorms = 8 };

template <typename T, int kA, bool kPost, bool kGate, int G, int kUse>
__global__ void __launch_bounds__(32 * BackShape<T, kA, kPost, kGate, G>::kWarps, 1)
    join_back_kernel(const __grid_constant__ JoinArgs p, const __grid_constant__ BackGeom g,
                     float* ws) {
    using S = BackShape<T, kA, kPost, kGate, G>;
    // With a norm after the block and a gate gradient, sum_qw and sum_qb are those of one gate row
    // without its gate: bs*gy*hh and bs*gy. Where the gate row ends they give its gradient,
    // w*sum_qw + b*sum_qb, and, multiplied by the gate, go into the norm's own sums in shared
    // memory. With a gate gradient alone, sum_qw is bs*gy*h.
    constexpr bool kBoth = kPost && kGate;
    __shared__ float part[2][kMaxWarps * kMaxCluster][4];
    // column sums beside the registers; at the end the teams' sums meet in the first of them
    __shared__ float held[kBoth ? 2 : 1][kBoth ? G : 1][S::kWarps][8][32];
    const uint32_t warp = threadIdx.x >> 5, team = warp / g.warps;
    uint32_t rank = 0;
    if (g.ctas > 1) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const uint32_t cluster = g.ctas > 1 ? blockIdx.x / g.ctas : blockIdx.x;
    Team t{part, threadIdx.x & 31u, warp - team * g.warps, team * g.warps, g.warps, g.ctas, rank,
           team + 1, 0};
    Cols<kA> c[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
        c[i] = Cols<kA>((i * g.ctas + rank) * g.warps + t.warp, t.lane, p.cols);
    const bool has_du = kUse != kAny || p.du.p, has_dy = kUse != kAny || p.dy.p;
    const bool has_dx = kUse != kAny || p.dx.p, has_dh = kUse != kAny || p.dh.p;
    const bool y_codes = kUse == kAny ? p.x_codes : (kUse & kCodes) != 0;
    const bool h_codes = kUse == kAny ? p.h_codes : (kUse & kCodes) != 0;
    const bool has_gate = kUse & kNorms ? kGate : p.gate_rows != 0;
    const bool pre_layer = kUse & kNorms ? (kUse & kLayer) != 0 : has_du && p.pre == ZERO_NORM_LAYER;
    const bool post_layer =
        kPost && (kUse & kNorms ? (kUse & kLayer) != 0 : p.post == ZERO_NORM_LAYER);
    F8 sum_pw[G] = {}, sum_pb[G] = {}, sum_qw[G] = {}, sum_qb[G] = {};
    if (kBoth) {
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                held[0][i][warp][j][t.lane] = held[kBoth][i][warp][j][t.lane] = 0.0f;
    }
    grid_wait();
    if (g.ctas > 1) cluster_barrier();   // every CTA of the cluster is there before the first store

    // the vectors, and rows on their way, in this thread's slots of shared memory
    extern __shared__ uint4 dynamic[];
    const Slots<T> slots(smem_addr(dynamic), S::kSlots);
    auto fetch = [&](uint32_t r, uint32_t stage) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const uint32_t n = S::kVectors * G + stage * S::kOps * G + i;
            if (has_du) {
                slots.template copy_row<kA>(n, p.x, y_codes, p.ck, r, c[i]);
                slots.template copy<kA>(n + G, row_of<T>(p.du, r), c[i]);
            }
            if (has_dy) slots.template copy<kA>(n + 2 * G, row_of<T>(p.dy, r), c[i]);
            if (has_gate)
                slots.template copy<kA>(n + 3 * G, row_of<T>(p.gate, r / p.gate_rows), c[i]);
            if (kPost || kGate)
                slots.template copy_row<kA>(n + 4 * G, p.h, h_codes, p.ck, r, c[i]);
        }
    };
    auto vector = [&](int n, int i, const void* v, float none, F8& out) {
        if (v) {
            widen<T>(slots.get(n * G + i), out);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) out[k] = both(none);
        }
    };
    {
        const void* const vectors[3] = {p.pre_w, p.post_w, p.post_b};
#pragma unroll
        for (int i = 0; i < G; ++i) {
            if (!c[i].whole())
                for (uint32_t n = i; n < S::kSlots; n += G) slots.clear(n);
#pragma unroll
            for (int n = 0; n < (int)S::kVectors; ++n)
                if (vectors[n]) slots.put(n * G + i, load_raw<T, kA>((const T*)vectors[n], c[i]));
        }
    }
    Walk in(cluster * g.teams + team), at = in;
    in.open(g, p.rows);
    at.open(g, p.rows);
#pragma unroll
    for (uint32_t k = 0; k < S::kDepth; ++k) {
        if (in.row < in.end) {
            fetch(in.row, k);
            in.next(g, p.rows);
        }
        copy_commit();
    }
    uint32_t stage = 0;
    while (at.row < at.end) {
        const uint32_t r = at.row, unit = at.unit;
        F8 y[G], h[G], du[G], gy[G], gate[G];
        copy_wait<S::kDepth - 1>();
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const uint32_t n = S::kVectors * G + stage * S::kOps * G + i;
            if (has_du) {
                widen_row<T>(slots.template get_row<kA>(n, p.x, y_codes, r, c[i]), y_codes, y[i]);
                widen<T>(slots.template get<kA>(n + G, p.du, r, c[i]), du[i]);
            }
            if (has_dy) widen<T>(slots.template get<kA>(n + 2 * G, p.dy, r, c[i]), gy[i]);
            if (has_gate)
                widen<T>(slots.template get<kA>(n + 3 * G, p.gate, r / p.gate_rows, c[i]), gate[i]);
            if (kPost || kGate)
                widen_row<T>(slots.template get_row<kA>(n + 4 * G, p.h, h_codes, r, c[i]), h_codes,
                             h[i]);
            if (!has_dy) {
#pragma unroll
                for (int k = 0; k < 4; ++k) gy[i][k] = 0;
            }
        }
        const bool turn = at.next(g, p.rows);
        if (in.row < in.end) {   // into the slots just read
            fetch(in.row, stage);
            in.next(g, p.rows);
        }
        copy_commit();
        stage = stage + 1 == S::kDepth ? 0 : stage + 1;

        if (pre_layer || post_layer) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < G; ++i) {
                if (pre_layer) s[0] = __fadd_rn(s[0], sum8(y[i]));
                if (post_layer) s[1] = __fadd_rn(s[1], sum8(h[i]));
            }
            team_sum<2>(t, s);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                if (pre_layer) {
                    const uint64_t m = both(__fmul_rn(s[0], -g.inv_cols));
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[i][k] = f2_add(y[i][k], m);
                    clear_missing<kA>(c[i], y[i]);
                }
                if (post_layer) {
                    const uint64_t m = both(__fmul_rn(s[1], -g.inv_cols));
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[i][k] = f2_add(h[i][k], m);
                    clear_missing<kA>(c[i], h[i]);
                }
            }
        }
        float hr = 1.0f;
        if (has_du || kPost) {
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            F8 gu[G];
#pragma unroll
            for (int i = 0; i < G; ++i) {
                if (has_du) {
                    F8 w;
                    vector(0, i, p.pre_w, 1.0f, w);
#pragma unroll
                    for (int k = 0; k < 4; ++k) gu[i][k] = f2_mul(du[i][k], w[k]);
                    s[0] = __fadd_rn(s[0], dot8(y[i], y[i]));
                    s[1] = __fadd_rn(s[1], sum8(gu[i]));
                    s[2] = __fadd_rn(s[2], dot8(gu[i], y[i]));
                }
                if (kPost) s[3] = __fadd_rn(s[3], dot8(h[i], h[i]));
            }
            team_sum<4>(t, s);
            if (kPost)
                hr = __frsqrt_rn(__fadd_rn(__fmul_rn(s[3], g.inv_cols), p.post_eps));
            if (has_du) {
                const float yr = __frsqrt_rn(__fadd_rn(__fmul_rn(s[0], g.inv_cols), p.pre_eps));
                const float m1 = pre_layer ? __fmul_rn(s[1], g.inv_cols) : 0.0f;
                const float m2 = __fmul_rn(__fmul_rn(s[2], yr), g.inv_cols);
#pragma unroll
                for (int i = 0; i < G; ++i) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t yh = f2_mul(y[i][k], both(yr));
                        sum_pw[i][k] = f2_fma(du[i][k], yh, sum_pw[i][k]);
                        sum_pb[i][k] = f2_add(sum_pb[i][k], du[i][k]);
                        const uint64_t d = f2_fma(yh, both(-m2), f2_add(gu[i][k], both(-m1)));
                        gy[i][k] = f2_fma(both(yr), d, gy[i][k]);
                    }
                    if (pre_layer) clear_missing<kA>(c[i], gy[i]);
                }
            }
        }
        if (has_dx) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                F8 dx;
#pragma unroll
                for (int k = 0; k < 4; ++k) dx[k] = f2_mul(both(p.rs), gy[i][k]);
                store_raw<T, kA>(row_of<T>(p.dx, r), c[i], narrow<T>(dx));
            }
        }
        if (has_dh || (p.has_branch && (kPost || kGate))) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < G; ++i) {   // gy becomes t = bs*gate*gy
                F8 v;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    gy[i][k] = f2_mul(both(p.bs), gy[i][k]);
                    if (kPost) h[i][k] = f2_mul(h[i][k], both(hr));
                }
                if (kGate) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        sum_qw[i][k] = f2_fma(gy[i][k], h[i][k], sum_qw[i][k]);
                        if (kPost) sum_qb[i][k] = f2_add(sum_qb[i][k], gy[i][k]);
                    }
                }
                if (has_gate) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) gy[i][k] = f2_mul(gy[i][k], gate[i][k]);
                }
                if (kPost) {
                    vector(1, i, p.post_w, 1.0f, v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (!kGate) {
                            sum_qw[i][k] = f2_fma(gy[i][k], h[i][k], sum_qw[i][k]);
                            sum_qb[i][k] = f2_add(sum_qb[i][k], gy[i][k]);
                        }
                        gy[i][k] = f2_mul(gy[i][k], v[k]);
                    }
                    s[0] = __fadd_rn(s[0], sum8(gy[i]));
                    s[1] = __fadd_rn(s[1], dot8(gy[i], h[i]));
                }
            }
            if (has_dh) {
                if (kPost) {
                    team_sum<2>(t, s);
                    const float n1 = post_layer ? __fmul_rn(s[0], g.inv_cols) : 0.0f;
                    const float n2 = __fmul_rn(s[1], g.inv_cols);
#pragma unroll
                    for (int i = 0; i < G; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            gy[i][k] = f2_mul(both(hr), f2_fma(h[i][k], both(-n2),
                                                               f2_add(gy[i][k], both(-n1))));
                }
#pragma unroll
                for (int i = 0; i < G; ++i)
                    store_raw<T, kA>(row_of<T>(p.dh, r), c[i], narrow<T>(gy[i]));
            }
        }
        if (kGate && turn) {   // the unit's part of its gate row's gradient
            const uint32_t group = unit / g.parts;
#pragma unroll
            for (int i = 0; i < G; ++i) {
                F8 part_g;
                if (kPost) {
                    F8 w, b;
                    vector(1, i, p.post_w, 1.0f, w);
                    vector(2, i, p.post_b, 0.0f, b);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        part_g[k] = f2_fma(sum_qw[i][k], w[k], f2_mul(sum_qb[i][k], b[k]));
                        float* qw = &held[0][i][warp][2 * k][t.lane];
                        float* qb = &held[kBoth][i][warp][2 * k][t.lane];
                        f2_unpack(f2_fma(sum_qw[i][k], gate[i][k], f2_pack(qw[0], qw[32])), qw[0],
                                  qw[32]);
                        f2_unpack(f2_fma(sum_qb[i][k], gate[i][k], f2_pack(qb[0], qb[32])), qb[0],
                                  qb[32]);
                        sum_qw[i][k] = sum_qb[i][k] = 0;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        part_g[k] = sum_qw[i][k];
                        sum_qw[i][k] = 0;
                    }
                }
                float f[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) f2_unpack(part_g[k], f[2 * k], f[2 * k + 1]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (!(c[i].mask >> j & 1u)) continue;
                    if (g.parts > 1)
                        ws[vector_partials(p.cols) + (uint64_t)unit * p.cols + c[i].at(j)] = f[j];
                    else
                        put_sum<T>(row_of<T>(p.dgate, group), c[i].at(j), f[j],
                                   p.accumulate & ZERO_ACC_GATE);
                }
            }
        }
    }
    if (ws) grid_launch_next();
    // the teams' column sums, added in order; to the workspace, or as they are if one CTA had all
    void* const outs[4] = {p.dpost_w, p.dpost_b, p.dpre_w, p.dpre_b};
#pragma unroll
    for (int k = 0; k < 4; ++k) {   // (held[0] holds the first one until it is done)
        if (!outs[k]) continue;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const bool there = kBoth && k < 2;   // already in shared memory
            float(*comb)[8][32] = there ? held[k][i] : held[0][0];
            __syncthreads();
            if (!there) {
                const F8& s = k == 0 ? sum_qw[i] : k == 1 ? sum_qb[i] : k == 2 ? sum_pw[i] : sum_pb[i];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f2_unpack(s[j], comb[warp][2 * j][t.lane], comb[warp][2 * j + 1][t.lane]);
                __syncthreads();
            }
            if (team != 0) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!(c[i].mask >> j & 1u)) continue;
                float v = 0.0f;
                for (uint32_t n = 0; n < g.teams; ++n)
                    v = __fadd_rn(v, comb[n * g.warps + t.warp][j][t.lane]);
                if (g.clusters > 1)
                    ws[((uint64_t)cluster * 4 + k) * p.cols + c[i].at(j)] = v;
                else
                    put_sum<T>(outs[k], c[i].at(j), v, p.accumulate & ZERO_ACC_PARAMS);
            }
        }
    }
    if (g.ctas > 1) cluster_barrier();   // no CTA leaves while another may still store into it
}

// Column sums from the workspace: 32 columns by 16 rows of partial sums per CTA. blockIdx.y < 4:
// a vector's (if they are split); above, a gate row's. Without partial sums (no rows): zeros.
constexpr int kSumRows = 16;

template <typename T>
__global__ void __launch_bounds__(32 * kSumRows)
    join_vectors_kernel(const __grid_constant__ JoinArgs p, const __grid_constant__ BackGeom g,
                        bool vectors, const float* ws) {
    __shared__ float part[kSumRows][32];
    grid_wait();
    const uint32_t cx = threadIdx.x & 31u, ry = threadIdx.x >> 5, c = blockIdx.x * 32u + cx;
    const uint32_t k = blockIdx.y;
    void* out = k == 0 ? p.dpost_w : k == 1 ? p.dpost_b : k == 2 ? p.dpre_w : k == 3 ? p.dpre_b
                                                                          : p.dgate.p;
    if (!out || (k < 4 && !vectors)) return;
    const uint64_t stride = k < 4 ? 4ull * p.cols : p.cols;
    const float* src = k < 4 ? ws + (uint64_t)k * p.cols
                             : ws + vector_partials(p.cols) + (uint64_t)(k - 4) * g.parts * p.cols;
    uint32_t n = p.rows ? g.clusters : 0;
    if (k >= 4) {   // the last gate row may be shorter: parts that have rows
        const uint32_t left = p.rows - (k - 4) * g.group_rows;
        n = ((left < g.group_rows ? left : g.group_rows) + g.part_rows - 1) / g.part_rows;
    }
    float s = 0.0f;
    if (c < p.cols) {
#pragma unroll 4
        for (uint32_t i = ry; i < n; i += kSumRows) s = __fadd_rn(s, src[i * stride + c]);
    }
    part[ry][cx] = s;
    __syncthreads();
    if (ry != 0 || c >= p.cols) return;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) v = __fadd_rn(v, part[i][cx]);
    if (k < 4)
        put_sum<T>(out, c, v, p.accumulate & ZERO_ACC_PARAMS);
    else
        put_sum<T>(row_of<T>(p.dgate, k - 4), c, v, p.accumulate & ZERO_ACC_GATE);
}

template <typename T, int kA, bool kPost, bool kGate, int G, int kUse>
cudaError_t run_back_use(const JoinArgs& a, const DevInfo& di, float* ws, BackGeom* geom,
                            cudaStream_t stream) {
    using S = BackShape<T, kA, kPost, kGate, G>;
    const BackGeom g = back_geom(a.rows, a.cols, a.dgate.p ? a.gate_rows : 0, G, S::kWarps,
                                 (uint32_t)di.sms);
    *geom = g;
    if (a.rows == 0) return cudaSuccess;
    auto kernel = join_back_kernel<T, kA, kPost, kGate, G, kUse>;
    const unsigned threads = 32 * g.warps * g.teams;
    const size_t smem = Slots<T>::bytes(S::kSlots, threads);
    int ctas = 1;
    const cudaError_t e = resident(kernel, di.dev, threads, smem, Slots<T>::bytes(S::kSlots, 32 * S::kWarps),
                                   &ctas);
    if (e != cudaSuccess) return e;
    // a second kernel follows exactly if partial sums are left in the workspace
    const bool used = ((a.dpost_w || a.dpost_b || a.dpre_w || a.dpre_b) && g.clusters > 1) ||
                      (a.dgate.p && g.parts > 1);
    return launch_clusters(kernel, g.clusters, g.ctas, threads, smem, stream, a, g,
                           used ? ws : (float*)nullptr);
}

template <typename T, int kA, bool kPost, bool kGate, int G>
cudaError_t run_back_kernel(const JoinArgs& a, const DevInfo& di, float* ws, BackGeom* g,
                            cudaStream_t stream) {
    const bool h = kPost || kGate;
    const bool usual = a.dy.p && a.du.p && a.dx.p && a.dh.p && (!h || a.h_codes == a.x_codes);
    const bool norms = (!kPost || a.post == a.pre) && (kGate || !a.gate.p);
    const bool layer = a.pre == ZERO_NORM_LAYER;
    constexpr int kM = kUsual, kC = kUsual | kCodes;
    if constexpr (kA == kWide) {
        if (usual && norms && !a.x_codes)
            return layer ? run_back_use<T, kA, kPost, kGate, G, kM | kNorms | kLayer>(a, di, ws, g, stream)
                         : run_back_use<T, kA, kPost, kGate, G, kM | kNorms>(a, di, ws, g, stream);
        if constexpr (sizeof(T) == 2) {   // (32-bit activations are rarely kept in 8 bits)
            if (usual && norms)
                return layer ? run_back_use<T, kA, kPost, kGate, G, kC | kNorms | kLayer>(a, di, ws, g, stream)
                             : run_back_use<T, kA, kPost, kGate, G, kC | kNorms>(a, di, ws, g, stream);
        }
    } else if (usual) {
        if (!a.x_codes) return run_back_use<T, kA, kPost, kGate, G, kM>(a, di, ws, g, stream);
        if constexpr (sizeof(T) == 2 && !kPost)   // (with a norm after the block: registers)
            return run_back_use<T, kA, kPost, kGate, G, kC>(a, di, ws, g, stream);
    }
    return run_back_use<T, kA, kPost, kGate, G, kAny>(a, di, ws, g, stream);
}

// Two chunks per lane for 16-bit rows wider than one in a boundary without a norm after the block
// and a gate (16384 x 2048 fp16: 89 us, with one 93); with them the column sums of two chunks and
// their rows on the way do not fit an SM with as many warps. The choice does not go by the
// outputs asked for: dx and dh have the same bits with and without the others.
template <typename T, int kA>
cudaError_t run_back_any(const JoinArgs& a, const DevInfo& di, float* ws, BackGeom* g,
                         cudaStream_t stream) {
    const bool post = a.post != ZERO_NORM_NONE && (a.dh.p || a.dgate.p || a.dpost_w || a.dpost_b);
    if (post)
        return a.dgate.p ? run_back_kernel<T, kA, true, true, 1>(a, di, ws, g, stream)
                         : run_back_kernel<T, kA, true, false, 1>(a, di, ws, g, stream);
    if (a.dgate.p) return run_back_kernel<T, kA, false, true, 1>(a, di, ws, g, stream);
    if constexpr (sizeof(T) == 2 && kA == kWide) {
        if (chunks_of(a.cols) > 1 && a.post == ZERO_NORM_NONE && !a.gate.p)
            return run_back_kernel<T, kA, false, false, 2>(a, di, ws, g, stream);
    }
    return run_back_kernel<T, kA, false, false, 1>(a, di, ws, g, stream);
}

template <typename T>
cudaError_t run_join_back(const JoinArgs& a, float* ws, cudaStream_t stream) {
    DevInfo di;
    cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    BackGeom g = {};
    e = all_access<T>(a) == kWide ? run_back_any<T, kWide>(a, di, ws, &g, stream)
                                  : run_back_any<T, kNarrow>(a, di, ws, &g, stream);
    if (e != cudaSuccess) return e;
    const bool vectors = (a.dpost_w || a.dpost_b || a.dpre_w || a.dpre_b) &&
                         (g.clusters > 1 || a.rows == 0);
    const uint32_t gates = a.dgate.p && a.rows && g.parts > 1 ? g.units / g.parts : 0;
    if (!vectors && !gates) return cudaSuccess;
    return launch_act(join_vectors_kernel<T>, dim3((a.cols + 31) / 32, 4 + gates), 32 * kSumRows,
                      0, stream, a, g, vectors, (const float*)ws);
}

}  // namespace
}  // namespace zk
