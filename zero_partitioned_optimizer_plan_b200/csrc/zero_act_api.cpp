// C ABI of the activation-side calls (8-bit checkpoints, block boundary, weight gradient from a
// checkpoint): argument checks and launches. Every function returns a zero_status and never
// throws.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/libzero.h"
#include "zero_act.h"
#include "zero_internal.h"

namespace zk {
namespace {

constexpr uint64_t kMaxBytes = UINT64_MAX / 2;   // every matrix fits in 63 bits of bytes

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool dtype_ok(int t) { return t == ZERO_F16 || t == ZERO_BF16 || t == ZERO_F32; }
bool norm_ok(int n) { return n == ZERO_NORM_NONE || n == ZERO_NORM_RMS || n == ZERO_NORM_LAYER; }
uint64_t elem(int t) { return t == ZERO_F32 ? 4 : 2; }

// A buffer a call reads or writes: rows of `width` bytes, `pitch` bytes apart.
struct Span {
    const void* p;
    uint64_t rows, width, pitch;
    uint64_t bytes() const { return rows ? (rows - 1) * pitch + width : 0; }
};

// Do two buffers share a byte? Rows of one pitch may interleave (column slices of one matrix).
bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || !a.rows || !b.rows || !a.width || !b.width) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (x >= y + b.bytes() || y >= x + a.bytes()) return false;
    if (a.pitch != b.pitch || a.rows == 1 || b.rows == 1) return true;
    const uint64_t d = y >= x ? (y - x) % a.pitch : (a.pitch - (x - y) % a.pitch) % a.pitch;
    return d < a.width || d + b.width > a.pitch;
}

// rows x cols with stride ld: the stride covers a row and the whole fits in 63 bits.
bool shape_ok(uint64_t rows, uint64_t cols, uint64_t ld, uint64_t es) {
    if (ld < cols || ld > kMaxBytes / es) return false;
    return rows == 0 || ld == 0 || rows <= kMaxBytes / (ld * es);
}

Span mat_span(const void* p, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t es) {
    return Span{p, rows, cols * es, ld * es};
}

Span ckpt_span(const void* p, uint64_t rows, uint64_t cols) {
    const uint64_t rb = ZERO_CKPT_ROW_BYTES(cols);
    return Span{p, rows, rb, rb};
}

Span vec_span(const void* p, uint64_t bytes) { return Span{p, 1, bytes, bytes}; }

zero_status check_ckpt_call(uint64_t rows, uint64_t cols, int dtype, const void* m, uint64_t ld,
                            const uint8_t* ckpt) {
    if (!dtype_ok(dtype) || cols >= (1ull << 31) || !shape_ok(rows, cols, ld, elem(dtype)) ||
        (rows && rows > kMaxBytes / (ZERO_CKPT_ROW_BYTES(cols) + 1)))
        return ZERO_EINVAL;
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!m || !ckpt) return ZERO_EINVAL;
    if (!aligned(m, elem(dtype)) || !aligned(ckpt, 16)) return ZERO_EALIGN;
    if (overlap(mat_span(m, rows, cols, ld, elem(dtype)), ckpt_span(ckpt, rows, cols)))
        return ZERO_EINVAL;
    return ZERO_OK;
}

// The boundary's calls keep row numbers and row pitches (bytes) in 32 bits.
constexpr uint64_t kMaxRows = 1ull << 31;

// The description's own rules (no buffers but the gate and the vectors).
zero_status check_desc(const zero_block_desc* d) {
    if (!d || !dtype_ok(d->dtype) || !norm_ok(d->post_norm) || !norm_ok(d->pre_norm))
        return ZERO_EINVAL;
    if (d->cols > ZERO_JOIN_MAX_COLS || d->rows >= kMaxRows) return ZERO_EINVAL;
    if (!std::isfinite(d->post_eps) || d->post_eps < 0 || !std::isfinite(d->pre_eps) ||
        d->pre_eps < 0 || !std::isfinite(d->residual_scale) || !std::isfinite(d->branch_scale))
        return ZERO_EINVAL;
    if ((d->gate_rows == 0) != (d->gate == nullptr) && d->rows && d->cols) return ZERO_EINVAL;
    if (d->post_norm == ZERO_NORM_NONE && (d->post_w || d->post_b)) return ZERO_EINVAL;
    if (d->pre_norm == ZERO_NORM_NONE && (d->pre_w || d->pre_b)) return ZERO_EINVAL;
    return ZERO_OK;
}

// (any gate_rows: the sum rows + gate_rows may pass 64 bits)
uint64_t gate_count(const zero_block_desc* d) {
    return d->gate_rows && d->rows ? (d->rows - 1) / d->gate_rows + 1 : 0;
}

// The buffers of one boundary call: every one checked for its shape and alignment as it is
// added, then every output against everything else.
struct Buffers {
    static constexpr int kMax = 24;
    Span s[kMax];
    bool out[kMax];
    int n = 0;
    uint64_t max_pitch = kMaxBytes;
    zero_status st = ZERO_OK;

    void add(const Span& sp, uint64_t align, bool is_out) {
        if (!sp.p || !sp.rows) return;
        if (st == ZERO_OK && !aligned(sp.p, align)) st = ZERO_EALIGN;
        s[n] = sp;
        out[n++] = is_out;
    }
    void mat(const void* p, uint64_t rows, uint64_t cols, uint64_t ld, uint64_t es, bool is_out) {
        if (!p) return;
        if (!shape_ok(rows, cols, ld, es) || ld * es >= max_pitch) {
            st = ZERO_EINVAL;
            return;
        }
        add(mat_span(p, rows, cols, ld, es), es, is_out);
    }
    // `alias`: an output that may be exactly this input (same address and pitch)
    zero_status check(const void* out_p, const void* in_p) const {
        if (st != ZERO_OK) return st;
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < n; ++j) {
                if (i == j || !out[i] || (out[j] && j < i)) continue;
                if (out_p && s[i].p == out_p && s[j].p == in_p && in_p == out_p && !out[j] &&
                    s[i].pitch == s[j].pitch && s[i].width == s[j].width)
                    continue;
                if (overlap(s[i], s[j])) return ZERO_EINVAL;
            }
        return ZERO_OK;
    }
};

void add_desc(Buffers& b, const zero_block_desc* d) {
    const uint64_t es = elem(d->dtype), vb = d->cols * es;
    b.max_pitch = kMaxRows;
    b.mat(d->gate, gate_count(d), d->cols, d->ldg, es, false);
    b.add(vec_span(d->post_w, vb), es, false);
    b.add(vec_span(d->post_b, vb), es, false);
    b.add(vec_span(d->pre_w, vb), es, false);
    b.add(vec_span(d->pre_b, vb), es, false);
}

Rows rows_of(const zero_block_desc* d, const void* p, uint64_t ld) {
    return Rows{const_cast<void*>(p), (uint32_t)(ld * elem(d->dtype))};
}

// A matrix or a checkpoint.
Rows source(const zero_block_desc* d, const void* p, uint64_t ld, const uint8_t* ck) {
    if (ck) return Rows{const_cast<uint8_t*>(ck), (uint32_t)ZERO_CKPT_ROW_BYTES(d->cols)};
    return rows_of(d, p, ld);
}

JoinArgs join_args(const zero_block_desc* d) {
    JoinArgs a = {};
    a.rows = (uint32_t)d->rows;
    a.cols = (uint32_t)d->cols;
    a.post = d->post_norm;
    a.pre = d->pre_norm;
    a.post_eps = d->post_eps;
    a.pre_eps = d->pre_eps;
    a.rs = d->residual_scale;
    a.bs = d->branch_scale;
    a.gate_rows = (uint32_t)(d->gate_rows < d->rows ? d->gate_rows : d->rows);
    a.gate = rows_of(d, d->gate, d->ldg);
    a.post_w = d->post_w;
    a.post_b = d->post_b;
    a.pre_w = d->pre_w;
    a.pre_b = d->pre_b;
    a.ck = ckpt_shape(d->cols);
    return a;
}

Mat mat(const void* p, uint64_t ld) { return Mat{const_cast<void*>(p), ld}; }

}  // namespace
}  // namespace zk

using namespace zk;

extern "C" {

zero_status zero_ckpt_save_q8(uint64_t rows, uint64_t cols, zero_dtype dtype, const void* x,
                              uint64_t ldx, uint8_t* ckpt, zero_stream_t stream) {
    const zero_status st = check_ckpt_call(rows, cols, dtype, x, ldx, ckpt);
    if (st != ZERO_OK || rows == 0 || cols == 0) return st;
    return from_cuda(launch_ckpt_save(rows, ckpt_shape(cols), dtype, mat(x, ldx), ckpt,
                                      (cudaStream_t)stream));
}

zero_status zero_ckpt_load_q8(uint64_t rows, uint64_t cols, const uint8_t* ckpt, zero_dtype dtype,
                              void* out, uint64_t ldo, zero_stream_t stream) {
    const zero_status st = check_ckpt_call(rows, cols, dtype, out, ldo, ckpt);
    if (st != ZERO_OK || rows == 0 || cols == 0) return st;
    return from_cuda(launch_ckpt_load(rows, ckpt_shape(cols), dtype, ckpt, mat(out, ldo),
                                      (cudaStream_t)stream));
}

static bool wgrad_sizes_ok(uint64_t t, uint64_t o, uint64_t i) {
    return t < (1ull << 31) && o < (1ull << 30) && i < (1ull << 30);
}

zero_status zero_ckpt_wgrad_q8_workspace(uint64_t tokens, uint64_t out_features,
                                         uint64_t in_features, uint64_t* bytes) {
    if (!bytes || !wgrad_sizes_ok(tokens, out_features, in_features)) return ZERO_EINVAL;
    *bytes = wgrad_workspace(tokens, out_features, in_features);
    return ZERO_OK;
}

zero_status zero_ckpt_wgrad_q8(uint64_t tokens, uint64_t out_features, uint64_t in_features,
                               zero_dtype dtype, const void* dy, uint64_t lddy,
                               const uint8_t* ckpt, void* dw, uint64_t lddw, int accumulate,
                               void* workspace, uint64_t workspace_bytes, uint32_t* d_status,
                               zero_stream_t stream) {
    if (!wgrad_sizes_ok(tokens, out_features, in_features) || !d_status ||
        (dtype != ZERO_F16 && dtype != ZERO_BF16))
        return ZERO_EINVAL;
    const uint64_t es = elem(dtype);
    if (!shape_ok(tokens, out_features, lddy, es) || !shape_ok(out_features, in_features, lddw, es))
        return ZERO_EINVAL;
    if (out_features == 0 || in_features == 0) return ZERO_OK;
    if (!dw || (tokens && (!dy || !ckpt))) return ZERO_EINVAL;
    const uint64_t need = wgrad_workspace(tokens, out_features, in_features);
    if (need && !workspace) return ZERO_EINVAL;
    if (workspace_bytes < need) return ZERO_ENOMEM;
    if (!aligned(dw, es) || !aligned(d_status, 4) || (need && !aligned(workspace, 16)) ||
        (tokens && (!aligned(dy, es) || !aligned(ckpt, 16))))
        return ZERO_EALIGN;
    Buffers b;
    b.mat(dw, out_features, in_features, lddw, es, true);
    b.add(vec_span(need ? workspace : nullptr, need), 16, true);
    b.add(vec_span(d_status, 4), 4, true);
    if (tokens) {
        b.mat(dy, tokens, out_features, lddy, es, false);
        b.add(ckpt_span(ckpt, tokens, in_features), 16, false);
    }
    const zero_status st = b.check(nullptr, nullptr);
    if (st != ZERO_OK) return st;
    if (tokens == 0 && accumulate) return ZERO_OK;
    WgradArgs a = {};
    a.tokens = tokens;
    a.outf = (uint32_t)out_features;
    a.inf = (uint32_t)in_features;
    a.dy = mat(dy, lddy);
    a.dw = mat(dw, lddw);
    a.ckpt = ckpt;
    a.ck = ckpt_shape(in_features);
    a.accumulate = accumulate != 0;
    a.status = d_status;
    return from_cuda(launch_wgrad(a, dtype, workspace, (cudaStream_t)stream));
}

zero_status zero_block_join(const zero_block_desc* desc, const void* x, uint64_t ldx,
                            const uint8_t* x_ckpt, const void* h, uint64_t ldh,
                            const uint8_t* h_ckpt, void* y, uint64_t ldy, void* u, uint64_t ldu,
                            uint8_t* save_y, uint8_t* save_h, zero_stream_t stream) {
    zero_status st = check_desc(desc);
    if (st != ZERO_OK) return st;
    if (desc->rows == 0 || desc->cols == 0) return ZERO_OK;
    if ((x != nullptr) == (x_ckpt != nullptr) || (h && h_ckpt)) return ZERO_EINVAL;
    const bool branch = h || h_ckpt;
    if (!branch && (desc->post_norm != ZERO_NORM_NONE || desc->gate)) return ZERO_EINVAL;
    if (!y && !u && !save_y && !save_h) return ZERO_EINVAL;
    if ((u && desc->pre_norm == ZERO_NORM_NONE) || (save_h && !h)) return ZERO_EINVAL;
    const uint64_t R = desc->rows, C = desc->cols, es = elem(desc->dtype);
    Buffers b;
    add_desc(b, desc);
    b.mat(x, R, C, ldx, es, false);
    b.add(ckpt_span(x_ckpt, R, C), 16, false);
    b.mat(h, R, C, ldh, es, false);
    b.add(ckpt_span(h_ckpt, R, C), 16, false);
    b.mat(y, R, C, ldy, es, true);
    b.mat(u, R, C, ldu, es, true);
    b.add(ckpt_span(save_y, R, C), 16, true);
    b.add(ckpt_span(save_h, R, C), 16, true);
    st = b.check(y, x);
    if (st != ZERO_OK) return st;
    JoinArgs a = join_args(desc);
    a.x = source(desc, x, ldx, x_ckpt);
    a.x_codes = x_ckpt != nullptr;
    a.h = source(desc, h, ldh, h_ckpt);
    a.h_codes = h_ckpt != nullptr;
    a.y = rows_of(desc, y, ldy);
    a.u = rows_of(desc, u, ldu);
    a.save_y = source(desc, nullptr, 0, save_y);
    a.save_h = source(desc, nullptr, 0, save_h);
    a.has_branch = branch;
    return from_cuda(launch_join(a, desc->dtype, (cudaStream_t)stream));
}

zero_status zero_block_join_backward_workspace(uint64_t rows, uint64_t cols, uint64_t gate_rows,
                                               uint64_t* bytes) {
    if (!bytes || cols > ZERO_JOIN_MAX_COLS || rows >= kMaxRows) return ZERO_EINVAL;
    *bytes = join_workspace(rows, cols, gate_rows);
    return ZERO_OK;
}

zero_status zero_block_join_backward(const zero_block_desc* desc, int has_branch, const void* y,
                                     uint64_t ldy, const uint8_t* y_ckpt, const void* h,
                                     uint64_t ldh, const uint8_t* h_ckpt, const void* dy,
                                     uint64_t lddy, const void* du, uint64_t lddu, void* dx,
                                     uint64_t lddx, void* dh, uint64_t lddh, void* dgate,
                                     uint64_t lddg, void* dpost_w, void* dpost_b, void* dpre_w,
                                     void* dpre_b, int accumulate, void* workspace,
                                     uint64_t workspace_bytes, zero_stream_t stream) {
    zero_status st = check_desc(desc);
    if (st != ZERO_OK) return st;
    if (desc->cols == 0) return ZERO_OK;
    const bool vectors = dgate || dpost_w || dpost_b || dpre_w || dpre_b;
    if ((y && y_ckpt) || (h && h_ckpt) || (!dx && !dh && !vectors) || (accumulate & ~3))
        return ZERO_EINVAL;
    if (!has_branch && (desc->post_norm != ZERO_NORM_NONE || desc->gate || h || h_ckpt || dh ||
                        dgate || dpost_w || dpost_b))
        return ZERO_EINVAL;
    if ((dgate && !desc->gate_rows) ||
        ((dpost_w || dpost_b) && desc->post_norm == ZERO_NORM_NONE) ||
        ((dpre_w || dpre_b || du) && desc->pre_norm == ZERO_NORM_NONE))
        return ZERO_EINVAL;
    if (desc->rows) {
        if (du && !y && !y_ckpt) return ZERO_EINVAL;
        if ((desc->post_norm != ZERO_NORM_NONE || dgate) && !h && !h_ckpt) return ZERO_EINVAL;
    }
    const uint64_t R = desc->rows, C = desc->cols, es = elem(desc->dtype), vb = C * es;
    const uint64_t need = vectors ? join_workspace(R, C, desc->gate_rows) : 0;
    if (need && !workspace) return ZERO_EINVAL;
    if (workspace_bytes < need) return ZERO_ENOMEM;
    Buffers b;
    add_desc(b, desc);
    b.mat(y, R, C, ldy, es, false);
    b.add(ckpt_span(y_ckpt, R, C), 16, false);
    b.mat(h, R, C, ldh, es, false);
    b.add(ckpt_span(h_ckpt, R, C), 16, false);
    b.mat(dy, R, C, lddy, es, false);
    b.mat(du, R, C, lddu, es, false);
    b.mat(dx, R, C, lddx, es, true);
    b.mat(dh, R, C, lddh, es, true);
    b.mat(dgate, gate_count(desc), C, lddg, es, true);
    b.add(vec_span(dpost_w, vb), es, true);
    b.add(vec_span(dpost_b, vb), es, true);
    b.add(vec_span(dpre_w, vb), es, true);
    b.add(vec_span(dpre_b, vb), es, true);
    b.add(vec_span(need ? workspace : nullptr, need), 16, true);
    st = b.check(dx, dy);
    if (st != ZERO_OK) return st;
    JoinArgs a = join_args(desc);
    a.x = source(desc, y, ldy, y_ckpt);
    a.x_codes = y_ckpt != nullptr;
    a.h = source(desc, h, ldh, h_ckpt);
    a.h_codes = h_ckpt != nullptr;
    a.dy = rows_of(desc, dy, lddy);
    a.du = rows_of(desc, du, lddu);
    a.dx = rows_of(desc, dx, lddx);
    a.dh = rows_of(desc, dh, lddh);
    a.dgate = rows_of(desc, dgate, lddg);
    a.dpost_w = dpost_w;
    a.dpost_b = dpost_b;
    a.dpre_w = dpre_w;
    a.dpre_b = dpre_b;
    a.has_branch = has_branch != 0;
    a.accumulate = accumulate;
    if (R == 0 && (!vectors || (accumulate & ZERO_ACC_PARAMS))) return ZERO_OK;
    return from_cuda(launch_join_backward(a, desc->dtype, workspace, (cudaStream_t)stream));
}

}  // extern "C"
