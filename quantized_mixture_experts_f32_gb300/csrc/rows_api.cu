// rows_api.cu -- the C ABI of the 8-bit path's row operators (include/qmoe.h): argument
// checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "../../include/qmoe.h"
#include "qmoe_internal.h"
#include "rows.cuh"

namespace qmoe {

CtxView ctx_view(qmoe_ctx* c);                // qmoe_api.cu
CtxView kv4_ctx_view(qmoe_kv4* h);            // kv4_api.cu
Kv4View kv4_view(qmoe_kv4* h);
qmoe_status kv4_check_cache(qmoe_kv4* h, const qmoe_kv4_cache* c);
Kv4Cache kv4_cache(const qmoe_kv4_cache* c);

}  // namespace qmoe

namespace {

using qmoe::CtxView;

qmoe_status fail(const CtxView& c, qmoe_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(c.err, c.err_bytes, fmt, ap);
    va_end(ap);
    return s;
}

// how a launch went, in the context's error text
qmoe_status done(const CtxView& c, cudaError_t e, const char* what) {
    if (e != cudaSuccess) return fail(c, QMOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    c.err[0] = 0;
    return QMOE_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool valid_dtype(int t) { return t == QMOE_F32 || t == QMOE_F16 || t == QMOE_BF16; }
int dtype_bytes(int t) { return t == QMOE_F32 ? 4 : 2; }

constexpr int ROWS_MAX = 1 << 24;             // rows, tokens and features of a call
constexpr int DIM_MAX = 32768;                // elements of a row that is normalised or quantised
constexpr int K_MAX = 1 << 20;                // in_features

// rows of `row` elements: 0 stands for contiguous rows
qmoe_status check_rows(const CtxView& c, const char* name, const void* p, int dtype, int64_t row, int64_t* stride) {
    if (!valid_dtype(dtype)) return fail(c, QMOE_ERR_INVALID_ARG, "%s: dtype %d (0 F32, 1 F16, 2 BF16)", name, dtype);
    if (*stride == 0) *stride = row;
    if (*stride < row || *stride > (int64_t)1 << 40)
        return fail(c, QMOE_ERR_SHAPE, "%s: stride %lld is not 0 or %lld..2^40", name, (long long)*stride, (long long)row);
    if (!aligned(p, 16) || (*stride * dtype_bytes(dtype)) % 16)
        return fail(c, QMOE_ERR_MISALIGNED, "%s: base and row stride must be 16-byte aligned", name);
    return QMOE_OK;
}

// `out` may be `in` where their rows lie alike
qmoe_status check_alias(const CtxView& c, const char* names, const void* out, int out_t, int64_t out_stride, const void* in,
                        int in_t, int64_t in_stride) {
    if (in && out == in && (out_t != in_t || out_stride != in_stride))
        return fail(c, QMOE_ERR_INVALID_ARG, "%s may be the same only with the same type and stride", names);
    return QMOE_OK;
}

qmoe_status check_norm(const CtxView& c, const float* w, const char* name, float eps) {
    if (!w) return QMOE_OK;
    if (!aligned(w, 16)) return fail(c, QMOE_ERR_MISALIGNED, "%s must be 16-byte aligned", name);
    if (!(eps > 0.f) || !isfinite(eps)) return fail(c, QMOE_ERR_INVALID_ARG, "eps is not positive and finite");
    return QMOE_OK;
}

qmoe_status check_rope(const CtxView& c, const qmoe_rope_config* r, int head_dim, int unit) {
    if (!r || !r->table) return fail(c, QMOE_ERR_INVALID_ARG, "null rope or table pointer");
    if (r->layout != QMOE_ROPE_HALF && r->layout != QMOE_ROPE_INTERLEAVED)
        return fail(c, QMOE_ERR_INVALID_ARG, "rope layout %d (0 halves, 1 interleaved)", r->layout);
    if (r->rot_dim < unit || r->rot_dim > head_dim || r->rot_dim % unit)
        return fail(c, QMOE_ERR_SHAPE, "rot_dim=%d is not a multiple of %d in %d..%d", r->rot_dim, unit, unit, head_dim);
    if (r->n_pos < 1 || r->n_pos > ROWS_MAX) return fail(c, QMOE_ERR_SHAPE, "n_pos=%d outside 1..2^24", r->n_pos);
    if (!aligned(r->table, 16)) return fail(c, QMOE_ERR_MISALIGNED, "the rope table must be 16-byte aligned");
    return QMOE_OK;
}

bool positive(double x) { return x > 0.0 && isfinite(x); }

qmoe_status run_norm(const CtxView& c, const qmoe::NormArgs& a, const char* what) {
    qmoe::OnDevice dev(c.device);
    if (dev.e != cudaSuccess) return done(c, dev.e, "device select");
    return done(c, qmoe::launch_rmsnorm_rows(a, c.num_sms, c.stream), what);
}

}  // namespace

extern "C" {

qmoe_status qmoe_rmsnorm(qmoe_ctx* ctx, const void* x, qmoe_dtype x_t, int64_t x_stride, const void* residual,
                         qmoe_dtype res_t, int64_t res_stride, void* sum, const float* weight, float eps, int n_rows,
                         int dim, void* y, qmoe_dtype y_t, int64_t y_stride, float* y_scale) {
    if (!ctx) return QMOE_ERR_INVALID_ARG;
    const CtxView c = qmoe::ctx_view(ctx);
    if (!x || !y) return fail(c, QMOE_ERR_INVALID_ARG, "null pointer");
    if (n_rows < 1 || n_rows > ROWS_MAX) return fail(c, QMOE_ERR_SHAPE, "n_rows=%d outside 1..2^24", n_rows);
    if (dim < 16 || dim > DIM_MAX || dim % 16)
        return fail(c, QMOE_ERR_SHAPE, "dim=%d is not a multiple of 16 in 16..%d", dim, DIM_MAX);
    qmoe_status s = check_rows(c, "x", x, x_t, dim, &x_stride);
    if (s == QMOE_OK && residual) s = check_rows(c, "residual", residual, res_t, dim, &res_stride);
    if (s != QMOE_OK) return s;
    if (sum && !residual) return fail(c, QMOE_ERR_INVALID_ARG, "sum without a residual");
    if (!aligned(sum, 16)) return fail(c, QMOE_ERR_MISALIGNED, "sum must be 16-byte aligned");
    if (!(eps > 0.f) || !isfinite(eps)) return fail(c, QMOE_ERR_INVALID_ARG, "eps is not positive and finite");
    s = check_norm(c, weight, "weight", eps);
    if (s != QMOE_OK) return s;
    if (y_t == QMOE_E4M3) {
        if (!y_scale) return fail(c, QMOE_ERR_INVALID_ARG, "8-bit rows need y_scale");
        if (y_stride != 0 && y_stride != dim) return fail(c, QMOE_ERR_SHAPE, "8-bit rows are contiguous: y_stride 0 or dim");
        if (!aligned(y, 16) || !aligned(y_scale, 4))
            return fail(c, QMOE_ERR_MISALIGNED, "y must be 16-byte, y_scale 4-byte aligned");
        y_stride = dim;
        if (y == x || y == residual) return fail(c, QMOE_ERR_INVALID_ARG, "8-bit rows must not overlap an input");
    } else {
        if (y_scale) return fail(c, QMOE_ERR_INVALID_ARG, "y_scale is for 8-bit rows");
        s = check_rows(c, "y", y, y_t, dim, &y_stride);
        if (s == QMOE_OK) s = check_alias(c, "y and x", y, y_t, y_stride, x, x_t, x_stride);
        if (s != QMOE_OK) return s;
        if (y == residual) return fail(c, QMOE_ERR_INVALID_ARG, "y must not be the residual");
    }
    if (sum) {
        s = check_alias(c, "sum and x", sum, res_t, res_stride, x, x_t, x_stride);
        if (s != QMOE_OK) return s;
        if (sum == y) return fail(c, QMOE_ERR_INVALID_ARG, "sum and y must not be the same");
    }
    return run_norm(c, {x, residual, sum, weight, y, y_scale, x_stride, res_stride, y_stride, (int)x_t, (int)res_t, (int)y_t,
                        n_rows, dim, eps, 1}, "rmsnorm launch");
}

qmoe_status qmoe_fp8_quantize(qmoe_ctx* ctx, const void* x, qmoe_dtype x_t, int64_t x_stride, int n_rows, int cols,
                              void* codes, float* scale) {
    if (!ctx) return QMOE_ERR_INVALID_ARG;
    const CtxView c = qmoe::ctx_view(ctx);
    if (!x || !codes || !scale) return fail(c, QMOE_ERR_INVALID_ARG, "null pointer");
    if (n_rows < 1 || n_rows > ROWS_MAX) return fail(c, QMOE_ERR_SHAPE, "n_rows=%d outside 1..2^24", n_rows);
    if (cols < 16 || cols > DIM_MAX || cols % 16)
        return fail(c, QMOE_ERR_SHAPE, "cols=%d is not a multiple of 16 in 16..%d", cols, DIM_MAX);
    const qmoe_status s = check_rows(c, "x", x, x_t, cols, &x_stride);
    if (s != QMOE_OK) return s;
    if (!aligned(codes, 16) || !aligned(scale, 4))
        return fail(c, QMOE_ERR_MISALIGNED, "codes must be 16-byte, scale 4-byte aligned");
    if (codes == x) return fail(c, QMOE_ERR_INVALID_ARG, "codes must not overlap x");
    return run_norm(c, {x, nullptr, nullptr, nullptr, codes, scale, x_stride, 0, cols, (int)x_t, 0, QMOE_E4M3, n_rows, cols,
                        1.f, 0}, "quantise launch");
}

qmoe_status qmoe_linear_fp8(qmoe_ctx* ctx, const void* x_codes, const float* x_scale, int n_tokens, int in_features,
                            const void* w_codes, const float* w_scale, int out_features, const float* bias,
                            qmoe_act act, const void* residual, int64_t res_stride, void* out, qmoe_dtype out_t,
                            int64_t out_stride) {
    if (!ctx) return QMOE_ERR_INVALID_ARG;
    const CtxView c = qmoe::ctx_view(ctx);
    if (!x_codes || !x_scale || !w_codes || !w_scale || !out) return fail(c, QMOE_ERR_INVALID_ARG, "null pointer");
    if (n_tokens < 1 || n_tokens > ROWS_MAX) return fail(c, QMOE_ERR_SHAPE, "n_tokens=%d outside 1..2^24", n_tokens);
    if (out_features < 1 || out_features > ROWS_MAX)
        return fail(c, QMOE_ERR_SHAPE, "out_features=%d outside 1..2^24", out_features);
    if (in_features < 16 || in_features > K_MAX || in_features % 16)
        return fail(c, QMOE_ERR_SHAPE, "in_features=%d is not a multiple of 16 in 16..2^20", in_features);
    if (act < QMOE_ACT_NONE || act > QMOE_ACT_GELU) return fail(c, QMOE_ERR_INVALID_ARG, "activation %d", (int)act);
    if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4))
        return fail(c, QMOE_ERR_MISALIGNED, "codes must be 16-byte, scales and bias 4-byte aligned");
    qmoe_status s = check_rows(c, "out", out, out_t, out_features, &out_stride);
    if (s == QMOE_OK && residual) s = check_rows(c, "residual", residual, out_t, out_features, &res_stride);
    if (s == QMOE_OK) s = check_alias(c, "out and residual", out, out_t, out_stride, residual, out_t, res_stride);
    if (s != QMOE_OK) return s;
    if (out == x_codes || out == w_codes) return fail(c, QMOE_ERR_INVALID_ARG, "out must not overlap the codes");
    // what a tensor map can hold
    if (out_stride >= (int64_t)1 << 38 || (residual && res_stride >= (int64_t)1 << 38))
        return fail(c, QMOE_ERR_SHAPE, "out and residual: strides of 2^38 elements and more are not served");
    qmoe::OnDevice dev(c.device);
    if (dev.e != cudaSuccess) return done(c, dev.e, "device select");
    const qmoe::LinearArgs a{static_cast<const uint8_t*>(x_codes), x_scale, static_cast<const uint8_t*>(w_codes), w_scale,
                             bias, residual, out, res_stride, out_stride, n_tokens, in_features, out_features, (int)act,
                             (int)out_t, c.status, *c.stall_linear_ns};
    *c.stall_linear_ns = 0;
    return done(c, qmoe::launch_linear_fp8(a, {c.num_sms, c.stream, c.linear_ready}), "linear launch");
}

qmoe_status qmoe_debug_linear_choice(int num_sms, int n_tokens, int in_features, int out_features, int* tile, int* parts) {
    if (!tile || !parts || num_sms < 2 || n_tokens < 1 || n_tokens > ROWS_MAX || in_features < 16 || in_features > K_MAX ||
        in_features % 16 || out_features < 1 || out_features > ROWS_MAX)
        return QMOE_ERR_INVALID_ARG;
    const qmoe::LinearChoice c = qmoe::linear_fp8_choice(n_tokens, in_features, out_features, num_sms);
    *tile = c.tile;
    *parts = c.parts;
    return QMOE_OK;
}

qmoe_status qmoe_rope_table(qmoe_ctx* ctx, const qmoe_rope_config* r) {
    if (!ctx) return QMOE_ERR_INVALID_ARG;
    const CtxView c = qmoe::ctx_view(ctx);
    const qmoe_status s = check_rope(c, r, 256, 16);
    if (s != QMOE_OK) return s;
    if (!(r->base > 1.0) || !isfinite(r->base)) return fail(c, QMOE_ERR_INVALID_ARG, "rope base must be finite and above 1");
    if (r->scaling < QMOE_ROPE_PLAIN || r->scaling > QMOE_ROPE_PARTS)
        return fail(c, QMOE_ERR_INVALID_ARG, "rope scaling %d (0 none, 1 linear, 2 by parts)", r->scaling);
    if (r->scaling != QMOE_ROPE_PLAIN && !positive(r->factor))
        return fail(c, QMOE_ERR_INVALID_ARG, "rope factor must be positive and finite");
    if (r->scaling == QMOE_ROPE_PARTS &&
        (!positive(r->orig_ctx) || !positive(r->beta_slow) || !positive(r->beta_fast) || r->beta_fast <= r->beta_slow))
        return fail(c, QMOE_ERR_INVALID_ARG, "by parts: orig_ctx and beta_fast > beta_slow must be positive and finite");
    if (!(r->mscale >= 0.0) || !isfinite(r->mscale)) return fail(c, QMOE_ERR_INVALID_ARG, "rope mscale must be finite, not negative");
    const double pi = 3.14159265358979323846;
    const int half = r->rot_dim / 2;
    double lo = 0.0, hi = 0.0;
    if (r->scaling == QMOE_ROPE_PARTS) {
        const double unit = r->rot_dim / (2.0 * log(r->base));
        lo = fmax(floor(unit * log(r->orig_ctx / (2.0 * pi * r->beta_fast))), 0.0);
        hi = fmin(ceil(unit * log(r->orig_ctx / (2.0 * pi * r->beta_slow))), (double)(r->rot_dim - 1));
    }
    qmoe::RopeFreq f;
    for (int j = 0; j < 128; ++j) {
        if (j >= half) {
            f.f[j] = 0.0;
            continue;
        }
        double v = pow(r->base, -2.0 * j / r->rot_dim);
        if (r->scaling == QMOE_ROPE_LINEAR) v /= r->factor;
        if (r->scaling == QMOE_ROPE_PARTS) {
            const double ramp = fmin(fmax((j - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
            v = v * (1.0 - ramp) + v / r->factor * ramp;
        }
        f.f[j] = v;
    }
    double mscale = r->mscale;
    if (mscale == 0.0) mscale = r->scaling == QMOE_ROPE_PARTS && r->factor > 1.0 ? 0.1 * log(r->factor) + 1.0 : 1.0;
    qmoe::OnDevice dev(c.device);
    if (dev.e != cudaSuccess) return done(c, dev.e, "device select");
    return done(c, qmoe::launch_rope_rows_table(f, half, r->n_pos, mscale, r->table, c.stream), "rope table launch");
}

qmoe_status qmoe_rope(qmoe_ctx* ctx, const qmoe_rope_config* rope, const void* x, qmoe_dtype x_t, int64_t x_stride,
                      int n_tokens, int n_heads, int head_dim, const int32_t* positions, const float* norm, float eps,
                      void* out, int64_t out_stride) {
    if (!ctx) return QMOE_ERR_INVALID_ARG;
    const CtxView c = qmoe::ctx_view(ctx);
    if (!x || !positions || !out) return fail(c, QMOE_ERR_INVALID_ARG, "null pointer");
    if (n_tokens < 1 || n_tokens > 1 << 20) return fail(c, QMOE_ERR_SHAPE, "n_tokens=%d outside 1..2^20", n_tokens);
    if (n_heads < 1 || n_heads > 1024) return fail(c, QMOE_ERR_SHAPE, "n_heads=%d outside 1..1024", n_heads);
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(c, QMOE_ERR_SHAPE, "head_dim=%d is not 64, 128 or 256", head_dim);
    qmoe_status s = check_rope(c, rope, head_dim, 16);
    const int64_t row = (int64_t)n_heads * head_dim;
    if (s == QMOE_OK) s = check_rows(c, "x", x, x_t, row, &x_stride);
    if (s == QMOE_OK) s = check_rows(c, "out", out, x_t, row, &out_stride);
    if (s == QMOE_OK) s = check_alias(c, "out and x", out, x_t, out_stride, x, x_t, x_stride);
    if (s == QMOE_OK) s = check_norm(c, norm, "norm", eps);
    if (s != QMOE_OK) return s;
    if (!aligned(positions, 4)) return fail(c, QMOE_ERR_MISALIGNED, "positions must be 4-byte aligned");
    qmoe::OnDevice dev(c.device);
    if (dev.e != cudaSuccess) return done(c, dev.e, "device select");
    qmoe::RopeArgs a{};
    a.table = rope->table;
    a.n_pos = rope->n_pos;
    a.rot = rope->rot_dim;
    a.interleaved = rope->layout == QMOE_ROPE_INTERLEAVED;
    a.t = x_t;
    a.n_tokens = n_tokens;
    a.hd = head_dim;
    a.pos = positions;
    a.q = x;
    a.q_out = out;
    a.q_stride = x_stride;
    a.q_out_stride = out_stride;
    a.nq = n_heads;
    a.q_norm = norm;
    a.eps = eps;
    a.status = c.status;
    return done(c, qmoe::launch_rope(a, c.stream), "rope launch");
}

qmoe_status qmoe_kv4_append_rope(qmoe_kv4* kv, const qmoe_kv4_cache* cache, const qmoe_rope_config* rope, const void* q,
                                 const void* k, const void* v, qmoe_dtype dtype, int n_tokens, int64_t q_stride,
                                 int64_t k_stride, int64_t v_stride, const int32_t* positions, const int64_t* slots,
                                 const float* q_norm, const float* k_norm, float eps, void* q_out,
                                 int64_t q_out_stride, float* k_hat, float* v_hat) {
    if (!kv) return QMOE_ERR_INVALID_ARG;
    const CtxView c = qmoe::kv4_ctx_view(kv);
    const qmoe::Kv4View h = qmoe::kv4_view(kv);
    if (!k || !v || !positions || !slots) return fail(c, QMOE_ERR_INVALID_ARG, "null pointer");
    if (!q != !q_out) return fail(c, QMOE_ERR_INVALID_ARG, "q and q_out: both or neither");
    if (!q && q_norm) return fail(c, QMOE_ERR_INVALID_ARG, "q_norm without q");
    qmoe_status s = qmoe::kv4_check_cache(kv, cache);
    if (s != QMOE_OK) return s;
    if (n_tokens < 1 || n_tokens > h.max_tokens)
        return fail(c, QMOE_ERR_SHAPE, "n_tokens=%d outside 1..max_tokens=%d", n_tokens, h.max_tokens);
    s = check_rope(c, rope, h.s.hd, 32);
    const int64_t qrow = (int64_t)h.s.nq * h.s.hd, row = (int64_t)h.s.nkv * h.s.hd;
    if (s == QMOE_OK && q) s = check_rows(c, "q", q, dtype, qrow, &q_stride);
    if (s == QMOE_OK && q) s = check_rows(c, "q_out", q_out, dtype, qrow, &q_out_stride);
    if (s == QMOE_OK && q) s = check_alias(c, "q_out and q", q_out, dtype, q_out_stride, q, dtype, q_stride);
    if (s == QMOE_OK) s = check_rows(c, "k", k, dtype, row, &k_stride);
    if (s == QMOE_OK) s = check_rows(c, "v", v, dtype, row, &v_stride);
    if (s == QMOE_OK) s = check_norm(c, q_norm, "q_norm", eps);
    if (s == QMOE_OK) s = check_norm(c, k_norm, "k_norm", eps);
    if (s != QMOE_OK) return s;
    if (q_out == k || q_out == v) return fail(c, QMOE_ERR_INVALID_ARG, "q_out must not overlap k or v");
    if (!aligned(positions, 4) || !aligned(slots, 8) || !aligned(k_hat, 16) || !aligned(v_hat, 16))
        return fail(c, QMOE_ERR_MISALIGNED, "positions must be 4-byte, slots 8-byte, k_hat and v_hat 16-byte aligned");
    qmoe::OnDevice dev(c.device);
    if (dev.e != cudaSuccess) return done(c, dev.e, "device select");
    const qmoe::RopeArgs a{rope->table, rope->n_pos, rope->rot_dim, rope->layout == QMOE_ROPE_INTERLEAVED, (int)dtype,
                           n_tokens, h.s.hd, positions, q, q_out, q_stride, q_out_stride, q ? h.s.nq : 0, q_norm, k_norm,
                           eps, h.status, h.s.nkv, k, v, k_stride, v_stride, slots, k_hat, v_hat, qmoe::kv4_cache(cache),
                           h.s.page, h.s.page_log2, h.s.n_pages};
    return done(c, qmoe::launch_rope(a, c.stream), "append launch");
}

}  // extern "C"
