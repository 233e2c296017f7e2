// kv4_api.cu -- the C ABI of the paged 4-bit KV cache (include/qmoe.h): handles,
// argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <new>

#include "../../include/qmoe.h"
#include "kv4.cuh"
#include "qmoe_internal.h"

struct qmoe_kv4 {
    qmoe_kv4_config cfg;
    cudaStream_t stream;
    int device, num_sms;
    char err[512];
    void* ws;
    int* status;          // device status word
    unsigned* arrive;     // arrival counter of the plan kernel
    qmoe::Kv4Work work;   // attention
    unsigned long long stall_ns;   // test hook: work.stall_ns of the next attention
};

namespace {

constexpr int NOMINAL_SMS = 152;   // qmoe_kv4_workspace_bytes needs no device: a GB300's multiprocessors

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct Layout {
    size_t status, arrive, items, ext_items, ext_total, parts, ext_parts, total;
};

Layout layout(const qmoe_kv4_config* c, int num_sms) {
    Layout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off = align256(off + bytes); return o; };
    L.status = take(sizeof(int));
    L.arrive = take(sizeof(unsigned));
    L.items = take(sizeof(unsigned) * qmoe::kv4_arrive_words(num_sms));
    L.ext_items = take(sizeof(unsigned) * qmoe::kv4_arrive_words(num_sms));
    L.ext_total = take(sizeof(unsigned));
    L.parts = take(sizeof(float) * qmoe::kv4_decode_part_floats(c->head_dim, num_sms));
    L.ext_parts = take(sizeof(float) * qmoe::kv4_extend_part_floats(c->head_dim, num_sms,
                                                                    (long long)c->max_tokens * (c->n_heads / c->n_kv_heads)));
    L.total = off;
    return L;
}

bool config_ok(const qmoe_kv4_config* c, char* why, size_t n) {
    if (!c) { snprintf(why, n, "config is NULL"); return false; }
    if (c->n_heads < 1 || c->n_heads > 1024 || c->n_kv_heads < 1 || c->n_heads % c->n_kv_heads) { snprintf(why, n, "n_heads=%d (1..1024) must be a positive multiple of n_kv_heads=%d", c->n_heads, c->n_kv_heads); return false; }
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) { snprintf(why, n, "head_dim=%d is not 64, 128 or 256", c->head_dim); return false; }
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) { snprintf(why, n, "page_size=%d is not 16, 32, 64, 128 or 256", c->page_size); return false; }
    if (c->n_pages < 1 || c->n_pages > (1 << 30)) { snprintf(why, n, "n_pages=%d outside 1..2^30", c->n_pages); return false; }
    if (c->max_seqs < 1 || c->max_seqs > 4096) { snprintf(why, n, "max_seqs=%d outside 1..4096", c->max_seqs); return false; }
    if (c->max_tokens < 1 || c->max_tokens > (1 << 20)) { snprintf(why, n, "max_tokens=%d outside 1..2^20", c->max_tokens); return false; }
    if (c->max_pages_per_seq < 1 || (long long)c->max_pages_per_seq * c->page_size > (1ll << 30)) { snprintf(why, n, "max_pages_per_seq=%d must be positive and at most 2^30/page_size", c->max_pages_per_seq); return false; }
    return true;
}

qmoe_status fail(qmoe_kv4* h, qmoe_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(h->err, sizeof(h->err), fmt, ap);
    va_end(ap);
    return s;
}

qmoe_status cuda_fail(qmoe_kv4* h, cudaError_t e, const char* what) {
    return fail(h, QMOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool valid_dtype(int t) { return t == QMOE_F32 || t == QMOE_F16 || t == QMOE_BF16; }
int dtype_bytes(int t) { return t == QMOE_F32 ? 4 : 2; }

qmoe::Kv4Shape shape(const qmoe_kv4* h) {
    const qmoe_kv4_config& c = h->cfg;
    int log2 = 0;
    while ((1 << log2) < c.page_size) ++log2;
    return {c.n_heads, c.n_kv_heads, c.head_dim, c.page_size, c.n_pages, c.max_pages_per_seq, log2};
}

qmoe_status check_cache(qmoe_kv4* h, const qmoe_kv4_cache* c) {
    if (!c || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !c->k_global || !c->v_global)
        return fail(h, QMOE_ERR_INVALID_ARG, "null cache pointer");
    if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
        !aligned(c->v_scales, 16) || !aligned(c->k_global, 4) || !aligned(c->v_global, 4))
        return fail(h, QMOE_ERR_MISALIGNED, "cache codes and scales must be 16-byte aligned, globals 4-byte");
    return QMOE_OK;
}

qmoe::Kv4Cache cache_of(const qmoe_kv4_cache* c) {
    return {static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->k_scales),
            static_cast<uint8_t*>(c->v_codes), static_cast<uint8_t*>(c->v_scales), c->k_global, c->v_global};
}

// rows of `row` elements: 0 stands for contiguous rows
qmoe_status check_rows(qmoe_kv4* h, const char* name, const void* p, int dtype, int64_t row, int64_t* stride) {
    if (!valid_dtype(dtype)) return fail(h, QMOE_ERR_INVALID_ARG, "%s: dtype %d (0 F32, 1 F16, 2 BF16)", name, dtype);
    if (*stride == 0) *stride = row;
    if (*stride < row || *stride > (int64_t)1 << 40)
        return fail(h, QMOE_ERR_SHAPE, "%s: stride %lld is not 0 or %lld..2^40", name, (long long)*stride, (long long)row);
    if (!aligned(p, 16) || (*stride * dtype_bytes(dtype)) % 16)
        return fail(h, QMOE_ERR_MISALIGNED, "%s: base and row stride must be 16-byte aligned", name);
    return QMOE_OK;
}

}  // namespace

namespace qmoe {

Kv4View kv4_view(qmoe_kv4* h) {
    return {shape(h), h->work, h->status, &h->stall_ns, h->stream, h->device, h->cfg.max_seqs, h->cfg.max_tokens};
}

qmoe_status kv4_check_cache(qmoe_kv4* h, const qmoe_kv4_cache* c) { return check_cache(h, c); }

Kv4Cache kv4_cache(const qmoe_kv4_cache* c) { return cache_of(c); }

}  // namespace qmoe

extern "C" {

size_t qmoe_kv4_workspace_bytes(const qmoe_kv4_config* cfg) {
    char why[256];
    return config_ok(cfg, why, sizeof(why)) ? layout(cfg, NOMINAL_SMS).total : 0;
}

qmoe_status qmoe_kv4_create(const qmoe_kv4_config* cfg, qmoe_kv4** out) {
    qmoe::create_error("");
    if (!out) {
        qmoe::create_error("out is NULL");
        return QMOE_ERR_INVALID_ARG;
    }
    *out = nullptr;
    char why[256];
    if (!config_ok(cfg, why, sizeof(why))) {
        qmoe::create_error("%s", why);
        return QMOE_ERR_INVALID_ARG;
    }
    qmoe_kv4* h = new (std::nothrow) qmoe_kv4();
    if (!h) {
        qmoe::create_error("host allocation of the handle failed");
        return QMOE_ERR_NO_MEMORY;
    }
    h->cfg = *cfg;
    h->stream = static_cast<cudaStream_t>(cfg->stream);
    cudaError_t e = cudaGetDevice(&h->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
    if (e != cudaSuccess) {
        qmoe::create_error("device query: %s", cudaGetErrorString(e));
        delete h;
        return QMOE_ERR_CUDA;
    }
    e = qmoe::kv4_plan_prepare();
    if (e == cudaSuccess) e = qmoe::kv4_decode_prepare();
    if (e == cudaSuccess) e = qmoe::kv4_extend_prepare();
    if (e != cudaSuccess) {
        qmoe::create_error("kernel set-up: %s", cudaGetErrorString(e));
        delete h;
        return QMOE_ERR_CUDA;
    }
    const Layout L = layout(cfg, h->num_sms);
    e = qmoe::fail_next_alloc() ? cudaErrorMemoryAllocation : cudaMalloc(&h->ws, L.total);
    if (e != cudaSuccess) {
        cudaGetLastError();
        qmoe::create_error("workspace allocation of %zu bytes failed: %s", L.total, cudaGetErrorString(e));
        delete h;
        return QMOE_ERR_NO_MEMORY;
    }
    char* b = static_cast<char*>(h->ws);
    h->status = reinterpret_cast<int*>(b + L.status);
    h->arrive = reinterpret_cast<unsigned*>(b + L.arrive);
    h->work = {reinterpret_cast<float*>(b + L.parts), reinterpret_cast<float*>(b + L.ext_parts),
               reinterpret_cast<unsigned*>(b + L.items), reinterpret_cast<unsigned*>(b + L.ext_items),
               reinterpret_cast<unsigned*>(b + L.ext_total), h->num_sms, 0};
    e = cudaMemsetAsync(h->ws, 0, L.parts, h->stream);   // all but the attention's parts
    if (e == cudaSuccess) e = cudaStreamSynchronize(h->stream);
    if (e != cudaSuccess) {
        qmoe::create_error("workspace clear: %s", cudaGetErrorString(e));
        cudaFree(h->ws);
        delete h;
        return QMOE_ERR_CUDA;
    }
    *out = h;
    return QMOE_OK;
}

void qmoe_kv4_destroy(qmoe_kv4* h) {
    if (!h) return;
    {
        qmoe::OnDevice dev(h->device);
        cudaStreamSynchronize(h->stream);
        cudaFree(h->ws);
    }
    delete h;
}

qmoe_status qmoe_kv4_set_stream(qmoe_kv4* h, void* stream) {
    if (!h) return QMOE_ERR_INVALID_ARG;
    h->stream = static_cast<cudaStream_t>(stream);
    h->cfg.stream = stream;
    return QMOE_OK;
}

const char* qmoe_kv4_last_error(qmoe_kv4* h) { return h ? h->err : qmoe_last_error(nullptr); }

qmoe_status qmoe_kv4_get_status(qmoe_kv4* h) {
    if (!h) return QMOE_ERR_INVALID_ARG;
    qmoe::OnDevice dev(h->device);
    if (dev.e != cudaSuccess) return cuda_fail(h, dev.e, "device select");
    int st = 0;
    cudaError_t e = cudaMemcpyAsync(&st, h->status, sizeof(int), cudaMemcpyDeviceToHost, h->stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(h->stream);
    if (e != cudaSuccess) return cuda_fail(h, e, "status read");
    if (st == 0) return QMOE_OK;
    e = cudaMemsetAsync(h->status, 0, sizeof(int), h->stream);
    if (e != cudaSuccess) return cuda_fail(h, e, "status clear");
    return fail(h, static_cast<qmoe_status>(st), "device reported status %d", st);
}

qmoe_status qmoe_kv4_plan(qmoe_kv4* h, int n_seqs, const int32_t* seq_len, const int32_t* new_len,
                          int32_t* block_table, int32_t* free_pages, const int32_t* n_free,
                          int cap_tokens, int32_t* seq_len_out, int32_t* n_free_out,
                          int32_t* cu_tokens, int32_t* positions, int64_t* slots) {
    if (!h) return QMOE_ERR_INVALID_ARG;
    if (!seq_len || !new_len || !block_table || !free_pages || !n_free || !seq_len_out || !n_free_out ||
        !cu_tokens || !positions || !slots)
        return fail(h, QMOE_ERR_INVALID_ARG, "null pointer");
    const qmoe_kv4_config& c = h->cfg;
    if (n_seqs < 1 || n_seqs > c.max_seqs)
        return fail(h, QMOE_ERR_SHAPE, "n_seqs=%d outside 1..max_seqs=%d", n_seqs, c.max_seqs);
    if (cap_tokens < 1 || cap_tokens > c.max_tokens)
        return fail(h, QMOE_ERR_SHAPE, "cap_tokens=%d outside 1..max_tokens=%d", cap_tokens, c.max_tokens);
    if (!aligned(seq_len, 4) || !aligned(new_len, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
        !aligned(n_free, 4) || !aligned(seq_len_out, 4) || !aligned(n_free_out, 4) || !aligned(cu_tokens, 4) ||
        !aligned(positions, 4) || !aligned(slots, 8))
        return fail(h, QMOE_ERR_MISALIGNED, "int32 arrays must be 4-byte aligned, slots 8-byte");
    if (seq_len_out == new_len || cu_tokens == seq_len || cu_tokens == new_len || cu_tokens == seq_len_out)
        return fail(h, QMOE_ERR_INVALID_ARG, "only seq_len_out = seq_len and n_free_out = n_free may alias");
    qmoe::OnDevice dev(h->device);
    if (dev.e != cudaSuccess) return cuda_fail(h, dev.e, "device select");
    const qmoe::Kv4PlanArgs a{n_seqs, c.page_size, c.n_pages, c.max_pages_per_seq, cap_tokens, seq_len, new_len,
                              block_table, free_pages, n_free, seq_len_out, n_free_out, cu_tokens, positions,
                              slots, h->arrive, h->status};
    const cudaError_t e = qmoe::launch_kv4_plan(a, h->num_sms, h->stream);
    if (e != cudaSuccess) return cuda_fail(h, e, "plan launch");
    h->err[0] = 0;
    return QMOE_OK;
}

qmoe_status qmoe_kv4_append(qmoe_kv4* h, const qmoe_kv4_cache* cache, const void* k, const void* v,
                            qmoe_dtype dtype, int n_tokens, int64_t k_stride, int64_t v_stride,
                            const int64_t* slots, float* k_hat, float* v_hat) {
    if (!h) return QMOE_ERR_INVALID_ARG;
    if (!k || !v || !slots) return fail(h, QMOE_ERR_INVALID_ARG, "null pointer");
    qmoe_status s = check_cache(h, cache);
    if (s != QMOE_OK) return s;
    const qmoe_kv4_config& c = h->cfg;
    if (n_tokens < 1 || n_tokens > c.max_tokens)
        return fail(h, QMOE_ERR_SHAPE, "n_tokens=%d outside 1..max_tokens=%d", n_tokens, c.max_tokens);
    const int64_t row = (int64_t)c.n_kv_heads * c.head_dim;
    s = check_rows(h, "k", k, dtype, row, &k_stride);
    if (s == QMOE_OK) s = check_rows(h, "v", v, dtype, row, &v_stride);
    if (s != QMOE_OK) return s;
    if (!aligned(slots, 8) || !aligned(k_hat, 16) || !aligned(v_hat, 16))
        return fail(h, QMOE_ERR_MISALIGNED, "slots must be 8-byte, k_hat and v_hat 16-byte aligned");
    qmoe::OnDevice dev(h->device);
    if (dev.e != cudaSuccess) return cuda_fail(h, dev.e, "device select");
    const qmoe::Kv4AppendArgs a{shape(h), cache_of(cache), k, v, (int)dtype, n_tokens, k_stride, v_stride, slots,
                                k_hat, v_hat, h->status};
    const cudaError_t e = qmoe::launch_kv4_append(a, h->stream);
    if (e != cudaSuccess) return cuda_fail(h, e, "append launch");
    h->err[0] = 0;
    return QMOE_OK;
}

qmoe_status qmoe_kv4_attention(qmoe_kv4* h, const qmoe_kv4_cache* cache, const void* q,
                               qmoe_dtype q_t, int64_t q_stride, int n_seqs, int n_tokens,
                               int max_new, const int32_t* cu_tokens, const int32_t* seq_len,
                               const int32_t* block_table, float scale, void* out,
                               qmoe_dtype out_t, int64_t out_stride, float* lse) {
    if (!h) return QMOE_ERR_INVALID_ARG;
    if (!q || !cu_tokens || !seq_len || !block_table || !out)
        return fail(h, QMOE_ERR_INVALID_ARG, "null pointer");
    qmoe_status s = check_cache(h, cache);
    if (s != QMOE_OK) return s;
    const qmoe_kv4_config& c = h->cfg;
    if (n_seqs < 1 || n_seqs > c.max_seqs)
        return fail(h, QMOE_ERR_SHAPE, "n_seqs=%d outside 1..max_seqs=%d", n_seqs, c.max_seqs);
    if (n_tokens < 1 || n_tokens > c.max_tokens)
        return fail(h, QMOE_ERR_SHAPE, "n_tokens=%d outside 1..max_tokens=%d", n_tokens, c.max_tokens);
    if (max_new < 1 || max_new > n_tokens)
        return fail(h, QMOE_ERR_SHAPE, "max_new=%d outside 1..n_tokens=%d", max_new, n_tokens);
    if (!isfinite(scale)) return fail(h, QMOE_ERR_INVALID_ARG, "scale is not finite");
    const int64_t row = (int64_t)c.n_heads * c.head_dim;
    s = check_rows(h, "q", q, q_t, row, &q_stride);
    if (s == QMOE_OK) s = check_rows(h, "out", out, out_t, row, &out_stride);
    if (s != QMOE_OK) return s;
    if (!aligned(cu_tokens, 4) || !aligned(seq_len, 4) || !aligned(block_table, 4) || !aligned(lse, 4))
        return fail(h, QMOE_ERR_MISALIGNED, "cu_tokens, seq_len, block_table and lse must be 4-byte aligned");
    if (out == q) return fail(h, QMOE_ERR_INVALID_ARG, "out must not overlap q");
    qmoe::OnDevice dev(h->device);
    if (dev.e != cudaSuccess) return cuda_fail(h, dev.e, "device select");
    const qmoe::Kv4AttnArgs a{shape(h), cache_of(cache), q, (int)q_t, (int)out_t, q_stride, out_stride, n_seqs,
                              n_tokens, max_new, cu_tokens, seq_len, block_table, scale, out, lse, h->status};
    qmoe::Kv4Work w = h->work;
    w.stall_ns = h->stall_ns;
    h->stall_ns = 0;
    const cudaError_t e = qmoe::launch_kv4_attention(a, w, h->stream);
    if (e != cudaSuccess) return cuda_fail(h, e, "attention launch");
    h->err[0] = 0;
    return QMOE_OK;
}

qmoe_status qmoe_kv4_debug_stall_next(qmoe_kv4* h, uint64_t wait_ns) {
    if (!h || wait_ns == 0 || wait_ns > 1000000000ull) return QMOE_ERR_INVALID_ARG;
    h->stall_ns = wait_ns;
    return QMOE_OK;
}

}  // extern "C"
