// Host side of the paged cache: validation, buffer sizes, launches.  Stateless: every
// buffer is the caller's, so that calls can be captured into graphs.  No exceptions
// cross the C ABI.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "dq_internal.h"
#include "pages_internal.h"

namespace {

dq_status fail(dq_status s, const char *fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return dq::set_last_error(s, msg);
}
dq_status ok() { return dq::set_last_error(DQ_OK, ""); }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

dq_status check_cfg(const dq_pages_config *c) {
    if (!c) return fail(DQ_EINVAL, "NULL argument");
    if (c->n_layers < 1 || c->n_layers > 4096) return fail(DQ_EINVAL, "n_layers outside [1, 4096]");
    if (c->n_pages < 1 || c->n_pages > DQ_PAGES_MAX_PAGES)
        return fail(DQ_EINVAL, "n_pages outside [1, %d]", DQ_PAGES_MAX_PAGES);
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return fail(DQ_EUNSUPPORTED, "page_size must be 16, 32, 64 or 128 (got %d)", c->page_size);
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(DQ_EUNSUPPORTED, "head_dim must be 64 or 128 (got %d)", c->head_dim);
    if (c->n_kv_heads < 1 || c->n_kv_heads > 128) return fail(DQ_EINVAL, "n_kv_heads outside [1, 128]");
    if (c->n_q_heads < c->n_kv_heads || c->n_q_heads % c->n_kv_heads)
        return fail(DQ_EINVAL, "n_q_heads (%d) is no multiple of n_kv_heads (%d)", c->n_q_heads, c->n_kv_heads);
    if (c->n_q_heads / c->n_kv_heads > 16) return fail(DQ_EUNSUPPORTED, "more than 16 query heads per KV head");
    if (c->max_seqs < 1 || c->max_seqs > DQ_PAGES_MAX_ROWS)
        return fail(DQ_EINVAL, "max_seqs outside [1, %d]", DQ_PAGES_MAX_ROWS);
    if (c->max_pages_per_seq < 1 || c->max_pages_per_seq > 65536 ||
        static_cast<long long>(c->max_pages_per_seq) * c->page_size > (1 << 22))
        return fail(DQ_EINVAL, "max_pages_per_seq outside [1, 65536], or more than 2^22 tokens in a row");
    if (c->dtype != DQ_F16 && c->dtype != DQ_BF16) return fail(DQ_EUNSUPPORTED, "dtype must be f16 or bf16");
    if (c->k_exp < -16 || c->k_exp > 16 || c->v_exp < -16 || c->v_exp > 16)
        return fail(DQ_EINVAL, "k_exp and v_exp must be in [-16, 16]");
    return DQ_OK;
}

int page_bytes(const dq_pages_config *c) { return c->page_size * c->head_dim * 9 / 8; }
int sum_bytes(const dq_pages_config *c) { return 2 * c->head_dim + 16; }

int device_sms() {  // of the current device; looked up once for each device
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// Config and buffers -> the view that kernels take; `layer` < 0: the whole pool.
dq_status view(const dq_pages_config *c, const dq_pages_buffers *b, int layer, bool workspace, dq::PagesView &v) {
    dq_status s = check_cfg(c);
    if (s != DQ_OK) return s;
    if (!b || !b->pages || !b->summary || !b->table || !b->seq_len || !b->refs || !b->status ||
        (workspace && !b->workspace))
        return fail(DQ_EINVAL, "a pool buffer is NULL");
    if (!aligned16(b->pages) || !aligned16(b->summary) || !aligned16(b->table) || !aligned16(b->seq_len) ||
        !aligned16(b->refs) || !aligned16(b->status) || !aligned16(b->workspace))
        return fail(DQ_EALIGN, "a pool buffer is not 16-byte aligned");
    if (layer >= c->n_layers) return fail(DQ_EINVAL, "layer %d outside [0, %d)", layer, c->n_layers);
    v.n_layers = c->n_layers;
    v.n_pages = c->n_pages;
    v.P = c->page_size;
    v.Hkv = c->n_kv_heads;
    v.Hq = c->n_q_heads;
    v.G = c->n_q_heads / c->n_kv_heads;
    v.d = c->head_dim;
    v.max_seqs = c->max_seqs;
    v.M = c->max_pages_per_seq;
    v.bf16 = c->dtype == DQ_BF16;
    v.blk = c->page_size < 64 ? c->page_size : 64;
    v.page_bytes = page_bytes(c);
    v.sum_bytes = sum_bytes(c);
    v.k_exp = c->k_exp;
    v.v_exp = c->v_exp;
    const size_t at = static_cast<size_t>(layer < 0 ? 0 : layer) * c->n_pages * c->n_kv_heads;
    v.pages = static_cast<uint8_t *>(b->pages) + at * v.page_bytes;
    v.summary = static_cast<uint8_t *>(b->summary) + at * v.sum_bytes;
    v.table = b->table;
    v.seq_len = b->seq_len;
    v.refs = b->refs;
    v.status = static_cast<unsigned *>(b->status);
    return DQ_OK;
}

dq_status call_rows(const dq_pages_config *c, int layer, const int *rows, const int *cu, int n_rows, int n_tok, int max_new,
                    dq::PagesRows &r) {
    if (layer < 0) return fail(DQ_EINVAL, "layer %d is negative", layer);
    if (n_rows < 1 || n_rows > DQ_PAGES_MAX_ROWS)
        return fail(DQ_EINVAL, "n_rows outside [1, %d]", DQ_PAGES_MAX_ROWS);
    if (!rows && n_rows > c->max_seqs) return fail(DQ_EINVAL, "%d rows in a table of %d", n_rows, c->max_seqs);
    if (!aligned4(rows) || !aligned4(cu)) return fail(DQ_EALIGN, "rows / cu not aligned to 4 bytes");
    if (n_tok < 1 || n_tok > (1 << 24)) return fail(DQ_EINVAL, "n_tok outside [1, 2^24]");
    if (max_new < 1 || max_new > n_tok) return fail(DQ_EINVAL, "max_new outside [1, n_tok]");
    if (!cu && (n_tok != n_rows || max_new != 1))
        return fail(DQ_EINVAL, "without cu there is one token for each row (n_tok %d, n_rows %d)", n_tok, n_rows);
    r = dq::PagesRows{rows, cu, n_rows, n_tok, max_new};
    return DQ_OK;
}

dq_status launched(int e, const char *what) {
    if (e != 0) return fail(DQ_ECUDA, "%s: %s", what, cudaGetErrorString(static_cast<cudaError_t>(e)));
    return ok();
}

// What turns a product of a query and a key's code values into a logit in log2 units.
float logit_scale(const dq_pages_config *c, float sm_scale) {
    return static_cast<float>(std::ldexp(static_cast<double>(sm_scale) * 1.4426950408889634074, c->k_exp));
}

constexpr int PAGES_MAX_TOKENS = 1 << 22;  // of a row

dq_status check_cap(int cap) {
    if (cap < 1 || cap > PAGES_MAX_TOKENS) return fail(DQ_EINVAL, "cap outside [1, 2^22]");
    return DQ_OK;
}

dq_status check_groups(const int *groups, int n_groups, int n_rows, const int *plan) {
    if (n_groups < 1 || n_groups > n_rows || (!groups && n_groups != 1))
        return fail(DQ_EINVAL, "n_groups outside [1, n_rows], or more than 1 without groups");
    if (!plan) return fail(DQ_EINVAL, "plan is NULL");
    if (!aligned4(groups) || (reinterpret_cast<uintptr_t>(plan) & 7u)) return fail(DQ_EALIGN, "groups not aligned to 4 bytes, or plan to 8");
    return DQ_OK;
}

// Checked arguments of an attention call.
dq_status attention_args(dq::PagesAttnArgs &a, const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                         long long q_tok_stride, long long q_head_stride, void *out, float *lse, const int *rows, const int *cu,
                         int n_rows, int n_tok, int max_new, const int *sel, int n_sel, float sm_scale) {
    dq_status s = view(cfg, bufs, layer, true, a.p);
    if (s != DQ_OK) return s;
    if ((s = call_rows(cfg, layer, rows, cu, n_rows, n_tok, max_new, a.r)) != DQ_OK) return s;
    if (!q || !out) return fail(DQ_EINVAL, "q / out is NULL");
    if (!aligned16(q) || !aligned16(out) || (q_tok_stride | q_head_stride) & 7)
        return fail(DQ_EALIGN, "q / out not 16-byte aligned, or a stride is no multiple of 8 elements");
    if (!aligned4(lse) || !aligned4(sel)) return fail(DQ_EALIGN, "lse / sel not aligned to 4 bytes");
    if (!std::isfinite(sm_scale)) return fail(DQ_EINVAL, "sm_scale is not finite");
    if (sel && (n_sel < 1 || n_sel > DQ_PAGES_MAX_SELECT))
        return fail(DQ_EINVAL, "n_sel outside [1, %d]", DQ_PAGES_MAX_SELECT);
    if (sel && cu) return fail(DQ_EUNSUPPORTED, "chosen pages go with one query token for each row (cu must be NULL)");
    a.q = static_cast<const uint16_t *>(q);
    a.qt = q_tok_stride;
    a.qh = q_head_stride;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.sel = sel;
    a.n_sel = sel ? n_sel : 0;
    a.scale_log2 = logit_scale(cfg, sm_scale);
    a.out_scale = std::ldexp(1.0f, cfg->v_exp);
    uint8_t *ws = static_cast<uint8_t *>(bufs->workspace) + dq::pages_ws_lists(cfg->n_pages);
    a.tickets = reinterpret_cast<int *>(ws);
    a.joins = reinterpret_cast<int *>(ws + dq::PAGES_MAX_CTAS * 4);
    a.records = reinterpret_cast<float *>(ws + dq::PAGES_MAX_CTAS * 20);
    a.wait_ns = dq::PAGES_WAIT_NS;
    a.owed = 0;
    return DQ_OK;
}

// The same of a call of shared attention.
dq_status shared_args(dq::PagesAttnArgs &a, const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                      long long q_tok_stride, long long q_head_stride, void *out, float *lse, const int *rows, const int *cu, int n_rows,
                      int n_tok, int max_new, const int *groups, int n_groups, int max_group, const int *plan, void *scratch,
                      float sm_scale) {
    dq_status s = attention_args(a, cfg, bufs, layer, q, q_tok_stride, q_head_stride, out, lse, rows, cu, n_rows, n_tok, max_new,
                                 nullptr, 0, sm_scale);
    if (s != DQ_OK) return s;
    if ((s = check_groups(groups, n_groups, n_rows, plan)) != DQ_OK) return s;
    if (max_group < 1 || max_group > n_tok) return fail(DQ_EINVAL, "max_group outside [1, n_tok]");
    if (!scratch) return fail(DQ_EINVAL, "scratch is NULL");
    if (!aligned16(scratch)) return fail(DQ_EALIGN, "scratch not 16-byte aligned");
    a.groups = groups;
    a.plan = plan;
    a.call_rows = n_rows;
    a.part = static_cast<float *>(scratch);
    uint8_t *ws = static_cast<uint8_t *>(bufs->workspace) + dq::pages_ws_own(cfg->n_pages);
    a.own_tickets = reinterpret_cast<int *>(ws);
    a.own_records = reinterpret_cast<float *>(ws + dq::PAGES_MAX_CTAS * 4);
    return DQ_OK;
}

// Checked arguments of a call that weighs.
dq_status weigh_args(dq::PagesWeighArgs &a, const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                     long long q_tok_stride, long long q_head_stride, const float *lse, float *scores, int cap, const int *rows,
                     const int *cu, int n_rows, int n_tok, int max_new, float sm_scale) {
    dq_status s = view(cfg, bufs, layer, true, a.p);
    if (s != DQ_OK) return s;
    if ((s = call_rows(cfg, layer, rows, cu, n_rows, n_tok, max_new, a.r)) != DQ_OK) return s;
    if (!q || !lse || !scores) return fail(DQ_EINVAL, "q / lse / scores is NULL");
    if (!aligned16(q) || (q_tok_stride | q_head_stride) & 7)
        return fail(DQ_EALIGN, "q not 16-byte aligned, or a stride is no multiple of 8 elements");
    if (!aligned4(lse) || !aligned4(scores)) return fail(DQ_EALIGN, "lse / scores not aligned to 4 bytes");
    if ((s = check_cap(cap)) != DQ_OK) return s;
    if (!std::isfinite(sm_scale)) return fail(DQ_EINVAL, "sm_scale is not finite");
    a.q = static_cast<const uint16_t *>(q);
    a.qt = q_tok_stride;
    a.qh = q_head_stride;
    a.lse = lse;
    a.scores = scores;
    a.cap = cap;
    a.scale_log2 = logit_scale(cfg, sm_scale);
    uint8_t *ws = static_cast<uint8_t *>(bufs->workspace) + dq::pages_ws_lists(cfg->n_pages);
    a.tickets = reinterpret_cast<int *>(ws);
    a.records = reinterpret_cast<float *>(ws + dq::PAGES_MAX_CTAS * 20);
    a.wait_ns = dq::PAGES_WAIT_NS;
    a.owed = 0;
    return DQ_OK;
}

unsigned long long expire_limit(unsigned long long ns) { return ns < 1000ULL ? 1000ULL : (ns > 1000000000ULL ? 1000000000ULL : ns); }

}  // namespace

extern "C" {

dq_status dq_pages_sizes(const dq_pages_config *cfg, size_t bytes[DQ_PAGES_NUM_BUFFERS]) {
    if (!cfg || !bytes) return fail(DQ_EINVAL, "NULL argument");
    const dq_status s = check_cfg(cfg);
    if (s != DQ_OK) return s;
    const size_t n = static_cast<size_t>(cfg->n_layers) * cfg->n_pages * cfg->n_kv_heads;
    bytes[0] = n * page_bytes(cfg);
    bytes[1] = n * sum_bytes(cfg);
    bytes[2] = static_cast<size_t>(cfg->max_seqs) * cfg->max_pages_per_seq * 4;
    bytes[3] = static_cast<size_t>(cfg->max_seqs) * 4;
    bytes[4] = static_cast<size_t>(cfg->n_pages) * 4;
    bytes[5] = 16;
    bytes[6] = dq::pages_ws_bytes(cfg->n_pages);
    return ok();
}

dq_status dq_pages_resize(const dq_pages_config *cfg, const dq_pages_buffers *bufs, const int *rows, const int *lens, int n,
                          void *stream) {
    dq::PagesView v;
    const dq_status s = view(cfg, bufs, -1, true, v);
    if (s != DQ_OK) return s;
    if (!lens) return fail(DQ_EINVAL, "lens is NULL");
    if (!aligned4(rows) || !aligned4(lens)) return fail(DQ_EALIGN, "rows / lens not aligned to 4 bytes");
    if (n < 1 || n > DQ_PAGES_MAX_ROWS || (!rows && n > cfg->max_seqs))
        return fail(DQ_EINVAL, "%d rows: outside [1, %d], or more than the table has", n, DQ_PAGES_MAX_ROWS);
    return launched(dq::launch_pages_resize(v, rows, lens, n, static_cast<int *>(bufs->workspace), device_sms(), stream),
                    "resize launch");
}

dq_status dq_pages_fork(const dq_pages_config *cfg, const dq_pages_buffers *bufs, const int *src, const int *dst, int n,
                        void *stream) {
    dq::PagesView v;
    const dq_status s = view(cfg, bufs, -1, false, v);
    if (s != DQ_OK) return s;
    if (!src || !dst) return fail(DQ_EINVAL, "src / dst is NULL");
    if (!aligned4(src) || !aligned4(dst)) return fail(DQ_EALIGN, "src / dst not aligned to 4 bytes");
    if (n < 1 || n > DQ_PAGES_MAX_ROWS) return fail(DQ_EINVAL, "n outside [1, %d]", DQ_PAGES_MAX_ROWS);
    return launched(dq::launch_pages_fork(v, src, dst, n, stream), "fork launch");
}

dq_status dq_pages_compact(const dq_pages_config *cfg, const dq_pages_buffers *bufs, void *stream) {
    dq::PagesView v;
    const dq_status s = view(cfg, bufs, -1, true, v);
    if (s != DQ_OK) return s;
    return launched(dq::launch_pages_compact(v, static_cast<int *>(bufs->workspace), device_sms(), stream), "compact launch");
}

dq_status dq_pages_append(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *k, const void *v,
                          long long k_tok_stride, long long k_head_stride, long long v_tok_stride, long long v_head_stride,
                          const int *rows, const int *cu, int n_rows, int n_tok, int max_new, void *stream) {
    dq::PagesStoreArgs a{};
    dq_status s = view(cfg, bufs, layer, false, a.p);
    if (s != DQ_OK) return s;
    if ((s = call_rows(cfg, layer, rows, cu, n_rows, n_tok, max_new, a.r)) != DQ_OK) return s;
    if (!k || !v) return fail(DQ_EINVAL, "k / v is NULL");
    if (!aligned16(k) || !aligned16(v) || (k_tok_stride | k_head_stride | v_tok_stride | v_head_stride) & 7)
        return fail(DQ_EALIGN, "k / v not 16-byte aligned, or a stride is no multiple of 8 elements");
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.kt = k_tok_stride;
    a.kh = k_head_stride;
    a.vt = v_tok_stride;
    a.vh = v_head_stride;
    return launched(dq::launch_pages_append(a, stream), "append launch");
}

dq_status dq_pages_read(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, void *k_out, void *v_out,
                        const int *rows, const int *cu, int n_rows, int n_tok, int max_new, void *stream) {
    dq::PagesReadArgs a{};
    dq_status s = view(cfg, bufs, layer, false, a.p);
    if (s != DQ_OK) return s;
    if ((s = call_rows(cfg, layer, rows, cu, n_rows, n_tok, max_new, a.r)) != DQ_OK) return s;
    if (!k_out || !v_out) return fail(DQ_EINVAL, "k_out / v_out is NULL");
    if (!aligned16(k_out) || !aligned16(v_out)) return fail(DQ_EALIGN, "k_out / v_out not 16-byte aligned");
    a.k = static_cast<uint16_t *>(k_out);
    a.v = static_cast<uint16_t *>(v_out);
    return launched(dq::launch_pages_read(a, stream), "read launch");
}

dq_status dq_pages_attention(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                             long long q_tok_stride, long long q_head_stride, void *out, float *lse, const int *rows,
                             const int *cu, int n_rows, int n_tok, int max_new, const int *sel, int n_sel, float sm_scale,
                             void *stream) {
    dq::PagesAttnArgs a{};
    const dq_status s = attention_args(a, cfg, bufs, layer, q, q_tok_stride, q_head_stride, out, lse, rows, cu, n_rows, n_tok,
                                       max_new, sel, n_sel, sm_scale);
    if (s != DQ_OK) return s;
    return launched(dq::launch_pages_attention(a, dq::PAGES_NEWEST, device_sms(), stream), "attention launch");
}

dq_status dq_pages_cross(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q, long long q_tok_stride,
                         long long q_head_stride, void *out, float *lse, const int *rows, const int *cu, int n_rows, int n_tok,
                         int max_new, float sm_scale, void *stream) {
    dq::PagesAttnArgs a{};
    const dq_status s = attention_args(a, cfg, bufs, layer, q, q_tok_stride, q_head_stride, out, lse, rows, cu, n_rows, n_tok,
                                       max_new, nullptr, 0, sm_scale);
    if (s != DQ_OK) return s;
    return launched(dq::launch_pages_attention(a, dq::PAGES_ALL, device_sms(), stream), "cross attention launch");
}

dq_status dq_pages_common(const dq_pages_config *cfg, const dq_pages_buffers *bufs, const int *rows, const int *cu, int n_rows,
                          const int *groups, int n_groups, int always, int *plan, void *stream) {
    dq::PagesCommonArgs a{};
    dq_status s = view(cfg, bufs, -1, false, a.p);
    if (s != DQ_OK) return s;
    constexpr int any = 1 << 24;  // tokens: none of them is looked at
    if ((s = call_rows(cfg, 0, rows, cu, n_rows, cu ? any : n_rows, cu ? any : 1, a.r)) != DQ_OK) return s;
    if ((s = check_groups(groups, n_groups, n_rows, plan)) != DQ_OK) return s;
    a.groups = groups;
    a.n_groups = n_groups;
    a.always = always;
    a.num_sms = device_sms();
    a.plan = plan;
    return launched(dq::launch_pages_common(a, stream), "common launch");
}

dq_status dq_pages_shared_bytes(const dq_pages_config *cfg, int n_tok, size_t *bytes) {
    if (!cfg || !bytes) return fail(DQ_EINVAL, "NULL argument");
    const dq_status s = check_cfg(cfg);
    if (s != DQ_OK) return s;
    if (n_tok < 1 || n_tok > (1 << 24)) return fail(DQ_EINVAL, "n_tok outside [1, 2^24]");
    *bytes = static_cast<size_t>(n_tok) * cfg->n_q_heads * (cfg->head_dim + 2) * 4;
    return ok();
}

dq_status dq_pages_shared(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q, long long q_tok_stride,
                          long long q_head_stride, void *out, float *lse, const int *rows, const int *cu, int n_rows, int n_tok,
                          int max_new, const int *groups, int n_groups, int max_group, const int *plan, void *scratch,
                          float sm_scale, void *stream) {
    dq::PagesAttnArgs a{};
    const dq_status s = shared_args(a, cfg, bufs, layer, q, q_tok_stride, q_head_stride, out, lse, rows, cu, n_rows, n_tok, max_new,
                                    groups, n_groups, max_group, plan, scratch, sm_scale);
    if (s != DQ_OK) return s;
    return launched(dq::launch_pages_shared(a, n_groups, max_group, device_sms(), stream), "shared attention launch");
}

dq_status dq_pages_weigh(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q, long long q_tok_stride,
                         long long q_head_stride, const float *lse, float *scores, int cap, const int *rows, const int *cu,
                         int n_rows, int n_tok, int max_new, float sm_scale, void *stream) {
    dq::PagesWeighArgs a{};
    const dq_status s = weigh_args(a, cfg, bufs, layer, q, q_tok_stride, q_head_stride, lse, scores, cap, rows, cu, n_rows, n_tok,
                                   max_new, sm_scale);
    if (s != DQ_OK) return s;
    return launched(dq::launch_pages_weigh(a, device_sms(), stream), "weigh launch");
}

dq_status dq_pages_evict(const dq_pages_config *cfg, const dq_pages_buffers *bufs, float *scores, int cap, const int *src,
                         const int *dst, int n, int keep_first, int keep_last, void *stream) {
    dq::PagesEvictArgs a{};
    dq_status s = view(cfg, bufs, -1, true, a.p);
    if (s != DQ_OK) return s;
    if (!scores || !src || !dst) return fail(DQ_EINVAL, "scores / src / dst is NULL");
    if (!aligned4(scores) || !aligned4(src) || !aligned4(dst)) return fail(DQ_EALIGN, "scores / src / dst not aligned to 4 bytes");
    if ((s = check_cap(cap)) != DQ_OK) return s;
    if (n < 1 || n > DQ_PAGES_MAX_ROWS) return fail(DQ_EINVAL, "n outside [1, %d]", DQ_PAGES_MAX_ROWS);
    if (keep_first < 0 || keep_last < 0 || keep_first > PAGES_MAX_TOKENS || keep_last > PAGES_MAX_TOKENS)
        return fail(DQ_EINVAL, "keep_first / keep_last outside [0, 2^22]");
    a.scores = scores;
    a.cap = cap;
    a.src = src;
    a.dst = dst;
    a.n = n;
    a.keep_first = keep_first;
    a.keep_last = keep_last;
    a.keeps = reinterpret_cast<int *>(static_cast<uint8_t *>(bufs->workspace) + dq::pages_ws_lists(cfg->n_pages) + dq::PAGES_MAX_CTAS * 20);
    return launched(dq::launch_pages_evict(a, device_sms(), stream), "evict launch");
}

dq_status dq_pages_test_expire_wait(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                                    long long q_tok_stride, long long q_head_stride, void *out, const int *cu, int n_rows,
                                    int n_tok, int max_new, unsigned long long limit_ns, void *stream) {
    dq::PagesAttnArgs a{};
    const dq_status s = attention_args(a, cfg, bufs, layer, q, q_tok_stride, q_head_stride, out, nullptr, nullptr, cu, n_rows,
                                       n_tok, max_new, nullptr, 0, 1.0f);
    if (s != DQ_OK) return s;
    a.owed = 1;
    a.wait_ns = expire_limit(limit_ns);
    return launched(dq::launch_pages_attention(a, dq::PAGES_NEWEST, device_sms(), stream), "expire-wait launch");
}

dq_status dq_pages_test_expire_cross(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                                     long long q_tok_stride, long long q_head_stride, void *out, const int *cu, int n_rows,
                                     int n_tok, int max_new, unsigned long long limit_ns, void *stream) {
    dq::PagesAttnArgs a{};
    const dq_status s = attention_args(a, cfg, bufs, layer, q, q_tok_stride, q_head_stride, out, nullptr, nullptr, cu, n_rows,
                                       n_tok, max_new, nullptr, 0, 1.0f);
    if (s != DQ_OK) return s;
    a.owed = 1;
    a.wait_ns = expire_limit(limit_ns);
    return launched(dq::launch_pages_attention(a, dq::PAGES_ALL, device_sms(), stream), "expire-cross launch");
}

dq_status dq_pages_test_expire_shared(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                                      long long q_tok_stride, long long q_head_stride, void *out, const int *cu, int n_rows,
                                      int n_tok, int max_new, const int *groups, int n_groups, int max_group, const int *plan,
                                      void *scratch, unsigned long long limit_ns, void *stream) {
    dq::PagesAttnArgs a{};
    const dq_status s = shared_args(a, cfg, bufs, layer, q, q_tok_stride, q_head_stride, out, nullptr, nullptr, cu, n_rows, n_tok,
                                    max_new, groups, n_groups, max_group, plan, scratch, 1.0f);
    if (s != DQ_OK) return s;
    a.owed = 1;
    a.wait_ns = expire_limit(limit_ns);
    return launched(dq::launch_pages_shared(a, n_groups, max_group, device_sms(), stream), "expire-shared launch");
}

dq_status dq_pages_test_expire_weigh(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                                     long long q_tok_stride, long long q_head_stride, const float *lse, float *scores, int cap,
                                     const int *cu, int n_rows, int n_tok, int max_new, unsigned long long limit_ns, void *stream) {
    dq::PagesWeighArgs a{};
    const dq_status s = weigh_args(a, cfg, bufs, layer, q, q_tok_stride, q_head_stride, lse, scores, cap, nullptr, cu, n_rows, n_tok,
                                   max_new, 1.0f);
    if (s != DQ_OK) return s;
    a.owed = 1;
    a.wait_ns = expire_limit(limit_ns);
    return launched(dq::launch_pages_weigh(a, device_sms(), stream), "expire-weigh launch");
}

dq_status dq_pages_select(const dq_pages_config *cfg, const dq_pages_buffers *bufs, int layer, const void *q,
                          long long q_tok_stride, long long q_head_stride, const int *rows, int n_rows, int *sel, int n_sel,
                          int keep_first, int keep_last, void *stream) {
    dq::PagesSelectArgs a{};
    dq_status s = view(cfg, bufs, layer, false, a.p);
    if (s != DQ_OK) return s;
    if ((s = call_rows(cfg, layer, rows, nullptr, n_rows, n_rows, 1, a.r)) != DQ_OK) return s;
    if (!q || !sel) return fail(DQ_EINVAL, "q / sel is NULL");
    if (!aligned16(q) || (q_tok_stride | q_head_stride) & 7)
        return fail(DQ_EALIGN, "q not 16-byte aligned, or a stride is no multiple of 8 elements");
    if (!aligned4(sel)) return fail(DQ_EALIGN, "sel not aligned to 4 bytes");
    if (n_sel < 1 || n_sel > DQ_PAGES_MAX_SELECT) return fail(DQ_EINVAL, "n_sel outside [1, %d]", DQ_PAGES_MAX_SELECT);
    if (cfg->max_pages_per_seq > dq::PAGES_SELECT_MAX)
        return fail(DQ_EUNSUPPORTED, "select: more than %d pages in a row", dq::PAGES_SELECT_MAX);
    if (keep_first < 0 || keep_last < 0 || static_cast<long long>(keep_first) + keep_last > n_sel)
        return fail(DQ_EINVAL, "keep_first + keep_last must be in [0, n_sel]");
    a.q = static_cast<const uint16_t *>(q);
    a.qt = q_tok_stride;
    a.qh = q_head_stride;
    a.sel = sel;
    a.n_sel = n_sel;
    a.keep_first = keep_first;
    a.keep_last = keep_last;
    return launched(dq::launch_pages_select(a, device_sms(), stream), "select launch");
}

dq_status dq_pages_check(const dq_pages_buffers *bufs, void *stream) {
    if (!bufs || !bufs->status) return fail(DQ_EINVAL, "NULL argument");
    const auto st = static_cast<cudaStream_t>(stream);
    static const struct {
        unsigned bit;
        dq_status status;
        const char *what;
    } latched[] = {  // the gravest first
        {dq::PST_TIMEOUT, DQ_ETIMEOUT, "a bounded device wait ran out"},
        {dq::PST_FULL, DQ_ENOMEM, "resize: too few free pages; nothing was changed"},
        {dq::PST_ARG, DQ_EINVAL, "a row, length or count is out of range, or a row was named twice"},
        {dq::PST_TABLE, DQ_EINVAL, "a table names no page of the pool"},
        {dq::PST_SHARED, DQ_EINVAL, "an append or an eviction met a page that several rows hold: resize after a fork"},
        {dq::PST_NONFINITE, DQ_ENONFINITE, "non-finite K/V input"}};
    unsigned w = 0;
    cudaError_t e = cudaMemcpyAsync(&w, bufs->status, sizeof w, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return fail(DQ_ECUDA, "status: %s", cudaGetErrorString(e));
    for (const auto &l : latched) {
        if (!(w & l.bit)) continue;
        // the reported bit alone is cleared: what another stream latches meanwhile stays
        e = static_cast<cudaError_t>(dq::launch_pages_clear(static_cast<unsigned *>(bufs->status), l.bit, stream));
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
        if (e != cudaSuccess) return fail(DQ_ECUDA, "status: %s", cudaGetErrorString(e));
        return fail(l.status, "%s", l.what);
    }
    return ok();
}

}  // extern "C"
