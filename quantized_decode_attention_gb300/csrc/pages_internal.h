// Internal declarations of the paged cache: geometry, kernel arguments, launchers.
#pragma once

#include <cstddef>
#include <cstdint>

#include "dq_pages.h"

namespace dq {

// Bits of the status word beside those of dq_internal.h that the paged cache shares
// (1 non-finite input, 2 timeout).
enum : unsigned {
    PST_NONFINITE = 1u,
    PST_TIMEOUT = 2u,
    PST_FULL = 64u,    // resize: too few free pages
    PST_ARG = 128u,    // a row, length or count out of range, or a row named twice
    PST_TABLE = 256u,  // a page number out of range
    PST_SHARED = 512u  // an append to a page that several rows hold
};

// Pool geometry and pointers, passed to every kernel by value.
struct PagesView {
    int n_layers, n_pages, P, Hkv, Hq, G, d, max_seqs, M;
    int bf16;             // dtype: 1 bf16, 0 fp16
    int blk;              // tokens per block, min(P, 64)
    int page_bytes;       // of one KV head
    int sum_bytes;
    int k_exp, v_exp;
    uint8_t *pages;       // the layer's first page (append .. select), or the pool's
    uint8_t *summary;
    int *table, *seq_len, *refs;
    unsigned *status;
};

constexpr unsigned long long PAGES_WAIT_NS = 2000000000ull;  // a healthy wait is over in microseconds

// Which rows and new tokens a call is about.
struct PagesRows {
    const int *rows, *cu;
    int n_rows, n_tok, max_new;
};

constexpr int PAGES_SELECT_MAX = 16384;  // pages of a row that a choice is made among (a key of each in shared memory)

// The int part of the workspace: [0] copies or moves of the last plan, [1] live pages
// below which moves end, then three lists of n_pages.
constexpr int PAGES_WS_HEAD = 16;
// Behind it, attention: CTAs of a launch (one per SM), and the floats of a record of 256
// query rows with head_dim 128 (accumulators, maximum and sum).
constexpr int PAGES_MAX_CTAS = 160;
constexpr int PAGES_REC_FLOATS = 256 * (128 + 2);
inline size_t pages_ws_lists(int n_pages) {  // bytes of the lists, a multiple of 16
    return (PAGES_WS_HEAD * 4 + 12 * static_cast<size_t>(n_pages) + 15) / 16 * 16;
}
inline size_t pages_ws_bytes(int n_pages) {
    return pages_ws_lists(n_pages) + PAGES_MAX_CTAS * 20 + static_cast<size_t>(PAGES_MAX_CTAS) * 2 * PAGES_REC_FLOATS * 4;
}

struct PagesStoreArgs {
    PagesView p;
    PagesRows r;
    const uint16_t *k, *v;
    long long kt, kh, vt, vh;
};
struct PagesReadArgs {
    PagesView p;
    PagesRows r;
    uint16_t *k, *v;
};
struct PagesAttnArgs {
    PagesView p;
    PagesRows r;
    const uint16_t *q;
    long long qt, qh;
    uint16_t *out;
    float *lse;
    const int *sel;
    int n_sel;
    int over, most;       // this launch takes the rows with over < n G <= most query rows for each KV head
    float scale_log2;     // sm_scale 2^k_exp log2(e)
    float out_scale;      // 2^v_exp
    int *tickets;         // workspace: [PAGES_MAX_CTAS], 0 between calls
    int *joins;           // workspace: [PAGES_MAX_CTAS][4], what the tensor-core kernel leaves to be joined
    float *records;       // workspace: [PAGES_MAX_CTAS][2][PAGES_REC_FLOATS]
    unsigned long long wait_ns;  // longest wait on a barrier
    unsigned owed;        // arrivals that barriers wait for and nobody makes: 0 but in tests of waits that run out
};
struct PagesSelectArgs {
    PagesView p;
    PagesRows r;
    const uint16_t *q;
    long long qt, qh;
    int *sel;
    int n_sel, keep_first, keep_last;
};

// launchers (return cudaError_t as int)
int launch_pages_resize(const PagesView &p, const int *rows, const int *lens, int n, int *ws, int num_sms, void *stream);
int launch_pages_clear(unsigned *status, unsigned bits, void *stream);
int launch_pages_fork(const PagesView &p, const int *src, const int *dst, int n, void *stream);
int launch_pages_compact(const PagesView &p, int *ws, int num_sms, void *stream);
int launch_pages_append(const PagesStoreArgs &a, void *stream);
int launch_pages_read(const PagesReadArgs &a, void *stream);
int launch_pages_attention(PagesAttnArgs a, int num_sms, void *stream);
// many new tokens: the tensor-core kernel on at most `grid` CTAs
int launch_pages_prompt(const PagesAttnArgs &a, int grid, void *stream);
int launch_pages_select(const PagesSelectArgs &a, int num_sms, void *stream);

}  // namespace dq
