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
    PST_SHARED = 512u  // an append or an eviction to a page that several rows hold
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

// Whether rows with few query rows (`few` at most, tokens times G) are likely beside those with many, so that they are worth a
// launch of their own: few on average in all rows but one that has as many tokens as a row may have.  With such a launch / all in the
// one for many, us: 16 rows of 1 token over 32768 beside one of 2048: weights 530 / 1632, cross 941 / 1151; 4 rows of 64 over 16384,
// where it has nothing to do: weights 57.8 / 54.2, cross 71.8 / 71.0, shared 82.4 / 78.0; 3 rows of 2 over 8192 beside one of 64, where
// each of the launches is short: weights 26.7 / 41.6, cross 56.1 / 44.4.
inline bool few_beside_most(const PagesRows &r, int G, int few) {
    return r.n_rows > 1 && (static_cast<long long>(r.n_tok) - r.max_new) * G <= static_cast<long long>(few) * (r.n_rows - 1);
}

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
// Then tickets and records (of 16 query rows) of its own for the launch of shared attention over the rows' own pages, which
// begins while the one over the common pages still runs.
constexpr int PAGES_OWN_REC_FLOATS = 16 * (128 + 2);
inline size_t pages_ws_own(int n_pages) {
    return pages_ws_lists(n_pages) + PAGES_MAX_CTAS * 20 + static_cast<size_t>(PAGES_MAX_CTAS) * 2 * PAGES_REC_FLOATS * 4;
}
inline size_t pages_ws_bytes(int n_pages) {
    return pages_ws_own(n_pages) + PAGES_MAX_CTAS * 4 + static_cast<size_t>(PAGES_MAX_CTAS) * 2 * PAGES_OWN_REC_FLOATS * 4;
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
constexpr int FEW_UNIT_COST = 2;  // the kernel for few tokens: chunks that a unit's beginning and end are worth
// Which queries an attention launch answers, over which of a row's tokens: a constant of each kernel
// (as a variable it costs attention of single tokens 7 %).
enum : int {
    PAGES_NEWEST = 0,  // the call's rows' newest tokens, over what they hold up to them
    PAGES_ALL = 1,     // queries of the call's rows, over all they hold
    PAGES_OWN = 2,     // the call's rows' newest tokens, over what is behind the pages that their groups have in common: parts
    PAGES_COMMON = 3   // the tokens of groups of rows, over those pages, and the parts with it
};
struct PagesAttnArgs {
    PagesView p;
    PagesRows r;          // (PAGES_COMMON: of the groups)
    const int *groups;    // where each group begins among call_rows rows (NULL: one group of all)
    const int *plan;      // [call_rows][2]: tokens in common, the table row that they are read from
    int call_rows;
    int *own_tickets;     // workspace: of the launch over the rows' own pages
    float *own_records;
    // The parts of the queries whose group has pages in common: accumulators [n_tok Hq][d], then [n_tok Hq][2] maximum and
    // sum, a maximum of +inf where the row holds nothing.
    float *part;
    int own_max_new;      // PAGES_COMMON: max_new of the launch over the rows' own pages
    int after_few;        // the launch before this one is the kernel for few tokens, whose end need not be waited for at the start
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
struct PagesCommonArgs {
    PagesView p;
    PagesRows r;
    const int *groups;
    int n_groups;
    int always;           // also where it does not pay
    int num_sms;
    int *plan;
};
struct PagesWeighArgs {
    PagesView p;
    PagesRows r;
    const uint16_t *q;
    long long qt, qh;
    const float *lse;
    float *scores;        // [max_seqs][Hkv][cap] of the layer
    int cap;
    float scale_log2;
    int over, most;       // this launch takes the rows with over < n G <= most query rows for each KV head
    int *tickets;         // workspace, as attention has them
    float *records;       // workspace: [PAGES_MAX_CTAS][2][256]
    unsigned long long wait_ns;
    unsigned owed;        // as attention's
};
struct PagesEvictArgs {
    PagesView p;          // of the pool
    float *scores;        // [n_layers][max_seqs][Hkv][cap]
    int cap;
    const int *src, *dst;
    int n, keep_first, keep_last;
    int *keeps;           // workspace: [n], the tokens that each pair keeps, 0 for one that is refused
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
int launch_pages_attention(const PagesAttnArgs &a, int mode, int num_sms, void *stream);
int launch_pages_few_shared(const PagesAttnArgs &a, int mode, int grid, void *stream);
// many new tokens: the tensor-core kernel on at most `grid` CTAs
int launch_pages_prompt(const PagesAttnArgs &a, int mode, int grid, void *stream);
int launch_pages_prompt_shared(const PagesAttnArgs &a, int mode, int grid, void *stream);
int launch_pages_select(const PagesSelectArgs &a, int num_sms, void *stream);
int launch_pages_common(const PagesCommonArgs &a, void *stream);
int launch_pages_shared(const PagesAttnArgs &a, int n_groups, int max_group, int num_sms, void *stream);
int launch_pages_weigh(PagesWeighArgs a, int num_sms, void *stream);
// many query rows: the tensor-core kernel on at most `grid` CTAs
int launch_pages_weigh_many(const PagesWeighArgs &a, int grid, void *stream);
int launch_pages_evict(const PagesEvictArgs &a, int num_sms, void *stream);

}  // namespace dq
