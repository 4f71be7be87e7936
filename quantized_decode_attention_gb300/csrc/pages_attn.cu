// Paged cache: attention's launches, and the kernel for few new tokens as attention and
// cross attention take it.
#include "pages_attn.cuh"

namespace dq {
namespace {

// Query rows of a row and KV head beyond which the tensor-core kernel takes over (8 rows of 32768 tokens, 4 query
// heads a KV head: 16 query rows 88 us, 32 160, 48 232, 64 304; that kernel 200 at up to 128).
constexpr int PROMPT_ROWS = 32;
// Groups of rows from which those with few query rows have a launch over their common pages beside one group with many (fewer only
// where all have few on average).  Such a launch / all in the one for many, us: 64 rows behind 4096 tokens and one group of 8 behind
// 2048 51 / 34, 4 groups of 2 behind 8192 84 / 73, 8 of 4 behind 8192 81 / 137, 8 of 2 behind 16384 98 / 238, 8 of 3 behind 32768
// 134 / 650.
constexpr int SOME_GROUPS = 4;

}  // namespace

// Attention's launches of one kind; mixed: rows with few query rows have a launch of their own.
static int launch_kind(PagesAttnArgs a, int mode, bool mixed, int num_sms, void *stream) {
    const int grid = num_sms < PAGES_MAX_CTAS ? num_sms : PAGES_MAX_CTAS;
    a.over = 0;
    a.most = 0x7fffffff;
    if (!a.sel && a.r.max_new * a.p.G > PROMPT_ROWS) {
        // rows with many new tokens on the tensor cores; those of a mixed batch with few, which wait
        // for the cache and not for products, by the kernel for few (one row alone: no second launch)
        a.over = mixed ? PROMPT_ROWS : 0;
        if (const int e = launch_pages_prompt(a, mode, grid, stream)) return e;
        if (!mixed) return 0;
        a.after_few = 0;
        a.over = 0;
        a.most = PROMPT_ROWS;
    }
    switch (mode) {
        case PAGES_NEWEST: return launch_few<PAGES_NEWEST>(a, grid, stream);
        case PAGES_ALL: return launch_few<PAGES_ALL>(a, grid, stream);
        default: return launch_pages_few_shared(a, mode, grid, stream);
    }
}

int launch_pages_attention(const PagesAttnArgs &a, int mode, int num_sms, void *stream) {
    return launch_kind(a, mode, mode == PAGES_ALL ? few_beside_most(a.r, a.p.G, PROMPT_ROWS) : a.r.n_rows > 1, num_sms, stream);
}

// The launch over the rows' own pages, then the one over what groups have in common.
int launch_pages_shared(const PagesAttnArgs &a, int n_groups, int max_group, int num_sms, void *stream) {
    const bool few = a.r.max_new * a.p.G <= PROMPT_ROWS || few_beside_most(a.r, a.p.G, PROMPT_ROWS);
    if (const int e = launch_kind(a, PAGES_OWN, few, num_sms, stream)) return e;
    PagesAttnArgs c = a;
    c.own_max_new = a.r.max_new;
    c.after_few = few;
    c.r.n_rows = n_groups;
    c.r.max_new = max_group;
    const bool few_all = n_groups > 1 && static_cast<long long>(a.r.n_tok) * a.p.G <= static_cast<long long>(PROMPT_ROWS) * n_groups;
    return launch_kind(c, PAGES_COMMON, few_all || (n_groups > SOME_GROUPS && few_beside_most(c.r, c.p.G, PROMPT_ROWS)), num_sms, stream);
}

}  // namespace dq
