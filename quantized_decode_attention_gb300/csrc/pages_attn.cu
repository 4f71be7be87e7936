// Paged cache: attention's launches, and the kernel for few new tokens as attention and
// cross attention take it.
#include "pages_attn.cuh"

namespace dq {
namespace {

// Query rows of a row and KV head beyond which the tensor-core kernel takes over (8 rows of 32768 tokens, 4 query
// heads a KV head; this kernel against that: 16 query rows 88 / 237 us, 32 160 / 237, 48 232 / 237, 64 304 / 237).
constexpr int PROMPT_ROWS = 32;

}  // namespace

int launch_pages_attention(PagesAttnArgs a, int mode, int num_sms, void *stream) {
    const int grid = num_sms < PAGES_MAX_CTAS ? num_sms : PAGES_MAX_CTAS;
    const int rows = a.r.max_new * a.p.G;
    a.over = 0;
    a.most = 0x7fffffff;
    if (!a.sel && rows > PROMPT_ROWS) {
        // rows with many new tokens on the tensor cores; those of a mixed batch with few, which wait
        // for the cache and not for products, by the kernel for few (one row alone: no second launch)
        a.over = a.r.n_rows == 1 ? 0 : PROMPT_ROWS;
        if (const int e = launch_pages_prompt(a, mode, grid, stream)) return e;
        if (a.r.n_rows == 1) return 0;
        a.over = 0;
        a.most = PROMPT_ROWS;
    }
    switch (mode) {
        case PAGES_NEWEST: return launch_few<PAGES_NEWEST>(a, grid, stream);
        case PAGES_ALL: return launch_few<PAGES_ALL>(a, grid, stream);
        default: return launch_pages_few_shared(a, mode, grid, stream);
    }
}

int launch_pages_shared(const PagesAttnArgs &a, int n_groups, int max_group, int num_sms, void *stream) {
    PagesAttnArgs c = a;
    c.r.n_rows = n_groups;
    c.r.max_new = max_group;
    if (const int e = launch_pages_attention(c, PAGES_COMMON, num_sms, stream)) return e;
    return launch_pages_attention(a, PAGES_OWN, num_sms, stream);
}

}  // namespace dq
