// Paged cache: the kernel for few new tokens as shared attention takes it, over what is behind the
// pages that groups of rows have in common, and over those.
#include "pages_attn.cuh"

namespace dq {

int launch_pages_few_shared(const PagesAttnArgs &a, int mode, int grid, void *stream) {
    return mode == PAGES_COMMON ? launch_few<PAGES_COMMON>(a, grid, stream) : launch_few<PAGES_OWN>(a, grid, stream);
}

}  // namespace dq
