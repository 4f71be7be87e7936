// Paged cache: the kernel for many new tokens as shared attention takes it, over what is behind the
// pages that groups of rows have in common, and over those.
#include "pages_prompt.cuh"

namespace dq {

int launch_pages_prompt_shared(const PagesAttnArgs &a, int mode, int grid, void *stream) {
    return mode == PAGES_COMMON ? launch_many<PAGES_COMMON>(a, grid, stream) : launch_many<PAGES_OWN>(a, grid, stream);
}

}  // namespace dq
