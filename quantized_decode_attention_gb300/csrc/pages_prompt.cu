// Paged cache: the kernel for many new tokens as attention and cross attention take it.
#include "pages_prompt.cuh"

namespace dq {

int launch_pages_prompt(const PagesAttnArgs &a, int mode, int grid, void *stream) {
    switch (mode) {
        case PAGES_NEWEST: return launch_many<PAGES_NEWEST>(a, grid, stream);
        case PAGES_ALL: return launch_many<PAGES_ALL>(a, grid, stream);
        default: return launch_pages_prompt_shared(a, mode, grid, stream);
    }
}

}  // namespace dq
