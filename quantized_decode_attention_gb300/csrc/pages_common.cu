// Paged cache: what the rows of a group have in common, read off their tables.
//
// A page is common where every row's table names the same page at the same ordinal and
// every new token of every row sees all of it: ordinals below (len - n) / P of the
// shortest.  One CTA a group: the warps take its rows in turn and look for the first
// ordinal that differs from the leader's, up to the least that any has found so far.
// Bound by latency (64 rows that share 128 pages: some 4 us, once for all layers).
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr int CO_THREADS = 512, CO_WARPS = CO_THREADS / 32;

__global__ void __launch_bounds__(CO_THREADS) common_kernel(PagesCommonArgs a) {
    __shared__ int least, leader, count, row_s[DQ_PAGES_MAX_ROWS];
    const PagesView &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_rows = a.r.n_rows;
    const int g0 = a.groups ? a.groups[blockIdx.x] : 0, g1 = a.groups ? a.groups[blockIdx.x + 1] : n_rows;
    int2 *plan = reinterpret_cast<int2 *>(a.plan);
    if (g0 < 0 || g1 > n_rows || g0 > g1) {
        if (tid == 0) atomicOr(p.status, PST_ARG);
        return;
    }
    if (tid == 0) {
        least = p.M;
        leader = n_rows;
        count = 0;
    }
    __syncthreads();
    // (places of the group that hold nothing or bring nothing do not count)
    for (int i = g0 + tid; i < g1; i += CO_THREADS) {
        const PageRow r = page_row(p, a.r, i);
        const bool is = r.row >= 0 && r.len > 0 && r.n > 0;
        row_s[i - g0] = is ? r.row : -1;
        if (is) {
            atomicMin(&least, r.len > r.n ? (r.len - r.n) / p.P : 0);
            atomicMin(&leader, i);
            atomicAdd(&count, 1);
        }
    }
    __syncthreads();
    const int first = leader < n_rows ? row_s[leader - g0] : 0;
    const int *mine = p.table + static_cast<long long>(first) * p.M;
    if (count > 1) {
        volatile int *end = &least;
        for (int i = warp; i < g1 - g0; i += CO_WARPS) {
            if (row_s[i] < 0 || row_s[i] == first) continue;
            const int *other = p.table + static_cast<long long>(row_s[i]) * p.M;
            for (int j = 0; j < *end; j += 128) {
                int at = p.M;  // the first of 4 x 32 ordinals that differs
#pragma unroll
                for (int k = 3; k >= 0; k--) {
                    const int o = j + 32 * k + lane;
                    if (o < p.M && mine[o] != other[o]) at = o;
                }
                at = __reduce_min_sync(FULL, at);
                if (at < p.M) {
                    if (lane == 0) atomicMin(&least, at);
                    break;
                }
            }
        }
        __syncthreads();
    }
    const int2 what = count > 1 ? make_int2(least * p.P, first) : make_int2(0, 0);
    for (int i = g0 + tid; i < g1; i += CO_THREADS) plan[i] = what;
    // rows of the call that are in no group
    if (blockIdx.x == 0)
        for (int i = tid; i < g0; i += CO_THREADS) plan[i] = make_int2(0, 0);
    if (blockIdx.x == gridDim.x - 1)
        for (int i = g1 + tid; i < n_rows; i += CO_THREADS) plan[i] = make_int2(0, 0);
}

}  // namespace

int launch_pages_common(const PagesCommonArgs &a, void *stream) {
    common_kernel<<<a.n_groups, CO_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace dq
