// Paged cache: what the rows of a group have in common, read off their tables.
//
// A page is common where every row's table names the same page at the same ordinal and
// every new token of every row sees all of it: ordinals below (len - n) / P of the
// shortest.  One CTA a group: the warps take its rows in turn and look for the first
// ordinal that differs from the leader's, up to the least that any has found so far.
// Bound by latency (64 rows that share 128 pages: 4.2 us, 8 that share 31: 2.9; once for all layers).
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr float BYTES_US = 5e6f, UNIT_US = 1.9f, COST_US = 20.f, SMS = 152.f;
constexpr int CO_THREADS = 1024, CO_WARPS = CO_THREADS / 32;

// Whether a group's `keys` common tokens, for `rows` rows with `tokens` new ones, are worth a launch of their own: the
// time of each row's reading them (the cache at 5 TB/s; for many query rows the products, 1.9 us a unit of 256 query
// rows and 128 keys on an SM), less that of one reading, against the launch's and the join's, which the groups share.
// A choice of speed alone: it takes all groups to be like this one.  Measured, attention with nothing common / in
// common, us (8 KV heads of 128, 4 query heads each): 8 rows behind 2048 tokens 17.3 / 22.2, 8192 25.8 / 29.4, 32768
// 61 / 53.5; 64 rows behind 512 21.8 / 27.2, 1024 28.7 / 27.4, 2048 42.8 / 28.8, 8192 112 / 38; 8 groups of 8 behind
// 512 19.7 / 19.7, 2048 40.6 / 37.7, 8192 110 / 87; rows of 16 tokens: 4 behind 8192 45 / 55.6, 8 behind 2048
// 36.5 / 54, 32 behind 2048 80 / 70, 16384 383 / 154.
__device__ __forceinline__ bool pays(const PagesCommonArgs &a, int rows, int tokens, int keys) {
    const PagesView &p = a.p;
    const float q = static_cast<float>(tokens) * p.G, heads = static_cast<float>(p.Hkv) * keys;  // query rows; keys of all heads
    float saved;  // us
    if (q <= 32.f * rows) saved = (rows - 1) * heads * (p.d * 9 / 8) / BYTES_US;
    else saved = (rows * ceilf(q / rows / 256.f) - ceilf(q / 256.f)) * (heads / 128.f) * UNIT_US / SMS;
    return saved * a.n_groups > COST_US;
}

__global__ void __launch_bounds__(CO_THREADS) common_kernel(PagesCommonArgs a) {
    __shared__ int least, leader, count, tokens, row_s[DQ_PAGES_MAX_ROWS];
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
        count = tokens = 0;
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
            atomicAdd(&tokens, r.n);
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
    const bool share = count > 1 && (a.always || pays(a, count, tokens, least * p.P));
    const int2 what = share ? make_int2(least * p.P, first) : make_int2(0, 0);
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
