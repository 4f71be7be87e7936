// Paged cache: what the rows of a group have in common, read off their tables.
//
// A page is common where every row's table names the same page at the same ordinal and
// every new token of every row sees all of it: ordinals below (len - n) / P of the
// shortest.  One CTA a group: the warps take its rows in turn and look for the first
// ordinal that differs from the leader's, up to the least that any has found so far.
// Then, where there are several groups, the choice of those that are worth it, by a CTA of its own.
// Bound by latency (64 rows that share 128 pages: 4.1 us, 8 that share 31: 2.9; 8 groups of 8 that share 128: 4.7, the choice 1.3 of
// them; once for all layers).
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr float BYTES_US = 5e6f, UNIT_US = 1.9f, COST_US = 20.f, GROUP_US = 1.5f;
constexpr int CO_THREADS = 1024, CO_WARPS = CO_THREADS / 32;

// What one reading of a group's `keys` common tokens saves, in us, for `rows` rows with `tokens` new ones: the time of each
// row's reading them (the cache at 5 TB/s; for many query rows the products, 1.9 us a unit of 256 query rows and 128 keys on
// an SM), less that of one reading.
__device__ __forceinline__ float saved_us(const PagesCommonArgs &a, int rows, int tokens, int keys) {
    const PagesView &p = a.p;
    const float q = static_cast<float>(tokens) * p.G, heads = static_cast<float>(p.Hkv) * keys;  // query rows; keys of all heads
    if (q <= 32.f * rows) return (rows - 1) * heads * (p.d * 9 / 8) / BYTES_US;
    return (rows * ceilf(q / rows / 256.f) - ceilf(q / 256.f)) * (heads / 128.f) * UNIT_US / a.num_sms;
}

// Which groups' common pages are taken, a choice of speed alone: all together save more than the launch over them and its join
// cost, COST_US, and each more than its own place there, GROUP_US (or less, where as many like it as there are would pay for the
// launch).  Measured, with nothing common / in common, us (8 KV heads of 128, 4 query heads each, rows of 64 tokens of
// their own): 8 rows behind 2048 tokens 17.3 / 22.5, 8192 26.4 / 29.7, 32768 62 / 53.5; 64 rows behind 512 21.9 / 27.8, 1024 29.1 / 28.0,
// 2048 43.2 / 29.0, 8192 113 / 38.7; 8 groups of 8 behind 512 19.7 / 19.9, 2048 41.1 / 38.5, 8192 112 / 88; rows of 16 tokens: 4 behind
// 8192 44.5 / 55.2, 8 behind 2048 36.5 / 54.6, 32 behind 2048 80.9 / 71.0, 16384 381 / 156.  Beside 64 rows behind 4096, one group of 4
// behind 2048 (1.4 us) apart 30.0 / in common 32.5, 8 behind 1024 (1.7) 30.8 / 34.0, 8 behind 2048 (3.3) 41.0 / 33.3, 16 behind 1024 (3.5)
// 40.0 / 34.0; 2 behind 16384 (3.8) 44.5 / 49.2, whose products are more than what is read.  13 behind 1488 and 4 behind 5184 beside them
// 46.2 / 37.2; 8 ragged groups of 4 KV heads, two of which save 1.8 and 2.1 us, 54.6 / 53.1.
struct Choice {
    float sum;   // of the groups that are worth their place
    int n;       // groups that have something in common
    __device__ __forceinline__ bool worth(float us) const { return us > GROUP_US || us * n > COST_US; }
    __device__ __forceinline__ bool takes(float us) const { return sum > COST_US && worth(us); }
};

__global__ void __launch_bounds__(CO_THREADS) common_kernel(PagesCommonArgs a) {
    __shared__ int least, leader, count, tokens, row_s[DQ_PAGES_MAX_ROWS];
    const PagesView &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_rows = a.r.n_rows;
    let_next_start();
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
    const float us = count > 1 ? saved_us(a, count, tokens, least * p.P) : 0.f;
    const bool share = count > 1 && (a.always || a.n_groups > 1 || Choice{us, 1}.takes(us));
    const int2 what = share ? make_int2(least * p.P, first) : make_int2(0, 0);
    // (where the groups' choice is still to come, the group's second place has what it saves)
    for (int i = g0 + tid; i < g1; i += CO_THREADS)
        plan[i] = i == g0 + 1 && !a.always && a.n_groups > 1 ? make_int2(__float_as_int(us), 0) : what;
    // rows of the call that are in no group
    if (blockIdx.x == 0)
        for (int i = tid; i < g0; i += CO_THREADS) plan[i] = make_int2(0, 0);
    if (blockIdx.x == gridDim.x - 1)
        for (int i = g1 + tid; i < n_rows; i += CO_THREADS) plan[i] = make_int2(0, 0);
}

// Several groups: the choice among them, from what each saves.  One CTA, a thread a group, then a warp a group.
__global__ void __launch_bounds__(CO_THREADS) choose_kernel(PagesCommonArgs a) {
    __shared__ float us_s[DQ_PAGES_MAX_ROWS], part[CO_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int2 *plan = reinterpret_cast<int2 *>(a.plan);
    await_previous();
    auto bounds = [&](int g, int &g0, int &g1) {  // false: out of order, or of a single place
        g0 = a.groups[g];
        g1 = a.groups[g + 1];
        return g0 >= 0 && g1 <= a.r.n_rows && g1 - g0 > 1;
    };
    int g0, g1;
    float us = 0.f;
    if (tid < a.n_groups && bounds(tid, g0, g1) && plan[g0].x > 0) us = __int_as_float(plan[g0 + 1].x);
    us_s[tid] = us;
    Choice c{0.f, __syncthreads_count(us > 0.f)};
    float sum = c.worth(us) ? us : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    for (int w = 0; w < CO_WARPS; w++) c.sum += part[w];
    for (int g = warp; g < a.n_groups; g += CO_WARPS) {
        if (!bounds(g, g0, g1)) continue;
        const int2 what = c.takes(us_s[g]) ? plan[g0] : make_int2(0, 0);
        __syncwarp();
        for (int i = g0 + lane; i < g1; i += 32) plan[i] = what;
    }
}

}  // namespace

int launch_pages_common(const PagesCommonArgs &a, void *stream) {
    static_assert(CO_THREADS >= DQ_PAGES_MAX_ROWS, "a thread a group");
    auto st = static_cast<cudaStream_t>(stream);
    common_kernel<<<a.n_groups, CO_THREADS, 0, st>>>(a);
    if (const cudaError_t e = cudaGetLastError()) return static_cast<int>(e);
    return a.always || a.n_groups == 1 ? 0 : launch_overlapping(choose_kernel, dim3(1), CO_THREADS, 0, st, a);
}

}  // namespace dq
