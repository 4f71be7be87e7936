// Paged cache: what the two kernels that weigh held tokens share: the call's rows.
#pragma once

#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {

constexpr float LOG2E = 1.4426950408889634f;

// The rows of the call that this launch weighs, in shared memory: keys_s is 0 for one that brings nothing or
// has its tokens weighed elsewhere, for one longer than the scores, and for one that is named twice (two
// warps would add to the same scores).  Then the line of all rows' work: `places(r)` of each.  All
// threads of a CTA of T.
template <int T, class F>
__device__ __forceinline__ long long weigh_rows(const PagesWeighArgs &a, int *row_s, int *keys_s, long long *first, long long *part, F places) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.r.n_rows;
    for (int i = tid; i < n; i += T) {
        const PageRow r = page_row(a.p, a.r, i);
        row_s[i] = r.row;
        keys_s[i] = r.n > 0 ? r.len : 0;
        if (keys_s[i] > a.cap) {
            atomicOr(a.p.status, PST_ARG);
            keys_s[i] = 0;
        }
    }
    __syncthreads();
    long long base = 0;
    for (int i0 = 0; i0 < n; i0 += T) {
        const int i = i0 + tid;
        long long w = 0;
        if (i < n && keys_s[i] > 0) {
            bool twice = false;
            if (a.r.rows)
                for (int k = 0; k < n; k++) twice |= row_s[k] == row_s[i] && k != i && (!a.r.cu || a.r.cu[k + 1] > a.r.cu[k]);
            PageRow r;
            r.len = keys_s[i];
            r.q0 = a.r.cu ? a.r.cu[i] : i;
            r.n = a.r.cu ? a.r.cu[i + 1] - r.q0 : 1;
            if (twice) atomicOr(a.p.status, PST_ARG);
            else if (r.n * a.p.G > a.over && r.n * a.p.G <= a.most) w = places(r);
        }
        long long s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(FULL, s, o);
            if (lane >= o) s += t;
        }
        if (lane == 31) part[warp] = s;
        __syncthreads();
        long long before = base;
        for (int k = 0; k < T / 32; k++) {
            const long long t = part[k];
            if (k < warp) before += t;
            base += t;
        }
        if (i < n) first[i] = before + s - w;
        __syncthreads();
    }
    if (tid == 0) first[n] = base;
    return base;
}

// The row whose work place x of the line is, and the row's number in the call.
__device__ __forceinline__ PageRow weigh_row_at(const PagesWeighArgs &a, const int *row_s, const int *keys_s, const long long *first, long long x, int &i) {
    int lo = 0, hi = a.r.n_rows - 1;
    while (lo < hi) {  // the last row that begins at or before x
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    i = lo;
    PageRow r;
    r.row = row_s[lo];
    r.len = keys_s[lo];
    r.from = 0;
    r.q0 = a.r.cu ? a.r.cu[lo] : lo;
    r.n = a.r.cu ? a.r.cu[lo + 1] - r.q0 : 1;
    return r;
}

__device__ __forceinline__ float *scores_of(const PagesWeighArgs &a, int row, int head) {
    return a.scores + (static_cast<long long>(row) * a.p.Hkv + head) * a.cap;
}

}  // namespace dq
