// Paged cache: lengths, forks and compaction.  One CTA plans (it alone changes the
// tables, counts and lengths, so that the outcome does not depend on timing) and a
// second kernel copies the pages that the plan names, in every layer.
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr int MV_THREADS = 1024, MV_WARPS = MV_THREADS / 32;

// Exclusive prefix of v over the CTA; `total` gets the sum.  `part` holds MV_WARPS + 1 ints.
__device__ int block_prefix(int v, int *part, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(FULL, s, o);
        if (lane >= o) s += t;
    }
    __syncthreads();
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        const int w = part[lane];
        int t = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(FULL, t, o);
            if (lane >= o) t += u;
        }
        part[lane] = t - w;
        if (lane == 31) part[32] = t;
    }
    __syncthreads();
    total = part[32];
    return part[warp] + s - v;
}

__device__ __forceinline__ int pages_for(int len, int P) { return (len + P - 1) / P; }

// Whether the page number is one of the pool's.
__device__ __forceinline__ bool page_ok(const PagesView &p, int id) {
    if (id >= 0 && id < p.n_pages) return true;
    atomicOr(p.status, PST_TABLE);
    return false;
}

// A plan's copies may be launched while it runs; they wait for its end before they read
// anything (the hardware's dependency between launches of one stream).
__device__ __forceinline__ void let_copies_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void await_plan() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

__global__ void __launch_bounds__(MV_THREADS) resize_kernel(PagesView p, const int *rows, const int *lens, int n, int *ws) {
    __shared__ unsigned seen[DQ_PAGES_MAX_ROWS / 32];
    __shared__ int part[MV_WARPS + 1], bad, found;
    __shared__ int row_s[DQ_PAGES_MAX_ROWS], had_s[DQ_PAGES_MAX_ROWS], has_s[DQ_PAGES_MAX_ROWS], page_s[DQ_PAGES_MAX_ROWS],
        first_s[DQ_PAGES_MAX_ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *list = ws + PAGES_WS_HEAD, *src = list + p.n_pages, *dst = src + p.n_pages;
    let_copies_start();
    if (tid == 0) {
        bad = found = 0;
        ws[0] = 0;
    }
    for (int i = tid; i < DQ_PAGES_MAX_ROWS / 32; i += MV_THREADS) seen[i] = 0;
    __syncthreads();
    // entry tid of the list (n <= MV_THREADS)
    int row = -1, before = 0, after = 0;
    if (tid < n) {
        row = rows ? rows[tid] : tid;
        if (row >= 0) {
            after = lens[tid];
            if (row >= p.max_seqs || after < 0 || after > p.M * p.P) bad = 1;
            else {
                if (atomicOr(&seen[row >> 5], 1u << (row & 31)) >> (row & 31) & 1u) bad = 1;
                before = p.seq_len[row];
                if (before < 0 || before > p.M * p.P) bad = 1;
            }
        }
    }
    __syncthreads();
    if (bad) {
        if (tid == 0) atomicOr(p.status, PST_ARG);
        return;
    }
    const int had = row >= 0 ? pages_for(before, p.P) : 0, has = row >= 0 ? pages_for(after, p.P) : 0;
    row_s[tid] = row;
    had_s[tid] = had;
    has_s[tid] = has;
    page_s[tid] = -1;
    __syncthreads();
    // pages behind the new lengths lose a reference (given back below if the call fails)
    for (int i = warp; i < n; i += MV_WARPS)
        for (int j = has_s[i] + lane; j < had_s[i]; j += 32) {
            const int id = p.table[static_cast<long long>(row_s[i]) * p.M + j];
            if (page_ok(p, id)) atomicSub(&p.refs[id], 1);
        }
    __syncthreads();
    int page = -1;
    if (row >= 0 && after > before && before % p.P) {
        page = p.table[static_cast<long long>(row) * p.M + before / p.P];
        if (!page_ok(p, page)) page = -1;
    }
    page_s[tid] = page;
    __syncthreads();
    bool copy = false;
    if (page >= 0) {
        int earlier = 0;
        for (int i = 0; i < tid; i++) earlier += page_s[i] == page;
        copy = p.refs[page] - earlier > 1;
    }
    const int need = (copy ? 1 : 0) + (has > had ? has - had : 0);
    int total, n_copy;
    const int first = block_prefix(need, part, total);
    first_s[tid] = first;
    const int at_copy = block_prefix(copy ? 1 : 0, part, n_copy);
    // the lowest `total` free pages
    for (int i0 = 0; i0 < p.n_pages && found < total; i0 += MV_THREADS) {
        const int i = i0 + tid, f = i < p.n_pages && p.refs[i] == 0;
        int some;
        const int at = found + block_prefix(f, part, some);
        if (f && at < total) list[at] = i;
        __syncthreads();
        if (tid == 0) found += some;
        __syncthreads();
    }
    if (found < total) {
        for (int i = warp; i < n; i += MV_WARPS)
            for (int j = has_s[i] + lane; j < had_s[i]; j += 32) {
                const int id = p.table[static_cast<long long>(row_s[i]) * p.M + j];
                if (id >= 0 && id < p.n_pages) atomicAdd(&p.refs[id], 1);
            }
        if (tid == 0) atomicOr(p.status, PST_FULL);
        return;
    }
    for (int i = tid; i < total; i += MV_THREADS) p.refs[list[i]] = 1;
    if (copy) {
        atomicSub(&p.refs[page], 1);
        src[at_copy] = page;
        dst[at_copy] = list[first];
        p.table[static_cast<long long>(row) * p.M + before / p.P] = list[first];
        first_s[tid] = first + 1;
    }
    if (row >= 0) p.seq_len[row] = after;
    if (tid == 0) ws[0] = n_copy;
    __syncthreads();
    for (int i = warp; i < n; i += MV_WARPS) {
        int *t = p.table + static_cast<long long>(row_s[i]) * p.M;
        for (int j = has_s[i] + lane; j < had_s[i]; j += 32) t[j] = -1;
        for (int j = had_s[i] + lane; j < has_s[i]; j += 32) t[j] = list[first_s[i] + j - had_s[i]];
    }
}

__global__ void __launch_bounds__(MV_THREADS) fork_kernel(PagesView p, const int *src, const int *dst, int n) {
    __shared__ unsigned is_dst[DQ_PAGES_MAX_ROWS / 32];
    __shared__ int bad, src_s[DQ_PAGES_MAX_ROWS], dst_s[DQ_PAGES_MAX_ROWS], len_s[DQ_PAGES_MAX_ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad = 0;
    for (int i = tid; i < DQ_PAGES_MAX_ROWS / 32; i += MV_THREADS) is_dst[i] = 0;
    __syncthreads();
    int s = -1, d = -1;
    if (tid < n) {
        s = src[tid];
        d = dst[tid];
        if (s < 0 || d < 0) s = d = -1;
    }
    if (d >= 0) {
        if (s >= p.max_seqs || d >= p.max_seqs) bad = 1;
        else {
            if (atomicOr(&is_dst[d >> 5], 1u << (d & 31)) >> (d & 31) & 1u) bad = 1;
            const int len = p.seq_len[s];
            if (p.seq_len[d] != 0 || len < 0 || len > p.M * p.P) bad = 1;
            len_s[tid] = len;
        }
    }
    src_s[tid] = s;
    dst_s[tid] = d;
    __syncthreads();
    if (d >= 0 && !bad && (is_dst[s >> 5] >> (s & 31) & 1u)) bad = 1;
    __syncthreads();
    if (bad) {
        if (tid == 0) atomicOr(p.status, PST_ARG);
        return;
    }
    for (int i = warp; i < n; i += MV_WARPS) {
        if (dst_s[i] < 0) continue;
        const int *from = p.table + static_cast<long long>(src_s[i]) * p.M;
        int *to = p.table + static_cast<long long>(dst_s[i]) * p.M;
        for (int j = lane; j < pages_for(len_s[i], p.P); j += 32) {
            const int id = from[j];
            to[j] = id;
            if (page_ok(p, id)) atomicAdd(&p.refs[id], 1);
        }
        if (lane == 0) p.seq_len[dst_s[i]] = len_s[i];
    }
}

// n = live pages; src: live pages numbered n or more, dst: free numbers below n, both
// ascending (there are as many of each); map[src] = dst.
__global__ void __launch_bounds__(MV_THREADS) compact_kernel(PagesView p, int *ws) {
    __shared__ int part[MV_WARPS + 1], n_src, n_dst;
    const int tid = threadIdx.x;
    int *map = ws + PAGES_WS_HEAD, *src = map + p.n_pages, *dst = src + p.n_pages;
    let_copies_start();
    if (tid == 0) n_src = n_dst = 0;
    __syncthreads();
    int mine = 0;
    for (int i = tid; i < p.n_pages; i += MV_THREADS) mine += p.refs[i] > 0;
    int total;
    block_prefix(mine, part, total);
    for (int i0 = 0; i0 < p.n_pages; i0 += MV_THREADS) {
        const int i = i0 + tid;
        const int in = i < p.n_pages, used = in && p.refs[i] > 0;
        const int s = used && i >= total, d = in && !used && i < total;
        int ts, td;
        const int as = n_src + block_prefix(s, part, ts), ad = n_dst + block_prefix(d, part, td);
        if (s) src[as] = i;
        if (d) dst[ad] = i;
        __syncthreads();
        if (tid == 0) {
            n_src += ts;
            n_dst += td;
        }
        __syncthreads();
    }
    for (int i = tid; i < n_src; i += MV_THREADS) {
        map[src[i]] = dst[i];
        p.refs[dst[i]] = p.refs[src[i]];
        p.refs[src[i]] = 0;
    }
    if (tid == 0) {
        ws[0] = n_src;
        ws[1] = total;
    }
}

// Copy the planned pages and summaries of every layer.  A layer's page (all heads, then
// its summaries) goes in slices of 16 KB, so that a few copies fill the card as evenly
// as many do; a thread has four 16-byte loads on their way before it stores.  What the
// plan names is disjoint: a destination was free.
constexpr int CP_THREADS = 256, CP_DEEP = 4, CP_SLICE = CP_THREADS * CP_DEEP;
// REMAP: the plan is a compaction; the table entries of moved pages follow (map[src] = dst), a row a CTA.
template <bool REMAP>
__global__ void __launch_bounds__(CP_THREADS) copy_kernel(PagesView p, const int *ws) {
    await_plan();
    const int n = ws[0];
    if (n == 0) return;
    if (REMAP) {
        const int *map = ws + PAGES_WS_HEAD, live = ws[1];
        for (int i = blockIdx.x; i < p.max_seqs; i += gridDim.x) {
            int len = p.seq_len[i];
            if (len < 0 || len > p.M * p.P) len = 0;
            int *t = p.table + static_cast<long long>(i) * p.M;
            for (int j = threadIdx.x; j < pages_for(len, p.P); j += CP_THREADS) {
                const int id = t[j];
                if (page_ok(p, id) && id >= live) t[j] = map[id];
            }
        }
    }
    const int *src = ws + PAGES_WS_HEAD + p.n_pages, *dst = src + p.n_pages;
    const int pb = p.Hkv * p.page_bytes / 16, sb = p.Hkv * p.sum_bytes / 16;  // 16-byte words of a page, of its summaries
    const int slices = (pb + sb + CP_SLICE - 1) / CP_SLICE;
    const long long items = static_cast<long long>(n) * p.n_layers * slices;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const long long u = it / slices;
        const int m = static_cast<int>(u / p.n_layers), w0 = static_cast<int>(it - u * slices) * CP_SLICE + threadIdx.x;
        const long long base = (u - static_cast<long long>(m) * p.n_layers) * p.n_pages, from = base + src[m], to = base + dst[m];
        const uint4 *ap = reinterpret_cast<const uint4 *>(p.pages) + from * pb, *as = reinterpret_cast<const uint4 *>(p.summary) + from * sb - pb;
        uint4 *bp = reinterpret_cast<uint4 *>(p.pages) + to * pb, *bs = reinterpret_cast<uint4 *>(p.summary) + to * sb - pb;
        uint4 v[CP_DEEP];
#pragma unroll
        for (int k = 0; k < CP_DEEP; k++) {
            const int w = w0 + k * CP_THREADS;
            if (w < pb + sb) v[k] = __ldcs((w < pb ? ap : as) + w);
        }
#pragma unroll
        for (int k = 0; k < CP_DEEP; k++) {
            const int w = w0 + k * CP_THREADS;
            if (w < pb + sb) __stcs((w < pb ? bp : bs) + w, v[k]);
        }
    }
}

}  // namespace

static int launch_copies(void (*kernel)(PagesView, const int *), const PagesView &p, const int *ws, int num_sms, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(6 * num_sms);
    cfg.blockDim = dim3(CP_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, p, ws));
}

int launch_pages_resize(const PagesView &p, const int *rows, const int *lens, int n, int *ws, int num_sms, void *stream) {
    auto st = static_cast<cudaStream_t>(stream);
    resize_kernel<<<1, MV_THREADS, 0, st>>>(p, rows, lens, n, ws);
    const int e = static_cast<int>(cudaGetLastError());
    return e ? e : launch_copies(copy_kernel<false>, p, ws, num_sms, st);
}

int launch_pages_fork(const PagesView &p, const int *src, const int *dst, int n, void *stream) {
    fork_kernel<<<1, MV_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p, src, dst, n);
    return static_cast<int>(cudaGetLastError());
}

int launch_pages_compact(const PagesView &p, int *ws, int num_sms, void *stream) {
    auto st = static_cast<cudaStream_t>(stream);
    compact_kernel<<<1, MV_THREADS, 0, st>>>(p, ws);
    const int e = static_cast<int>(cudaGetLastError());
    return e ? e : launch_copies(copy_kernel<true>, p, ws, num_sms, st);
}

}  // namespace dq
