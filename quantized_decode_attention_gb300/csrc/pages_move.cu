// Paged cache: lengths, forks and compaction.  One CTA plans (it alone changes the
// tables, counts and lengths, so that the outcome does not depend on timing) and a
// second kernel copies the pages that the plan names, in every layer.  A plan looks 8192 counts
// up a turn: resize of 64 rows 5 us where the free pages are found at once, 13 where they are the
// last of 65536, 140 of 2^20; compaction 4 us of 4096 pages, 13 of 65536, 174 of 2^20.  Copies
// run at 6.3 TB/s (78 MB read and as much written in 25 us).
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr int MV_THREADS = 1024, MV_WARPS = MV_THREADS / 32;
constexpr int MV_FRESH = 1024;  // new pages of a call that are listed in shared memory

// Exclusive prefix of v over the CTA; `total` gets the sum.  `part` holds MV_WARPS + 1 values.
template <class T>
__device__ T block_prefix(T v, T *part, T &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T t = __shfl_up_sync(FULL, s, o);
        if (lane >= o) s += t;
    }
    __syncthreads();
    if (lane == 31) part[warp] = s;
    __syncthreads();
    // every warp adds the warps' sums up for itself
    const T w = part[lane];
    T t = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(FULL, t, o);
        if (lane >= o) t += u;
    }
    total = __shfl_sync(FULL, t, 31);
    return __shfl_sync(FULL, t - w, warp) + s - v;
}

// Which of the 8 pages from `base` on (a multiple of 8) are held; those past the pool are not.
__device__ __forceinline__ unsigned held8(const PagesView &p, int base) {
    unsigned m = 0;
    if (base + 8 <= p.n_pages) {
        const int4 a = *reinterpret_cast<const int4 *>(p.refs + base), b = *reinterpret_cast<const int4 *>(p.refs + base + 4);
        m = (a.x > 0) | (a.y > 0) << 1 | (a.z > 0) << 2 | (a.w > 0) << 3 | (b.x > 0) << 4 | (b.y > 0) << 5 | (b.z > 0) << 6 | (b.w > 0) << 7;
    } else {
        for (int i = 0; base + i < p.n_pages; i++) m |= (p.refs[base + i] > 0) << i;
    }
    return m;
}
__device__ __forceinline__ unsigned in_pool8(const PagesView &p, int base) {
    return base + 8 <= p.n_pages ? 0xffu : (base < p.n_pages ? (1u << (p.n_pages - base)) - 1u : 0u);
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
    __shared__ long long part[MV_WARPS];
    __shared__ int bad, found, fresh[MV_FRESH];
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
    // pages behind the new lengths lose a reference (given back below if the call fails)
    const bool drops = __syncthreads_or(has < had);
    if (drops) {
        for (int i = warp; i < n; i += MV_WARPS)
            for (int j = has_s[i] + lane; j < had_s[i]; j += 32) {
                const int id = p.table[static_cast<long long>(row_s[i]) * p.M + j];
                if (page_ok(p, id)) atomicSub(&p.refs[id], 1);
            }
        __syncthreads();
    }
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
    // places among the new pages and among the copies, in one prefix
    long long both;
    const long long at = block_prefix(static_cast<long long>(need) << 32 | (copy ? 1 : 0), part, both);
    const int first = static_cast<int>(at >> 32), at_copy = static_cast<int>(at), n_copy = static_cast<int>(both);
    if (both >> 32 > p.n_pages) {  // (more than there are at all)
        if (tid == 0) found = -1;
    }
    const int total = both >> 32 > p.n_pages ? p.n_pages + 1 : static_cast<int>(both >> 32);
    first_s[tid] = first;
    __syncthreads();
    // the lowest `total` free pages, 8 a thread at a time
    auto fresh_page = [&](int k) -> int { return k < MV_FRESH ? fresh[k] : list[k]; };
    for (int i0 = 0; i0 < p.n_pages && found >= 0 && found < total; i0 += 8 * MV_THREADS) {
        const int base = i0 + 8 * tid;
        unsigned f = base < p.n_pages ? in_pool8(p, base) & ~held8(p, base) : 0u;
        long long some;
        int k = found + static_cast<int>(block_prefix(static_cast<long long>(__popc(f)), part, some));
        for (; f && k < total; f &= f - 1, k++) {
            const int id = base + __ffs(f) - 1;
            if (k < MV_FRESH) fresh[k] = id;
            else list[k] = id;
        }
        __syncthreads();
        if (tid == 0) found += static_cast<int>(some);
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
    for (int i = tid; i < total; i += MV_THREADS) p.refs[fresh_page(i)] = 1;
    if (copy) {
        const int to = fresh_page(first);
        atomicSub(&p.refs[page], 1);
        src[at_copy] = page;
        dst[at_copy] = to;
        p.table[static_cast<long long>(row) * p.M + before / p.P] = to;
        first_s[tid] = first + 1;
    }
    if (row >= 0) p.seq_len[row] = after;
    if (tid == 0) ws[0] = n_copy;
    __syncthreads();
    for (int i = warp; i < n; i += MV_WARPS) {
        int *t = p.table + static_cast<long long>(row_s[i]) * p.M;
        for (int j = has_s[i] + lane; j < had_s[i]; j += 32) t[j] = -1;
        for (int j = had_s[i] + lane; j < has_s[i]; j += 32) t[j] = fresh_page(first_s[i] + j - had_s[i]);
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
    __shared__ int part[MV_WARPS], n_src, n_dst;
    const int tid = threadIdx.x;
    int *map = ws + PAGES_WS_HEAD, *src = map + p.n_pages, *dst = src + p.n_pages;
    let_copies_start();
    if (tid == 0) n_src = n_dst = 0;
    __syncthreads();
    int mine = 0;
    for (int i = 8 * tid; i < p.n_pages; i += 8 * MV_THREADS) mine += __popc(held8(p, i));
    int total;
    block_prefix(mine, part, total);
    for (int i0 = 0; i0 < p.n_pages; i0 += 8 * MV_THREADS) {
        const int base = i0 + 8 * tid;
        unsigned s = 0, d = 0;
        if (base < p.n_pages) {
            const unsigned held = held8(p, base);
            const unsigned below = base + 8 <= total ? 0xffu : (base < total ? (1u << (total - base)) - 1u : 0u);
            s = held & ~below;
            d = ~held & below;
        }
        int some;  // both counts in one prefix: at most 8192 each
        const int at = block_prefix(__popc(s) | __popc(d) << 16, part, some);
        int as = n_src + (at & 0xffff), ad = n_dst + (at >> 16);
        for (; s; s &= s - 1) src[as++] = base + __ffs(s) - 1;
        for (; d; d &= d - 1) dst[ad++] = base + __ffs(d) - 1;
        __syncthreads();
        if (tid == 0) {
            n_src += some & 0xffff;
            n_dst += some >> 16;
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

__global__ void clear_kernel(unsigned *status, unsigned bits) { atomicAnd(status, ~bits); }

}  // namespace

int launch_pages_clear(unsigned *status, unsigned bits, void *stream) {
    clear_kernel<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>(status, bits);
    return static_cast<int>(cudaGetLastError());
}

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
