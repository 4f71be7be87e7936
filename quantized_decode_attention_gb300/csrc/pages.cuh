// Device code shared by the paged cache's kernels (sm_103a): rows and pages of a
// call, the 4-bit float and scale conversions, the byte layout of a page.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

#include "common.cuh"
#include "pages_internal.h"

namespace dq {

// ---- layout of a block of b tokens (see dq_pages.h) --------------------------------
template <int D>
struct PageBlock {
    // byte offsets of the four parts of a block of b tokens, and its size
    __host__ __device__ static constexpr int ks(int b) { return b * D / 2; }
    __host__ __device__ static constexpr int vc(int b) { return b * D * 9 / 16; }
    __host__ __device__ static constexpr int vs(int b) { return b * D * 17 / 16; }
    __host__ __device__ static constexpr int size(int b) { return b * D * 9 / 8; }
    // value codes of the 16 channels of scale block c16 of the token pair that holds t: 16 bytes
    __device__ static int vcode(int t, int c16) { return (((t >> 3) * (D / 16) + c16) * 4 + ((t >> 1) & 3)) * 16; }
    __device__ static int vscale(int t, int c16) { return (((t >> 3) * (D / 16) + c16) * 4 + ((t >> 1) & 3)) * 2 + (t & 1); }
};

// ---- launches -------------------------------------------------------------------------
// Let kernel K take `bytes` of shared memory: once for each device and kernel (0 or a cudaError_t).
template <auto K>
int allow_shared(int bytes) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (dev < 64 && done[dev].load(std::memory_order_relaxed)) return 0;
    e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_relaxed);
    return static_cast<int>(e);
}

// How many CTAs the launch over the rows' own pages takes, of `grid`, for n places of UNIT_COST and chunks of 32 tokens: few
// where they are done with it before the common pages are, which then have the other SMs at the same time.  With 32 / 48 / 64 / 96 CTAs
// for up to 6144 places, us (8 KV heads of 128, 4 query heads each): 64 rows of 64 own tokens behind 8192 common ones
// 36.5 / - / 38.8 / 43.3, behind 2048 29.3 / - / 29.5 / 31.2, of 250 behind 1536 30.0 / 32.0 / 28.8 / -; 16 of 1300 behind 6144
// 37.9 / 32.8 / 31.1 / -; 128 of 100 behind 1024 34.0 / 31.9 / 29.4 / -; 8 behind 32768 44.8 / - / 53.3 / 68.8; 8 groups of 8 behind 8192
// 68.9 / - / 85.5 / 126: few where the common pages are many, more where the own ones are; 64 loses least at either end.
__device__ __forceinline__ int own_ctas(int n, int grid) {
    constexpr int PLACES = 96, MOST = 64;
    return n <= PLACES * MOST ? MOST : grid;
}

// A kernel launched by launch_overlapping may start while the one before it in the stream still runs, once all of that
// one's CTAs have called let_next_start or ended; it waits for its end with await_previous.  Every CTA of it does, so that its
// own end is behind that one's too.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
template <class K, class... A>
int launch_overlapping(K kernel, dim3 grid, int threads, int smem, cudaStream_t st, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// ---- rows ----------------------------------------------------------------------------
struct PageRow {
    int row;    // table row, -1: padding (nothing held)
    int len;    // tokens held
    int q0, n;  // the call's tokens [q0, q0 + n) are positions [len - n, len)
    int from;   // attention: the first position that is looked at, a page's first
};

// Row i of the call, checked: whatever is out of range is latched and holds nothing.
__device__ __forceinline__ PageRow page_row(const PagesView &p, const PagesRows &r, int i) {
    PageRow o;
    o.row = r.rows ? r.rows[i] : i;
    o.q0 = r.cu ? r.cu[i] : i;
    o.n = r.cu ? r.cu[i + 1] - o.q0 : 1;
    bool bad = false;
    if (o.q0 < 0 || o.n < 0 || o.n > r.max_new || o.q0 > r.n_tok - o.n) {
        bad = true;
        o.q0 = o.n = 0;
    }
    o.len = o.from = 0;
    if (o.row >= p.max_seqs) {
        bad = true;
        o.row = -1;
    }
    if (o.row >= 0) {
        o.len = p.seq_len[o.row];
        if (o.len < 0 || o.len > p.M * p.P) {
            bad = true;
            o.len = 0;
        }
    }
    if (bad) atomicOr(p.status, PST_ARG);
    return o;
}

// The arguments of a kernel for launches of one kind; step: positions from one query token of a row
// to the next, 0 where all see the whole row.
template <int MODE>
struct InMode : PagesAttnArgs {
    static constexpr int mode = MODE, step = MODE == PAGES_NEWEST || MODE == PAGES_OWN;
};

// The last position that the first of a row's query tokens sees.
template <class A>
__device__ __forceinline__ int first_sees(const A &a, const PageRow &r) { return a.step ? r.len - r.n : r.len - 1; }

// Row i of an attention launch, checked.  A group's row is the one that its common pages are read
// from, as long as they are, and its tokens are those of all its rows.
template <class A>
__device__ __forceinline__ PageRow attn_row(const A &a, int i) {
    PageRow o;
    if (a.mode == PAGES_COMMON) {
        const int g0 = a.groups ? a.groups[i] : 0, g1 = a.groups ? a.groups[i + 1] : a.call_rows;
        o = PageRow{-1, 0, 0, 0, 0};
        if (g0 < 0 || g1 > a.call_rows || g0 > g1) {
            atomicOr(a.p.status, PST_ARG);
            return o;
        }
        if (g0 == g1) return o;
        const int2 what = reinterpret_cast<const int2 *>(a.plan)[g0];
        const int q0 = a.r.cu ? a.r.cu[g0] : g0, n = (a.r.cu ? a.r.cu[g1] : g1) - q0;
        if (what.x == 0) return o;
        if (q0 < 0 || n < 0 || n > a.r.max_new || q0 > a.r.n_tok - n || what.x < 0 || what.x % a.p.P || what.y < 0 || what.y >= a.p.max_seqs ||
            what.x > a.p.seq_len[what.y] || what.x > a.p.M * a.p.P) {
            atomicOr(a.p.status, PST_ARG);
            return o;
        }
        return PageRow{what.y, what.x, q0, n, 0};
    }
    o = page_row(a.p, a.r, i);
    if (a.mode == PAGES_OWN && o.len > 0 && o.n > 0) {  // (a row that brings nothing may be shorter than what the others share)
        o.from = a.plan[2 * i];
        if (o.from < 0 || o.from % a.p.P || (o.from > 0 && o.from > o.len - o.n)) {
            atomicOr(a.p.status, PST_ARG);
            o.from = 0;
        }
    }
    return o;
}
// The same, known to be in order: `row` and `keys` (len - from) are what the check found.
template <class A>
__device__ __forceinline__ PageRow known_row(const A &a, int i, int row, int keys) {
    PageRow o;
    o.row = row;
    if (a.mode == PAGES_COMMON) {
        const int g0 = a.groups ? a.groups[i] : 0, g1 = a.groups ? a.groups[i + 1] : a.call_rows;
        o.q0 = a.r.cu ? a.r.cu[g0] : g0;
        o.n = (a.r.cu ? a.r.cu[g1] : g1) - o.q0;
        o.len = keys;
        o.from = 0;
        return o;
    }
    o.q0 = a.r.cu ? a.r.cu[i] : i;
    o.n = a.r.cu ? a.r.cu[i + 1] - o.q0 : 1;
    o.len = a.mode == PAGES_OWN && row >= 0 ? a.p.seq_len[row] : keys;
    o.from = o.len - keys;
    return o;
}

// Where query row `row` (token, query head of the group) of a row and KV head stands among the call's queries.
template <class A>
__device__ __forceinline__ long long query_of(const A &a, const PageRow &r, int head, int row) {
    const int tok = row / a.p.G;
    return (static_cast<long long>(r.q0) + tok) * a.p.Hq + head * a.p.G + row - tok * a.p.G;
}
// Maxima and sums of the parts, behind their accumulators.
template <int D, class A>
__device__ __forceinline__ float *part_sums(const A &a) {
    return a.part + static_cast<long long>(a.r.n_tok) * a.p.Hq * D;
}

template <class A>
__device__ __forceinline__ bool takes(const A &a, const PageRow &r) { return r.n * a.p.G > a.over && r.n * a.p.G <= a.most; }

// Page number of ordinal j of a row (0 <= j < M), -1 (latched) where the table's entry
// is no page of the pool.
__device__ __forceinline__ int page_of(const PagesView &p, int row, int j) {
    const int id = p.table[static_cast<long long>(row) * p.M + j];
    if (id < 0 || id >= p.n_pages) {
        atomicOr(p.status, PST_TABLE);
        return -1;
    }
    return id;
}

__device__ __forceinline__ uint8_t *page_ptr(const PagesView &p, int id, int head) {
    return p.pages + (static_cast<long long>(id) * p.Hkv + head) * p.page_bytes;
}
__device__ __forceinline__ uint8_t *summary_ptr(const PagesView &p, int id, int head) {
    return p.summary + (static_cast<long long>(id) * p.Hkv + head) * p.sum_bytes;
}

// PAGES_COMMON: this thread's part of the places of the launch over the rows' own pages.  The upper half of the CTA's threads
// look at them, while the lower ones look at the groups.
template <int T, class A>
__device__ __forceinline__ long long own_places(const A &a) {
    long long n = 0;
    if (a.mode == PAGES_COMMON && a.after_few && threadIdx.x >= T / 2) {
        const int few = a.own_max_new * a.p.G <= 8 ? 8 : 16;
        PagesRows rows = a.r;
        rows.n_rows = a.call_rows;
        rows.max_new = a.own_max_new;
        for (int i = threadIdx.x - T / 2; i < a.call_rows; i += T / 2) {
            const int from = a.plan[2 * i];
            const PageRow r = page_row(a.p, rows, i);
            const int keys = r.len - (from > 0 && from <= r.len - r.n && from % a.p.P == 0 ? from : 0);
            if (r.len > 0) n += static_cast<long long>((r.n * a.p.G + few - 1) / few) * a.p.Hkv * ((keys + 31) / 32 + FEW_UNIT_COST);
        }
    }
    return n;
}
// CTAs that the launch has for itself: those that the one over the rows' own pages, which may still run, does not take.
template <int T, class A>
__device__ __forceinline__ int sms_left(const A &a, long long n, long long *part) {
    if (a.mode != PAGES_COMMON || !a.after_few) return gridDim.x;
    const int tid = threadIdx.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(FULL, n, o);
    __syncthreads();
    if ((tid & 31) == 0) part[tid >> 5] = n;
    __syncthreads();
    n = 0;
    for (int k = 0; k < T / 32; k++) n += part[k];
    const int left = static_cast<int>(gridDim.x) - (n > 1 << 30 ? static_cast<int>(gridDim.x) : own_ctas(static_cast<int>(n), gridDim.x));
    return left > 0 ? left : gridDim.x;
}

// ---- conversions -----------------------------------------------------------------------
__device__ __forceinline__ float from16(uint16_t x, bool bf16) {
    return bf16 ? __uint_as_float(static_cast<uint32_t>(x) << 16) : __half2float(__ushort_as_half(x));
}
__device__ __forceinline__ uint16_t to16(float x, bool bf16) {
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}
// The larger magnitudes (with signs of no meaning), NaN where there is one.
template <bool BF16>
__device__ __forceinline__ uint32_t max2_abs(uint32_t a, uint32_t b) {
    uint32_t r;
    if (BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool BF16>
__device__ __forceinline__ float2 pair_to_float(uint32_t w) {
    if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
// Four bytes of two codes each -> four half2 of code values (low nibble first).
__device__ __forceinline__ void e2m1x8_to_half(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Two e4m3 scales (low byte first) -> half2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t s) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(s));
    return h;
}
__device__ __forceinline__ float e4m3_to_float(uint8_t s) {
    const uint32_t h = e4m3x2_to_half2(s);
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
}
__device__ __forceinline__ uint8_t float_to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(0.f), "f"(x));
    return static_cast<uint8_t>(r & 0xff);
}
// Codes of eight values, the first in the lowest four bits.
__device__ __forceinline__ uint32_t float8_to_e2m1(float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(r)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3), "f"(x4), "f"(x5), "f"(x6), "f"(x7));
    return r;
}

}  // namespace dq
