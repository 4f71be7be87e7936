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

// ---- rows ----------------------------------------------------------------------------
struct PageRow {
    int row;    // table row, -1: padding (nothing held)
    int len;    // tokens held
    int q0, n;  // the call's tokens [q0, q0 + n) are positions [len - n, len)
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
    o.len = 0;
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

__device__ __forceinline__ bool takes(const PagesAttnArgs &a, const PageRow &r) { return r.n * a.p.G > a.over && r.n * a.p.G <= a.most; }

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

// ---- conversions -----------------------------------------------------------------------
__device__ __forceinline__ float from16(uint16_t x, bool bf16) {
    return bf16 ? __uint_as_float(static_cast<uint32_t>(x) << 16) : __half2float(__ushort_as_half(x));
}
__device__ __forceinline__ uint16_t to16(float x, bool bf16) {
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
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
