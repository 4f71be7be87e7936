// Paged cache: the pages that a cheap score chooses for each row and KV head.
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr int SE_THREADS = 256;

// Keys that order like the floats (no NaN), as unsigned.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The whole numbers round(Q+- 127 / max|Q+-|) of a row's group of query heads as bytes
// qi[0..D) (Q+) and qi[D..2D) (Q-).  Sums of 16-bit values in 64 bits do not depend on
// the order of the heads.
template <int D>
__device__ void group_query(const PagesSelectArgs &a, int q0, int head, int8_t *qi, float *red) {
    const PagesView &p = a.p;
    const int tid = threadIdx.x;
    double hi = 0., lo = 0.;
    if (tid < D)
        for (int g = 0; g < p.G; g++) {
            const double x = from16(a.q[static_cast<long long>(q0) * a.qt + (head * p.G + g) * a.qh + tid], p.bf16);
            hi += x > 0. ? x : 0.;
            lo += x < 0. ? x : 0.;
            if (x != x) hi = x;
        }
    float h = static_cast<float>(hi), l = static_cast<float>(lo);
    float m = tid < D ? fmaxf(h, -l) : 0.f;
    if (!(fabsf(h) < INFINITY) || !(fabsf(l) < INFINITY)) m = INFINITY;
    m = warp_max(m);
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    m = red[0];
    for (int i = 1; i < SE_THREADS / 32; i++) m = fmaxf(m, red[i]);
    if (tid < D) {
        const bool ok = m > 0.f && m < INFINITY;
        const float inv = ok ? __fdiv_rn(127.f, m) : 0.f;
        qi[tid] = ok ? static_cast<int8_t>(__float2int_rn(__fmul_rn(h, inv))) : 0;
        qi[D + tid] = ok ? static_cast<int8_t>(__float2int_rn(__fmul_rn(l, inv))) : 0;
    }
    __syncthreads();
}

// One CTA per (row, KV head): scores of all pages to shared memory; a page's place is the
// number of pages before it in the order (score down, ordinal up).
template <int D>
__global__ void __launch_bounds__(SE_THREADS) select_kernel(PagesSelectArgs a) {
    extern __shared__ uint32_t key[];
    __shared__ __align__(16) int8_t qi[2 * D];
    __shared__ float red[SE_THREADS / 32];
    __shared__ int wsum[SE_THREADS / 32], base;
    const PagesView &p = a.p;
    const PageRow r = page_row(p, a.r, blockIdx.x);
    const int head = blockIdx.y, tid = threadIdx.x;
    const int np = (r.len + p.P - 1) / p.P;
    int *out = a.sel + (static_cast<long long>(blockIdx.x) * p.Hkv + head) * a.n_sel;
    if (np <= a.n_sel) {
        for (int i = tid; i < a.n_sel; i += SE_THREADS) out[i] = i < np ? i : -1;
        return;
    }
    group_query<D>(a, r.q0, head, qi, red);
    for (int j = tid; j < np; j += SE_THREADS) {
        const int id = page_of(p, r.row, j);
        uint32_t k = 0;
        if (j < a.keep_first || j >= np - a.keep_last) k = 0xffffffffu;
        else if (id >= 0) {
            const int *s = reinterpret_cast<const int *>(summary_ptr(p, id, head));
            int v = 0;
            for (int c = 0; c < 2 * D / 4; c++) v = __dp4a(s[c], reinterpret_cast<const int *>(qi)[c], v);
            const int e = s[2 * D / 4];
            k = order_key(static_cast<float>(v) * pow2i(e < -100 ? -100 : (e > 100 ? 100 : e)) + 0.f);
        }
        key[j] = k;
    }
    if (tid == 0) base = 0;
    __syncthreads();
    for (int j0 = 0; j0 < np; j0 += SE_THREADS) {
        const int j = j0 + tid;
        int take = 0;
        if (j < np) {
            int rank = 0;
            for (int i = 0; i < np; i++) rank += key[i] > key[j] || (key[i] == key[j] && i < j);
            take = rank < a.n_sel;
        }
        const unsigned b = __ballot_sync(FULL, take);
        if ((tid & 31) == 0) wsum[tid >> 5] = __popc(b);
        __syncthreads();
        int at = base + __popc(b & ((1u << (tid & 31)) - 1u));
        for (int i = 0; i < tid >> 5; i++) at += wsum[i];
        if (take) out[at] = j;
        __syncthreads();
        if (tid == SE_THREADS - 1) base = at + take;
        __syncthreads();
    }
}

}  // namespace

int launch_pages_select(const PagesSelectArgs &a, void *stream) {
    const dim3 grid(a.r.n_rows, a.p.Hkv);
    const int smem = a.p.M * 4;
    auto st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (a.p.d == 128) {
        if ((e = cudaFuncSetAttribute(select_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) == cudaSuccess)
            select_kernel<128><<<grid, SE_THREADS, smem, st>>>(a);
    } else {
        if ((e = cudaFuncSetAttribute(select_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) == cudaSuccess)
            select_kernel<64><<<grid, SE_THREADS, smem, st>>>(a);
    }
    return static_cast<int>(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace dq
