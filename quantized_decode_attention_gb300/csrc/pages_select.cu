// Paged cache: the pages that a cheap score chooses for each row and KV head.
//
// score(page) = sum_c Q+_c largest_c + Q-_c smallest_c, both factors whole numbers of 8
// bits: 2 D products in D / 2 dp4a, exact.  A page costs its summary of 2 D + 4 bytes, so
// the kernel is bound by reading summaries, and for few rows by latency: a cluster of up
// to 8 CTAs shares the pages of one (row, KV head) and sends its scores to the first
// CTA's shared memory.  That CTA finds the n_sel-th largest score digit by digit (four
// histograms of 8 bits) and writes the pages above it, and the first of those equal to
// it, in order: counts and prefixes alone, so that the choice depends on nothing else.
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr int SE_THREADS = 512, SE_WARPS = SE_THREADS / 32;

// Keys that order like the floats (no NaN), as unsigned.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One channel of a group's query heads, loaded before anything else is known of the row.
struct GroupChannel {
    uint16_t x[16];
    __device__ __forceinline__ void load(const PagesSelectArgs &a, int token, int head, int c) {
        const uint16_t *q = a.q + static_cast<long long>(token) * a.qt + static_cast<long long>(head) * a.p.G * a.qh + c;
#pragma unroll
        for (int g = 0; g < 16; g++) x[g] = g < a.p.G ? q[g * a.qh] : 0;
    }
};

// The whole numbers round(Q+- 127 / max|Q+-|) of a row's group of query heads as bytes
// qi[0..D) (Q+) and qi[D..2D) (Q-).  Sums of 16-bit values in 64 bits do not depend on
// the order of the heads.
template <int D>
__device__ __forceinline__ void group_query(const PagesView &p, const GroupChannel &q, int8_t *qi, float *red) {
    const int tid = threadIdx.x;
    double hi = 0., lo = 0.;
    if (tid < D) {
#pragma unroll
        for (int g = 0; g < 16; g++) {
            if (g >= p.G) break;
            const float x = from16(q.x[g], p.bf16);
            if (x > 0.f) hi += x;
            else lo += x;  // (NaN too)
        }
    }
    const float h = static_cast<float>(hi), l = static_cast<float>(lo);
    float m = fmaxf(h, -l);
    if (!(fabsf(h) < INFINITY) || !(fabsf(l) < INFINITY)) m = INFINITY;
    m = warp_max(m);
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int i = 1; i < D / 32; i++) m = fmaxf(m, red[i]);
    if (tid < D) {
        const bool ok = m > 0.f && m < INFINITY;
        // (127 / m passes fp32 for m below 2^-121: such queries go by 2^100 first, which changes none of their bits)
        const float up = m < 0x1p-100f ? 0x1p100f : 1.f;
        const float inv = ok ? __fdiv_rn(127.f, m * up) : 0.f;
        qi[tid] = ok ? static_cast<int8_t>(__float2int_rn(__fmul_rn(h * up, inv))) : 0;
        qi[D + tid] = ok ? static_cast<int8_t>(__float2int_rn(__fmul_rn(l * up, inv))) : 0;
    }
    __syncthreads();
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// Store to the first CTA's shared memory.
__device__ __forceinline__ void store_first(uint32_t addr, uint32_t v) {
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(there) : "r"(addr));
    asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(there), "r"(v) : "memory");
}

// One cluster per (row, KV head).
template <int D>
__global__ void __launch_bounds__(SE_THREADS, 2) select_kernel(PagesSelectArgs a) {
    extern __shared__ uint32_t key[];  // [max_pages_per_seq], the first CTA's counts
    __shared__ __align__(16) int8_t qi[2 * D];
    __shared__ float red[SE_WARPS];
    __shared__ int hist[4 * 256], above[SE_WARPS], equal[SE_WARPS];
    const PagesView &p = a.p;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int row = blockIdx.x / ctas, head = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    GroupChannel channel;
    if (tid < D) channel.load(a, row, head, tid);  // (a token a row)
    const PageRow r = page_row(p, a.r, row);
    const int np = (r.len + p.P - 1) / p.P;
    int *out = a.sel + (static_cast<long long>(row) * p.Hkv + head) * a.n_sel;
    if (np <= a.n_sel) {  // the same for the whole cluster
        if (rank == 0)
            for (int i = tid; i < a.n_sel; i += SE_THREADS) out[i] = i < np ? i : -1;
        return;
    }
    // a page's summary is D / 8 lanes' 16 bytes; each warp has 4 x 32 / (D / 8) pages on their way, page
    // numbers ahead of them (the first while the query is put together)
    constexpr int LANES = D / 8, PER = 32 / LANES, DEEP = 4;
    const int part = lane % LANES, sub = lane / LANES;
    const int j0 = static_cast<int>(static_cast<long long>(np) * rank / ctas), j1 = static_cast<int>(static_cast<long long>(np) * (rank + 1) / ctas);
    const uint32_t keys = smem_u32(key);
    const int *pages = p.table + static_cast<long long>(r.row) * p.M;
    int ahead[DEEP];
    auto numbers = [&](int jw) {
#pragma unroll
        for (int k = 0; k < DEEP; k++) {
            const int j = jw + k * PER + sub;
            ahead[k] = j < j1 ? pages[j] : 0;
        }
    };
    int jw = j0 + warp * PER * DEEP;
    numbers(jw);
    for (int i = tid; i < 4 * 256; i += SE_THREADS) hist[i] = 0;
    group_query<D>(p, channel, qi, red);
    if (ctas > 1) cluster_sync_all();  // the first CTA is there
    const int4 q = *reinterpret_cast<const int4 *>(qi + 16 * part);
    for (; jw < j1; jw += SE_WARPS * PER * DEEP) {
        int id[DEEP];
        int4 s[DEEP];
        int e[DEEP];
#pragma unroll
        for (int k = 0; k < DEEP; k++) {
            id[k] = ahead[k];
            if (jw + k * PER + sub >= j1) {
                id[k] = -1;
            } else if (id[k] < 0 || id[k] >= p.n_pages) {
                atomicOr(p.status, PST_TABLE);
                id[k] = -1;
            }
        }
        numbers(jw + SE_WARPS * PER * DEEP);
#pragma unroll
        for (int k = 0; k < DEEP; k++) {
            s[k] = make_int4(0, 0, 0, 0);
            e[k] = 0;
            if (id[k] < 0) continue;
            const uint8_t *sum = summary_ptr(p, id[k], head);
            s[k] = *reinterpret_cast<const int4 *>(sum + 16 * part);
            e[k] = *reinterpret_cast<const int *>(sum + 2 * D);
        }
#pragma unroll
        for (int k = 0; k < DEEP; k++) {
            const int j = jw + k * PER + sub;
            int v = __dp4a(s[k].x, q.x, __dp4a(s[k].y, q.y, __dp4a(s[k].z, q.z, __dp4a(s[k].w, q.w, 0))));
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1) v += __shfl_xor_sync(FULL, v, o);
            if (part != 0 || j >= j1) continue;
            const int ex = e[k] < -100 ? -100 : (e[k] > 100 ? 100 : e[k]);
            uint32_t o = id[k] < 0 ? 0u : order_key(static_cast<float>(v) * pow2i(ex));
            if (j < a.keep_first || j >= np - a.keep_last) o = 0xffffffffu;
            if (ctas == 1) key[j] = o;
            else store_first(keys + 4 * j, o);
        }
    }
    if (ctas > 1) {
        cluster_sync_all();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    // The n_sel-th largest key, 8 bits at a time: `last` holds its digits so far, `take` its place among the keys
    // that share them.  Every warp reads the counts for itself.  Done early where all keys that share the digits are taken.
    uint32_t last = 0;
    int take = a.n_sel;
    for (int shift = 24; shift >= 0; shift -= 8) {
        int *h = hist + 32 * shift;
        for (int j = tid; j < np; j += SE_THREADS) {
            const uint32_t k = key[j];
            if (shift == 24 || (k ^ last) >> (shift + 8) == 0) atomicAdd(&h[k >> shift & 255u], 1);
        }
        __syncthreads();
        // lane l: digits 255 - 8 l down to 248 - 8 l
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) sum += c[i] = h[255 - 8 * lane - i];
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(FULL, before, o);
            if (lane >= o) before += t;
        }
        before -= sum;
        const unsigned here = __ballot_sync(FULL, before < take && before + sum >= take);
        int digit = 0, at = 0, count = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if (before < take && before + c[i] >= take) {
                digit = 255 - 8 * lane - i;
                at = take - before;
                count = c[i];
            }
            before += c[i];
        }
        const int from = __ffs(here) - 1;
        last |= static_cast<uint32_t>(__shfl_sync(FULL, digit, from)) << shift;
        take = __shfl_sync(FULL, at, from);
        if (__shfl_sync(FULL, count, from) == take && last > 0) {  // all of them: every key from `last` on
            last--;
            take = 0;
            break;
        }
    }
    // a warp's pages are neighbours: [b0, b1)
    const int b0 = static_cast<int>(static_cast<long long>(np) * warp / SE_WARPS), b1 = static_cast<int>(static_cast<long long>(np) * (warp + 1) / SE_WARPS);
    int na = 0, ne = 0;
    for (int j = b0; j < b1; j += 32) {
        const uint32_t k = j + lane < b1 ? key[j + lane] : 0;
        na += __popc(__ballot_sync(FULL, j + lane < b1 && k > last));
        ne += __popc(__ballot_sync(FULL, j + lane < b1 && k == last));
    }
    if (lane == 0) {
        above[warp] = na;
        equal[warp] = ne;
    }
    __syncthreads();
    na = ne = 0;
    for (int w = 0; w < warp; w++) {
        na += above[w];
        ne += equal[w];
    }
    const unsigned below = (1u << lane) - 1u;
    for (int j = b0; j < b1; j += 32) {
        const bool in = j + lane < b1;
        const uint32_t k = in ? key[j + lane] : 0;
        const unsigned ma = __ballot_sync(FULL, in && k > last), me = __ballot_sync(FULL, in && k == last);
        const int before_a = na + __popc(ma & below), before_e = ne + __popc(me & below);
        const bool mine = (ma >> lane & 1u) || ((me >> lane & 1u) && before_e < take);
        if (mine) out[before_a + (before_e < take ? before_e : take)] = j + lane;
        na += __popc(ma);
        ne += __popc(me);
    }
}

template <int D>
int launch_as(const PagesSelectArgs &a, int ctas, cudaStream_t st) {
    const int smem = a.p.M * 4;
    if (const int e = allow_shared<select_kernel<D>>(PAGES_SELECT_MAX * 4)) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.r.n_rows * ctas, a.p.Hkv);
    cfg.blockDim = dim3(SE_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel<D>, a);
    return static_cast<int>(e != cudaSuccess ? e : cudaGetLastError());
}

}  // namespace

int launch_pages_select(const PagesSelectArgs &a, int num_sms, void *stream) {
    // clusters while the card has room for them and a CTA keeps 128 pages (of a full table): with the attention
    // to the chosen pages, 1 row of 2048 pages 22.6 us (one CTA for each 37.0), 4 rows of 512 22.6 (25.0)
    int ctas = 1;
    while (ctas < 8 && a.r.n_rows * a.p.Hkv * ctas * 2 <= 2 * num_sms && a.p.M / (ctas * 2) >= 128) ctas *= 2;
    return a.p.d == 128 ? launch_as<128>(a, ctas, static_cast<cudaStream_t>(stream)) : launch_as<64>(a, ctas, static_cast<cudaStream_t>(stream));
}

}  // namespace dq
