// Paged cache: attention of each row's newest tokens over its 4-bit pages.
//
// For a query at position x, with z_j = sm_scale q . k_j over the visible keys j <= x:
//   m = max z_j, l = sum exp(z_j - m), out = sum exp(z_j - m) v_j / l, lse = m + log l
// in one pass: a running m, l and accumulator, rescaled when m grows.
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr int AT_THREADS = 128, AT_ROWS = 8, AT_CH = 32;
constexpr float LN2 = 0.69314718055994530942f;

// One CTA per (8 query rows of a row and KV head); a query row is a (token, query head
// of the group).  Keys and values of up to 32 tokens at a time are expanded to fp32.
template <int D>
__global__ void __launch_bounds__(AT_THREADS) attn_simple(PagesAttnArgs a) {
    __shared__ float kf[AT_CH][D + 1], vf[AT_CH][D];
    __shared__ float qf[AT_ROWS][D], pr[AT_ROWS][AT_CH], al[AT_ROWS], ls[AT_ROWS], ms[AT_ROWS];
    using B = PageBlock<D>;
    const PagesView &p = a.p;
    const PageRow r = page_row(p, a.r, blockIdx.y);
    const int head = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int m0 = blockIdx.x * AT_ROWS, rows = r.n * p.G;
    if (m0 >= rows) return;
    for (int i = tid; i < AT_ROWS * D; i += AT_THREADS) {
        const int m = m0 + i / D;
        float x = 0.f;
        if (m < rows) x = from16(a.q[(static_cast<long long>(r.q0) + m / p.G) * a.qt + (head * p.G + m % p.G) * a.qh + i % D], p.bf16);
        qf[i / D][i % D] = x;
    }
    if (tid < AT_ROWS) {
        ms[tid] = -INFINITY;
        ls[tid] = 0.f;
    }
    float acc[AT_ROWS];
#pragma unroll
    for (int i = 0; i < AT_ROWS; i++) acc[i] = 0.f;
    const int ch = p.P < AT_CH ? p.P : AT_CH;
    const int entries = a.sel ? a.n_sel : (r.len + p.P - 1) / p.P;
    for (int e = 0; e < entries; e++) {
        const int ord = a.sel ? a.sel[(static_cast<long long>(blockIdx.y) * p.Hkv + head) * a.n_sel + e] : e;
        if (ord < 0 || ord >= p.M || ord * p.P >= r.len) continue;
        const int id = page_of(p, r.row, ord);
        if (id < 0) continue;
        const uint8_t *page = page_ptr(p, id, head);
        for (int s0 = 0; s0 < p.P && ord * p.P + s0 < r.len; s0 += ch) {
            __syncthreads();
            const int pos0 = ord * p.P + s0;
            for (int i = tid; i < AT_CH * (D / 16); i += AT_THREADS) {
                const int t = i / (D / 16), c = i % (D / 16), tp = s0 + t, tb = tp % p.blk;
                const bool in = t < ch && pos0 + t < r.len;
                const uint8_t *blk = page + (tp / p.blk) * B::size(p.blk);
                const float ks = in ? e4m3_to_float(blk[B::ks(p.blk) + tb * (D / 16) + c]) : 0.f;
                const float vs = in ? e4m3_to_float(blk[B::vs(p.blk) + B::vscale(tb, c)]) : 0.f;
                const uint8_t *kc = blk + tb * (D / 2) + 8 * c, *vc = blk + B::vc(p.blk) + B::vcode(tb, c);
                for (int x = 0; x < 16; x++) {
                    kf[t][16 * c + x] = in ? e2m1_to_float((kc[x >> 1] >> (4 * (x & 1))) & 15u) * ks : 0.f;
                    vf[t][16 * c + x] = in ? e2m1_to_float((vc[x] >> (4 * (tp & 1))) & 15u) * vs : 0.f;
                }
            }
            __syncthreads();
            // warp w: query rows 2w and 2w + 1, lane = token
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int m = 2 * warp + i, pos = r.len - r.n + (m0 + m) / p.G;
                float z = 0.f;
                for (int c = 0; c < D; c++) z += qf[m][c] * kf[lane][c];
                z = m0 + m < rows && lane < ch && pos0 + lane <= pos ? z * a.scale_log2 : -INFINITY;
                const float mx = fmaxf(ms[m], warp_max(z)), mu = mx == -INFINITY ? 0.f : mx;
                const float w = exp2f(z - mu), sum = warp_sum(w);
                pr[m][lane] = w;
                __syncwarp();
                if (lane == 0) {
                    al[m] = exp2f(ms[m] - mu);
                    ls[m] = ls[m] * al[m] + sum;
                    ms[m] = mx;
                }
                __syncwarp();
            }
            __syncthreads();
            if (tid < D) {
#pragma unroll
                for (int m = 0; m < AT_ROWS; m++) {
                    acc[m] *= al[m];
                    for (int t = 0; t < AT_CH; t++) acc[m] += pr[m][t] * vf[t][tid];
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < AT_ROWS; m++) {
        if (m0 + m >= rows) break;
        const long long o = (static_cast<long long>(r.q0) + (m0 + m) / p.G) * p.Hq + head * p.G + (m0 + m) % p.G;
        if (tid < D) a.out[o * D + tid] = to16(ls[m] == 0.f ? 0.f : acc[m] * a.out_scale / ls[m], p.bf16);
        if (tid == 0 && a.lse) a.lse[o] = ls[m] == 0.f ? -INFINITY : (ms[m] + log2f(ls[m])) * LN2;
    }
}

}  // namespace

int launch_pages_attention(const PagesAttnArgs &a, void *stream) {
    const dim3 grid((a.r.max_new * a.p.G + AT_ROWS - 1) / AT_ROWS, a.r.n_rows, a.p.Hkv);
    auto st = static_cast<cudaStream_t>(stream);
    if (a.p.d == 128) attn_simple<128><<<grid, AT_THREADS, 0, st>>>(a);
    else attn_simple<64><<<grid, AT_THREADS, 0, st>>>(a);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace dq
