// Paged cache: the attention weight that each held token gets from the newest queries.
//
//   score_j (+)= sum over the row's newest tokens i that see j and the group's heads g of
//                exp(sm_scale q_ig . k_j - lse_ig)
// with lse from the attention of the same queries, so that one pass over the keys is
// enough.  Only the keys' half of the pages is read (D / 2 + D / 16 bytes a token and KV
// head) and 8 bytes of scores are read and written.
//
// All rows' chunks of 32 tokens, KV heads within a row, stand on a line that is cut into
// equal shares, one for each warp.  A lane (g, t) = (lane / 4, lane % 4) loads its operands of
// mma.sync m16n8k16 straight from the page (D / 4 channels at t D / 4 of tokens g and g + 8,
// K [16 tokens x 16 channels] . Q^T, 8 query rows in the n of 8), the next chunk's while it
// works on this one's, and the page number after that (16 rows of 4160: 15.3 -> 13.8 us).
// Every score is one thread's: nothing is joined, and the order of its sum is fixed.  More
// than 8 NT query rows go by blocks, the later ones adding to what the first stored.
//
// Bound by the lengths, the table and the first codes one after the other where rows are short, by
// mma.sync and the conversions of codes where they are long (16 rows of 4160 tokens, 32 / 8 heads, head_dim 128,
// one query each: 13.8 us, 43 MB; 8 of 32768 with 4: 65 us, 2.6 TB/s).
#include <cuda_runtime.h>

#include "pages_weigh.cuh"

namespace dq {
namespace {

constexpr int CHUNK = 32;
// Query rows of a row and KV head beyond which the tensor-core kernel takes over (8 rows of 32768 tokens, 8 KV heads; this kernel
// against that: 32 query rows 124 / 208 us, 48 181 / 208, 64 238 / 208; 1 row of 8192: 48 14.2 / 15.6, 64 17.3 / 15.6).
constexpr int MANY_ROWS = 48;

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// A chunk's keys as a lane holds them: tokens g, g + 8, g + 16, g + 24, D / 4 channels at t D / 4.
template <int D>
struct Keys {
    uint32_t w[4][D / 32];
    uint32_t s[2];  // scales of two tokens each: D / 64 bytes of a token, low half the first
    __device__ __forceinline__ void load(const PagesView &p, const uint8_t *page, int u) {  // chunk at token u of the page
        using B = PageBlock<D>;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int b = p.blk, ub = u % b;
        const uint8_t *blk = page + u / b * B::size(b);
        const uint8_t *kc = blk + (ub + g) * (D / 2) + t * (D / 8), *ks = blk + B::ks(b) + (ub + g) * (D / 16) + t * (D / 64);
        part(0, kc, ks);
        part(1, kc + 16 * (D / 2), ks + D);
    }
    __device__ __forceinline__ void part(int h, const uint8_t *kc, const uint8_t *ks) {  // 16 tokens
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const uint8_t *c = kc + e * 8 * (D / 2);
            if (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4 *>(c);
                w[2 * h + e][0] = x.x;
                w[2 * h + e][1] = x.y;
                w[2 * h + e][D == 128 ? 2 : 0] = x.z;
                w[2 * h + e][D == 128 ? 3 : 0] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(c);
                w[2 * h + e][0] = x.x;
                w[2 * h + e][1] = x.y;
            }
        }
        const uint32_t s0 = D == 128 ? *reinterpret_cast<const uint16_t *>(ks) : *ks;
        const uint32_t s1 = D == 128 ? *reinterpret_cast<const uint16_t *>(ks + D / 2) : ks[D / 2];
        s[h] = s0 | s1 << 16;
    }
    __device__ __forceinline__ void none(int h) {
#pragma unroll
        for (int i = 0; i < D / 32; i++) w[2 * h][i] = w[2 * h + 1][i] = 0;
        s[h] = 0;
    }
};

// 8 NT query rows as operands: lane (g, t) holds channels of row g, and what belongs to rows 2t and 2t + 1.
template <int D, int NT>
struct Queries {
    uint32_t q[NT][D / 16][2];
    float f[NT][2], less[NT][2];  // logit units; what a logit loses before the exponential, +inf: no row, or one that sees nothing
    int pos[NT][2];
    __device__ __forceinline__ void load(const PagesWeighArgs &a, const PageRow &r, int head, int row0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, rows = r.n * a.p.G;
#pragma unroll
        for (int n = 0; n < NT; n++) {
            const int row = row0 + 8 * n + g, tok = row / a.p.G;
            const uint16_t *src = a.q + (static_cast<long long>(r.q0) + tok) * a.qt + (head * a.p.G + row - tok * a.p.G) * a.qh + t * (D / 4);
            float x[D / 4], top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; i++) {
                const uint4 w = row < rows ? *reinterpret_cast<const uint4 *>(src + 8 * i) : make_uint4(0, 0, 0, 0);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    x[8 * i + 2 * j] = from16(static_cast<uint16_t>(u[j] & 0xffffu), a.p.bf16);
                    x[8 * i + 2 * j + 1] = from16(static_cast<uint16_t>(u[j] >> 16), a.p.bf16);
                }
            }
#pragma unroll
            for (int i = 0; i < D / 4; i++) top = fmaxf(top, fabsf(x[i]));
            top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
            top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
            // by a power of two below 2^14, as attention takes them
            int up = 13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
            up = top > 0.f ? (up > 126 ? 126 : up) : 0;
            const float s = pow2i(up);
#pragma unroll
            for (int i = 0; i < D / 16; i++) {
                q[n][i][0] = half2_of(x[4 * i] * s, x[4 * i + 1] * s);
                q[n][i][1] = half2_of(x[4 * i + 2] * s, x[4 * i + 3] * s);
            }
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int other = __shfl_sync(FULL, up, 4 * (2 * t + e)), rw = row0 + 8 * n + 2 * t + e, tk = rw / a.p.G;
                f[n][e] = a.scale_log2 * pow2i(-other);
                pos[n][e] = r.len - r.n + tk;
                less[n][e] = INFINITY;
                if (rw < rows) {
                    const float lse = a.lse[(static_cast<long long>(r.q0) + tk) * a.p.Hq + head * a.p.G + rw - tk * a.p.G];
                    if (lse != -INFINITY) less[n][e] = lse * LOG2E;
                }
            }
        }
    }
};

// Weights of a chunk's 32 tokens at `at` from these queries: this lane's token g + 8 t.
template <int D, int NT>
__device__ __forceinline__ float weigh_chunk(const Keys<D> &k, const Queries<D, NT> &q, int at, int least) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float got[4];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; n++) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        const uint32_t two0 = e4m3x2_to_half2(static_cast<uint16_t>(k.s[h])), two1 = e4m3x2_to_half2(static_cast<uint16_t>(k.s[h] >> 16));
        uint32_t sa[2], sb[2];
        sa[0] = __byte_perm(two0, two0, 0x1010);
        sb[0] = __byte_perm(two1, two1, 0x1010);
        sa[1] = D == 128 ? __byte_perm(two0, two0, 0x3232) : sa[0];
        sb[1] = D == 128 ? __byte_perm(two1, two1, 0x3232) : sb[0];
#pragma unroll
        for (int w = 0; w < D / 32; w++) {
            uint32_t a[4], b[4];
            e2m1x8_to_half(k.w[2 * h][w], a);
            e2m1x8_to_half(k.w[2 * h + 1][w], b);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                a[i] = hmul2(a[i], sa[w >> 1]);
                b[i] = hmul2(b[i], sb[w >> 1]);
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
                mma_f16(s[n], a[0], b[0], a[1], b[1], q.q[n][2 * w][0], q.q[n][2 * w][1]);
                mma_f16(s[n], a[2], b[2], a[3], b[3], q.q[n][2 * w + 1][0], q.q[n][2 * w + 1][1]);
            }
        }
        got[2 * h] = got[2 * h + 1] = 0.f;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) {  // token g + 16 h + 8 (i / 2), row 2t + i % 2
                float z = fmaf(s[n][i], q.f[n][i & 1], -q.less[n][i & 1]);
                if (at + CHUNK - 1 > least && at + 16 * h + g + 8 * (i >> 1) > q.pos[n][i & 1]) z = -INFINITY;
                got[2 * h + (i >> 1)] += q.less[n][i & 1] == INFINITY ? 0.f : ex2(z);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        got[i] += __shfl_xor_sync(FULL, got[i], 1);
        got[i] += __shfl_xor_sync(FULL, got[i], 2);
    }
    return t == 0 ? got[0] : (t == 1 ? got[1] : (t == 2 ? got[2] : got[3]));
}

constexpr int WARPS = 8;

template <int D, int NT>
__global__ void __launch_bounds__(32 * WARPS, 2) weigh_chunks(PagesWeighArgs a) {
    __shared__ long long first[DQ_PAGES_MAX_ROWS + 1], part[WARPS];
    __shared__ int row_s[DQ_PAGES_MAX_ROWS], keys_s[DQ_PAGES_MAX_ROWS];
    const PagesView &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long base = weigh_rows<32 * WARPS>(a, row_s, keys_s, first, part, [&](const PageRow &r) {
        return static_cast<long long>((r.len + CHUNK - 1) / CHUNK) * p.Hkv;
    });
    __syncthreads();
    const long long all = static_cast<long long>(gridDim.x) * WARPS, me = static_cast<long long>(blockIdx.x) * WARPS + warp;
    const long long x0 = base * me / all, x1 = base * (me + 1) / all;
    const int shift = 31 - __clz(p.P);  // (a power of two)
    for (long long x = x0; x < x1;) {
        int i;
        const PageRow r = weigh_row_at(a, row_s, keys_s, first, x, i);
        const int chunks = (r.len + CHUNK - 1) / CHUNK, at = static_cast<int>(x - first[i]);
        const int head = at / chunks, t0 = at % chunks;
        const int t1 = x1 - x < chunks - t0 ? t0 + static_cast<int>(x1 - x) : chunks;
        x += t1 - t0;
        float *scores = scores_of(a, r.row, head);
        const int *table = p.table + static_cast<long long>(r.row) * p.M;
        const int rows = r.n * p.G, old = r.len - r.n, mine = (lane >> 2) + 8 * (lane & 3);
        for (int row0 = 0; row0 < rows; row0 += 8 * NT) {
            const int least = old + row0 / p.G;
            // what the table has for a chunk's page (pages of 16: its two)
            auto entry = [&](int c) {
                const int *e = table + (c * CHUNK >> shift);
                return make_int2(e[0], p.P < CHUNK && c * CHUNK + 16 < r.len ? e[1] : 0);
            };
            auto checked = [&](int id) {
                if (id >= 0 && id < p.n_pages) return id;
                atomicOr(p.status, PST_TABLE);
                return -1;
            };
            auto load = [&](Keys<D> &k, float &s, int c, int2 e) {
                const int at = c * CHUNK;
                if (p.P >= CHUNK) {
                    const int id = checked(e.x);
                    if (id < 0) {
                        k.none(0);
                        k.none(1);
                    } else {
                        k.load(p, page_ptr(p, id, head), at & (p.P - 1));
                    }
                } else {
                    using B = PageBlock<D>;
                    const int g = lane >> 2, t = lane & 3;
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int id = at + 16 * h < r.len ? checked(h ? e.y : e.x) : -1;
                        if (id < 0) {
                            k.none(h);
                            continue;
                        }
                        const uint8_t *page = page_ptr(p, id, head);
                        k.part(h, page + g * (D / 2) + t * (D / 8), page + B::ks(16) + g * (D / 16) + t * (D / 64));
                    }
                }
                s = at + mine < r.len && (row0 > 0 || at + mine < old) ? scores[at + mine] : 0.f;
            };
            Keys<D> cur, nxt;
            float was, next_was;
            load(cur, was, t0, entry(t0));  // (on its way while the queries are put together)
            int2 ahead = t0 + 1 < t1 ? entry(t0 + 1) : make_int2(0, 0);
            Queries<D, NT> q;
            q.load(a, r, head, row0);
            for (int c = t0; c < t1; c++) {
                if (c + 1 < t1) load(nxt, next_was, c + 1, ahead);
                if (c + 2 < t1) ahead = entry(c + 2);
                const float got = weigh_chunk<D, NT>(cur, q, c * CHUNK, least);
                if (c * CHUNK + mine < r.len) scores[c * CHUNK + mine] = was + got;
                cur = nxt;
                was = next_was;
            }
        }
    }
}

template <int D, int NT>
int launch_as(const PagesWeighArgs &a, int num_sms, cudaStream_t st) {
    weigh_chunks<D, NT><<<2 * num_sms, 32 * WARPS, 0, st>>>(a);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_pages_weigh(PagesWeighArgs a, int num_sms, void *stream) {
    auto st = static_cast<cudaStream_t>(stream);
    const int rows = a.r.max_new * a.p.G;
    a.over = 0;
    a.most = 0x7fffffff;
    if (rows > MANY_ROWS) {  // rows with many query rows on the tensor cores, the others of a mixed batch here
        const bool mixed = few_beside_most(a.r, a.p.G, MANY_ROWS);
        a.over = mixed ? MANY_ROWS : 0;
        if (const int e = launch_pages_weigh_many(a, num_sms < PAGES_MAX_CTAS ? num_sms : PAGES_MAX_CTAS, stream)) return e;
        if (!mixed) return 0;
        a.over = 0;
        a.most = MANY_ROWS;
    }
    // two n tiles share the conversions of a chunk (16 query rows: 65 us, with one tile 116; four tiles: no less at 32 than two)
    if (rows <= 8) return a.p.d == 128 ? launch_as<128, 1>(a, num_sms, st) : launch_as<64, 1>(a, num_sms, st);
    return a.p.d == 128 ? launch_as<128, 2>(a, num_sms, st) : launch_as<64, 2>(a, num_sms, st);
}

}  // namespace dq
