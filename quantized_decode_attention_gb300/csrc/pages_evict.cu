// Paged cache: the tokens of a row with the highest scores, into the pages of another.
//
// Row dst has room for k tokens.  For each layer and KV head it gets, in order, the first
// keep_first and the last keep_last tokens of row src and of those between them the
// k - keep_first - keep_last with the highest scores (the earlier where scores are equal),
// with their scores and the pages' summaries.
//
// One CTA per (pair, KV head, layer).  The border between kept and evicted scores is found
// digit by digit (8 bits a pass over the scores, counts in shared memory).  Then the
// tokens are walked once more: kept ones queue up in shared memory, and whenever the queue
// holds a block of the destination page its bytes are put together, a 16-byte piece a
// thread, straight from the source pages: keys and scales as they are, values two tokens a
// byte.
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr int EV_THREADS = 256, EV_WARPS = EV_THREADS / 32, EV_PER = 4, EV_TURN = EV_THREADS * EV_PER;

// Keys that order like the scores, as unsigned: NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

struct Border {
    uint32_t last;  // keys above it are kept
    int take;       // and the first `take` of those equal to it
};

// The `take`-th largest key of scores [lo, hi), 1 <= take <= hi - lo.  `hist` holds 256 counts.
__device__ Border find_border(const float *scores, int lo, int hi, int take, int *hist) {
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t last = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += EV_THREADS) hist[i] = 0;
        __syncthreads();
        for (int j = lo + tid; j < hi; j += EV_THREADS) {
            const uint32_t k = order_key(scores[j]);
            if (shift == 24 || (k ^ last) >> (shift + 8) == 0) atomicAdd(&hist[k >> shift & 255u], 1);
        }
        __syncthreads();
        // lane l: digits 255 - 8 l down to 248 - 8 l
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) sum += c[i] = hist[255 - 8 * lane - i];
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(FULL, before, o);
            if (lane >= o) before += t;
        }
        before -= sum;
        const unsigned here = __ballot_sync(FULL, before < take && before + sum >= take);
        int digit = 0, at = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if (before < take && before + c[i] >= take) {
                digit = 255 - 8 * lane - i;
                at = take - before;
            }
            before += c[i];
        }
        const int from = __ffs(here) - 1;
        last |= static_cast<uint32_t>(__shfl_sync(FULL, digit, from)) << shift;
        take = __shfl_sync(FULL, at, from);
        __syncthreads();
    }
    return Border{last, take};
}

// Exclusive prefix of v over the CTA; `total` gets the sum.
__device__ __forceinline__ int block_prefix(int v, int *part, int &total) {
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
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < EV_WARPS; w++) {
        const int t = part[w];
        if (w < warp) before += t;
        total += t;
    }
    return before + s - v;
}

template <int D>
__global__ void __launch_bounds__(EV_THREADS) evict_kernel(PagesEvictArgs a) {
    using L = PageBlock<D>;
    constexpr int C = D / 16, QUEUE = 64 + EV_TURN;
    __shared__ __align__(16) uint8_t img[64 * D * 9 / 16];  // a block's key codes, then their scales
    __shared__ float top_s[EV_WARPS][D], low_s[EV_WARPS][D], red[EV_WARPS];
    __shared__ int hist[256], part[EV_WARPS];
    __shared__ int page_q[QUEUE];     // kept tokens that wait: their pages,
    __shared__ uint8_t token_q[QUEUE];  // and their places in them
    PagesView p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int src = a.src[blockIdx.x], dst = a.dst[blockIdx.x], head = blockIdx.y, layer = blockIdx.z;
    if (src < 0 || dst < 0) return;
    // is dst in order: a row of its own, named once?
    bool bad = src >= p.max_seqs || dst >= p.max_seqs || src == dst;
    for (int i = tid; i < a.n; i += EV_THREADS) {
        if (a.src[i] < 0 || a.dst[i] < 0) continue;
        bad |= a.src[i] == dst || (a.dst[i] == dst && i != static_cast<int>(blockIdx.x));
    }
    int len = 0, keep = 0;
    if (!bad) {
        len = p.seq_len[src];
        keep = p.seq_len[dst];
        bad = len < 0 || len > p.M * p.P || keep < 0 || keep > len || len > a.cap || (keep < len && a.keep_first + a.keep_last > keep);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) atomicOr(p.status, PST_ARG);
        return;
    }
    if (keep == 0) return;
    const long long at_layer = static_cast<long long>(layer) * p.n_pages * p.Hkv;
    p.pages += at_layer * p.page_bytes;
    p.summary += at_layer * p.sum_bytes;
    const float *scores = a.scores + ((static_cast<long long>(layer) * p.max_seqs + src) * p.Hkv + head) * a.cap;
    float *to_scores = a.scores + ((static_cast<long long>(layer) * p.max_seqs + dst) * p.Hkv + head) * a.cap;
    // the tokens between the ones kept anyway
    const int lo = keep < len ? a.keep_first : len, hi = keep < len ? len - a.keep_last : len;
    const int want = keep < len ? keep - a.keep_first - a.keep_last : 0;
    Border border{0xffffffffu, 0};
    if (want > 0) border = find_border(scores, lo, hi, want, hist);

    int queued = 0, written = 0, equals = 0, page = -1;
    uint32_t top[4], low[4];
    const int col = tid % (D / 8);
    const int B = p.blk;
    for (int j0 = 0; j0 < len; j0 += EV_TURN) {
        {  // up to EV_TURN more tokens, EV_PER neighbours a thread
            bool above[EV_PER], equal[EV_PER];
            float score[EV_PER];
            int n_above = 0, n_equal = 0;
#pragma unroll
            for (int i = 0; i < EV_PER; i++) {
                const int j = j0 + tid * EV_PER + i;
                above[i] = equal[i] = false;
                score[i] = j < len ? scores[j] : 0.f;
                if (j >= len) continue;
                if (j < lo || j >= hi) above[i] = true;
                else {
                    const uint32_t k = order_key(score[i]);
                    above[i] = k > border.last;
                    equal[i] = k == border.last;
                }
                n_above += above[i];
                n_equal += equal[i];
            }
            int some;
            const int before = block_prefix(n_above | n_equal << 16, part, some);
            int na = before & 0xffff, ne = equals + (before >> 16);
            // equals that are kept come first: those so far are min(ne, take)
            const int base = queued - (equals < border.take ? equals : border.take);
#pragma unroll
            for (int i = 0; i < EV_PER; i++) {
                const int j = j0 + tid * EV_PER + i;
                if (above[i] || (equal[i] && ne < border.take)) {
                    const int at = base + na + (ne < border.take ? ne : border.take);
                    if (written + at >= keep) break;  // (scores that change under the call)
                    page_q[at] = page_of(p, src, j / p.P);
                    token_q[at] = static_cast<uint8_t>(j % p.P);
                    to_scores[written + at] = score[i];
                }
                na += above[i];
                ne += equal[i];
            }
            const int all_equal = equals + (some >> 16);
            queued = base + (some & 0xffff) + (all_equal < border.take ? all_equal : border.take);
            queued = queued < keep - written ? queued : keep - written;
            equals = all_equal;
        }
        __syncthreads();
        // whole blocks of the destination, and what is left at the end
        int done = 0;
        while (queued - done >= B || (j0 + EV_TURN >= len && queued > done)) {
            const int n = queued - done < B ? queued - done : B;
            const int at = written % p.P;  // the block's first token in its page
            if (at == 0) {
                page = page_of(p, dst, written / p.P);
                if (page >= 0 && p.refs[page] != 1) {
                    if (tid == 0) atomicOr(p.status, PST_SHARED);
                    page = -1;
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    top[i] = 0xfc00fc00u;
                    low[i] = 0x7c007c00u;
                }
            }
            uint8_t *blk = page < 0 ? nullptr : page_ptr(p, page, head) + at / B * L::size(B);
            auto from = [&](int u, const uint8_t *&b) -> int {  // block and place of the u-th waiting token
                const int id = page_q[done + u], t = token_q[done + u];
                b = id < 0 ? nullptr : page_ptr(p, id, head) + t / B * L::size(B);
                return t % B;
            };
            for (int i = tid; i < n * (D / 32); i += EV_THREADS) {
                const uint8_t *b;
                const int u = i / (D / 32), c = i % (D / 32), t = from(u, b);
                const uint4 w = b ? *reinterpret_cast<const uint4 *>(b + t * (D / 2) + 16 * c) : make_uint4(0, 0, 0, 0);
                reinterpret_cast<uint4 *>(img)[i] = w;
                if (blk) reinterpret_cast<uint4 *>(blk)[i] = w;
            }
            for (int i = tid; i < n * (D / 64); i += EV_THREADS) {  // four scales
                const uint8_t *b;
                const int u = i / (D / 64), c = i % (D / 64), t = from(u, b);
                const uint32_t w = b ? *reinterpret_cast<const uint32_t *>(b + L::ks(B) + t * C + 4 * c) : 0u;
                reinterpret_cast<uint32_t *>(img + 64 * D / 2)[i] = w;
                if (blk) reinterpret_cast<uint32_t *>(blk + L::ks(B))[i] = w;
            }
            // values: (8 tokens, scale block, pair) in the order of the bytes
            for (int i = tid; i < (n + 1) / 2 * C; i += EV_THREADS) {
                // the last group of 8 may be short of pairs
                const int pairs = (n + 1) / 2, g = i / (4 * C), left = pairs - 4 * g < 4 ? pairs - 4 * g : 4;
                const int in = i - g * 4 * C, c = in / left, pr = 4 * g + in % left;
                const uint8_t *b0, *b1 = nullptr;
                const bool two = 2 * pr + 1 < n;
                const int t0 = from(2 * pr, b0), t1 = two ? from(2 * pr + 1, b1) : 0;
                const uint4 x = b0 ? *reinterpret_cast<const uint4 *>(b0 + L::vc(B) + L::vcode(t0, c)) : make_uint4(0, 0, 0, 0);
                const uint32_t s0 = b0 ? b0[L::vs(B) + L::vscale(t0, c)] : 0u;
                if (!blk) continue;
                uint4 *to = reinterpret_cast<uint4 *>(blk + L::vc(B) + L::vcode(2 * pr, c));
                uint8_t *to_s = blk + L::vs(B) + L::vscale(2 * pr, c);
                uint4 y;
                uint32_t s1;
                int odd;
                if (two) {
                    y = b1 ? *reinterpret_cast<const uint4 *>(b1 + L::vc(B) + L::vcode(t1, c)) : make_uint4(0, 0, 0, 0);
                    s1 = b1 ? b1[L::vs(B) + L::vscale(t1, c)] : 0u;
                    odd = t1 & 1;
                } else {  // the place behind the last token stays as it is
                    y = *to;
                    s1 = to_s[1];
                    odd = 1;
                }
                const int sx = 4 * (t0 & 1), sy = 4 * odd;
                auto both = [&](uint32_t u, uint32_t v) { return (u >> sx & 0x0f0f0f0fu) | (v >> sy & 0x0f0f0f0fu) << 4; };
                *to = make_uint4(both(x.x, y.x), both(x.y, y.y), both(x.z, y.z), both(x.w, y.w));
                *reinterpret_cast<uint16_t *>(to_s) = static_cast<uint16_t>(s0 | s1 << 8);
            }
            __syncthreads();
            for (int t = tid / (D / 8); t < n; t += EV_THREADS / (D / 8)) {
                uint32_t h[4];
                e2m1x8_to_half(*reinterpret_cast<const uint32_t *>(img + t * (D / 2) + 4 * col), h);
                const uint32_t s = e4m3x2_to_half2(img[64 * D / 2 + t * C + (col >> 1)]), s2 = __byte_perm(s, s, 0x1010);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    h[i] = hmul2(h[i], s2);  // exact
                    top[i] = hmax2(top[i], h[i]);
                    low[i] = hmin2(low[i], h[i]);
                }
            }
            written += n;
            done += n;
            if (written % p.P == 0 || written == keep) {  // the page is done: its summary
#pragma unroll
                for (int i = 0; i < 4; i++) {
#pragma unroll
                    for (int o = D / 8; o < 32; o <<= 1) {
                        top[i] = hmax2(top[i], __shfl_xor_sync(FULL, top[i], o));
                        low[i] = hmin2(low[i], __shfl_xor_sync(FULL, low[i], o));
                    }
                    if (lane < D / 8) {
                        const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&top[i])), l = __half22float2(*reinterpret_cast<const __half2 *>(&low[i]));
                        top_s[warp][8 * lane + 2 * i] = h.x;
                        top_s[warp][8 * lane + 2 * i + 1] = h.y;
                        low_s[warp][8 * lane + 2 * i] = l.x;
                        low_s[warp][8 * lane + 2 * i + 1] = l.y;
                    }
                }
                __syncthreads();
                float mx = -INFINITY, mn = INFINITY;
                if (tid < D)
#pragma unroll
                    for (int i = 0; i < EV_WARPS; i++) {
                        mx = fmaxf(mx, top_s[i][tid]);
                        mn = fminf(mn, low_s[i][tid]);
                    }
                const float w = warp_max(tid < D ? fmaxf(fabsf(mx), fabsf(mn)) : 0.f);
                if (lane == 0) red[warp] = w;
                __syncthreads();
                float most = red[0];
#pragma unroll
                for (int i = 1; i < EV_WARPS; i++) most = fmaxf(most, red[i]);
                // (held keys are multiples of 2^-10 below 2^12: as append has it)
                const int e = most > 0.f ? static_cast<int>(__float_as_uint(most) >> 23) - 126 - 7 : 0;
                if (page >= 0) {
                    uint8_t *sum = summary_ptr(p, page, head);
                    if (tid < D) {
                        const float unit = pow2i(-e);
                        reinterpret_cast<int8_t *>(sum)[tid] = static_cast<int8_t>(ceilf(mx * unit));
                        reinterpret_cast<int8_t *>(sum)[D + tid] = static_cast<int8_t>(floorf(mn * unit));
                    }
                    if (tid == 0) *reinterpret_cast<int *>(sum + 2 * D) = e;
                }
            }
            __syncthreads();
        }
        // what waits moves to the front
        const int left = queued - done;
        int id = 0, t = 0;
        if (tid < left) {
            id = page_q[done + tid];
            t = token_q[done + tid];
        }
        __syncthreads();
        if (done > 0 && tid < left) {
            page_q[tid] = id;
            token_q[tid] = static_cast<uint8_t>(t);
        }
        queued = left;
    }
}

}  // namespace

int launch_pages_evict(const PagesEvictArgs &a, int num_sms, void *stream) {
    (void)num_sms;
    const dim3 grid(a.n, a.p.Hkv, a.p.n_layers);
    auto st = static_cast<cudaStream_t>(stream);
    if (a.p.d == 128) evict_kernel<128><<<grid, EV_THREADS, 0, st>>>(a);
    else evict_kernel<64><<<grid, EV_THREADS, 0, st>>>(a);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace dq
