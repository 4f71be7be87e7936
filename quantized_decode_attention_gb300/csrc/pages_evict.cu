// Paged cache: the tokens of a row with the highest scores, into the pages of another.
//
// Row dst has room for k tokens.  For each layer and KV head it gets, in order, the first
// keep_first and the last keep_last tokens of row src and of those between them the
// k - keep_first - keep_last with the highest scores (the earlier where scores are equal),
// with their scores and the pages' summaries.
//
// choose_kernel, one CTA per (pair, KV head, layer): the border between kept and evicted
// scores, found digit by digit (2048 counts a digit; the scores are held in shared memory as
// far as they fit), then the kept positions in order.
// They go where the kept tokens' scores are to stand, so that no list needs room.
// gather_kernel, a CTA a page of dst at a time: positions, page numbers, then 16-byte
// pieces straight from the source pages to the destination's (keys and scales as they are,
// values two tokens a byte), the scores over the positions, and the page's summary.  The
// pages are independent.  What it reads is scattered: kept tokens are rarely neighbours, and a
// value's sector of 32 bytes holds 4 tokens' channels (keeping an eighth reads 289 MB where 145 are kept); where
// nearly all are kept it is instructions, the nibbles of values and the summaries, that count (60 % of the issue slots).
//
// 16 rows of 4160 tokens to 4096, two layers of 8 KV heads, head_dim 128: 91 us, some 14 of them to choose; four
// prompts of 16384 to 2048, eight layers: 92, 28 to choose.
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

// The variants below go by `cap`, the length of the caller's scores, for which the host knows no better: rows much shorter than it
// pay for one that could be long.  16 rows of 4160 tokens, two layers, with cap 4160 91 us, 32768 97, 131072 105; 64 of 1024 to 512 with
// cap 1024 63, 32768 80, 131072 104; 4 of 16384 to 2048, eight layers, with 16384 92, 131072 105.  (Below, cap is the rows' length.)
constexpr int CH_HELD = 48 << 10;  // keys of scores that shared memory holds, at most
// Longest rows (at most `cap` tokens) that 512 threads choose from, 1024 for longer ones.  512 / 1024, the whole eviction in us: 16 rows
// of 1024 tokens, two layers, 28 / 36, of 4160 91 / 97; 4 of 16384, eight layers, 92 / 98; 1 of 32768, two layers, 34 to 38 / 35, of
// 65536 112 / 66 to 75.  (256: 4 % less at 64 rows of 1024, more elsewhere.)
constexpr int CH_LONG = 32768;
// Keys held for which the gather's CTAs may come in while scores are chosen from: beside more shared memory their L1 is too
// small for the sectors that two tokens share.  Beside / after, us: 16 rows of 4160 tokens 91 / 93, of 6144 98 / 99; 4 of 8192 74 / 70,
// of 16384 121 / 92; 1 of 131072 183 / 170.
constexpr int CH_BESIDE = 6144;
constexpr int BIN_BITS = 11, BINS = 1 << BIN_BITS;

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

template <int T>
struct ChooseShared {
    int hist[BINS];
    int above[T / 32], equal[T / 32];
    uint32_t digit;
    int digit_above, digit_count;
};

// `held`: keys that the dynamic shared memory has room for behind the struct.
template <int T>
__global__ void __launch_bounds__(T, 2048 / T) choose_kernel(PagesEvictArgs a, int held) {
    constexpr int CH_WARPS = T / 32;
    extern __shared__ __align__(16) uint8_t raw[];
    using S = ChooseShared<T>;
    S &sh = *reinterpret_cast<S *>(raw);
    uint32_t *key = reinterpret_cast<uint32_t *>(raw + sizeof(S));
    const PagesView &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.y, layer = blockIdx.z, src = a.src[blockIdx.x], dst = a.dst[blockIdx.x];
    if (held <= CH_BESIDE) let_next_start();
    for (int i = tid; i < BINS; i += T) sh.hist[i] = 0;
    // is dst in order: a row of its own, named once?
    bool bad = src >= p.max_seqs || dst >= p.max_seqs || src == dst;
    for (int i = tid; i < a.n; i += T) {
        if (a.src[i] < 0 || a.dst[i] < 0) continue;
        bad |= a.src[i] == dst || (a.dst[i] == dst && i != static_cast<int>(blockIdx.x));
    }
    int len = 0, keep = 0;
    if (src >= 0 && dst >= 0) {
        if (!bad) {
            len = p.seq_len[src];
            keep = p.seq_len[dst];
            bad = len < 0 || len > p.M * p.P || keep < 0 || keep > len || len > a.cap || (keep < len && a.keep_first + a.keep_last > keep);
        }
        bad = __syncthreads_or(bad);
        if (bad && tid == 0) atomicOr(p.status, PST_ARG);
    } else {
        bad = true;
    }
    if (bad) keep = 0;
    if (tid == 0 && head == 0 && layer == 0) a.keeps[blockIdx.x] = keep;
    if (keep == 0) return;
    const long long at = static_cast<long long>(layer) * p.max_seqs;
    const float *scores = a.scores + ((at + src) * p.Hkv + head) * a.cap;
    int *out = reinterpret_cast<int *>(a.scores) + ((at + dst) * p.Hkv + head) * a.cap;
    if (keep == len) {
        for (int j = tid; j < len; j += T) out[j] = j;
        return;
    }
    // the tokens between the ones that are kept anyway
    const int lo = a.keep_first, n = len - a.keep_last - lo;
    const float *mid = scores + lo;
    auto key_at = [&](int j) { return j < held ? key[j] : order_key(mid[j]); };
    // The take-th largest key, a digit at a time: it is in [least, least + range], whose keys above it are counted off.
    uint32_t least = 0, range = 0xffffffffu;
    int take = keep - a.keep_first - a.keep_last, count = n;
    for (int shift = 32 - BIN_BITS; take > 0 && take < count;) {
        if (range == 0xffffffffu) {  // the first digit, as the scores come in
#pragma unroll 8
            for (int j = tid; j < n; j += T) {
                const uint32_t k = order_key(mid[j]);
                if (j < held) key[j] = k;
                atomicAdd(&sh.hist[k >> shift], 1);
            }
        } else {
#pragma unroll 4
            for (int j = tid; j < n; j += T) {
                const uint32_t k = key_at(j) - least;
                if (k <= range) atomicAdd(&sh.hist[k >> shift], 1);
            }
        }
        __syncthreads();
        // thread t: bins BINS - 1 - 4 t and the three below it
        constexpr int PER = BINS / T;
        int c[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; i++) sum += c[i] = sh.hist[BINS - 1 - PER * tid - i];
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(FULL, before, o);
            if (lane >= o) before += t;
        }
        if (lane == 31) sh.above[warp] = before;
        __syncthreads();
        before -= sum;
#pragma unroll
        for (int w = 0; w < CH_WARPS; w++) before += w < warp ? sh.above[w] : 0;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            if (before < take && before + c[i] >= take) {
                sh.digit = BINS - 1 - PER * tid - i;
                sh.digit_above = before;
                sh.digit_count = c[i];
            }
            before += c[i];
            sh.hist[BINS - 1 - PER * tid - i] = 0;
        }
        __syncthreads();
        least += sh.digit << shift;
        take -= sh.digit_above;
        count = sh.digit_count;
        range = (1u << shift) - 1u;
        if (shift == 0) break;
        shift = shift > BIN_BITS ? shift - BIN_BITS : 0;
    }
    // Kept: keys over least + range, and of those in [least, least + range], of which there are `count`, the first `take` (all of
    // them, or all are equal).
    // A warp's tokens are neighbours: [b0, b1).
    const int b0 = static_cast<int>(static_cast<long long>(len) * warp / CH_WARPS), b1 = static_cast<int>(static_cast<long long>(len) * (warp + 1) / CH_WARPS);
    const bool none = take == 0 && range == 0xffffffffu;  // of those between
    auto look = [&](int j, bool &above, bool &equal) {
        const bool in = j >= lo && j < lo + n, is = j < b1;
        const uint32_t k = is && in && !none ? key_at(j - lo) : 0u;
        equal = is && in && !none && k - least <= range;
        above = is && (!in || (!none && !equal && k > least));
    };
    int na = 0, ne = 0;
#pragma unroll 4
    for (int j = b0; j < b1; j += 32) {
        bool above, equal;
        look(j + lane, above, equal);
        na += __popc(__ballot_sync(FULL, above));
        ne += __popc(__ballot_sync(FULL, equal));
    }
    __syncthreads();
    if (lane == 0) {
        sh.above[warp] = na;
        sh.equal[warp] = ne;
    }
    __syncthreads();
    na = ne = 0;
    for (int w = 0; w < warp; w++) {
        na += sh.above[w];
        ne += sh.equal[w];
    }
    const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
    for (int j = b0; j < b1; j += 32) {
        bool above, equal;
        look(j + lane, above, equal);
        const unsigned ma = __ballot_sync(FULL, above), me = __ballot_sync(FULL, equal);
        const int before_a = na + __popc(ma & below), before_e = ne + __popc(me & below);
        const int to = before_a + (before_e < take ? before_e : take);
        if ((above || (equal && before_e < take)) && to < keep) out[to] = j + lane;  // (to < keep unless scores change under the call)
        na += __popc(ma);
        ne += __popc(me);
    }
}

constexpr int GA_THREADS = 128, GA_WARPS = GA_THREADS / 32, GA_CTAS = 8;  // CTAs of an SM (6: 2 % slower, 10, with spills: 30 %)

// One CTA row of the grid per (KV head, layer), which walks the pages of all pairs, a block of B = min(P, 64) tokens
// at a time.  Two blocks ahead the positions are on their way, one ahead the page numbers and scores.
template <int D, int B>
__global__ void __launch_bounds__(GA_THREADS, GA_CTAS) gather_kernel(PagesEvictArgs a) {
    using L = PageBlock<D>;
    constexpr int C = D / 16;
    extern __shared__ __align__(16) uint8_t dyn[];         // [n] src, dst, keep, pages before the pair
    __shared__ __align__(16) uint8_t img[B * D * 9 / 16];  // a block's key codes, then their scales
    __shared__ float red[GA_WARPS];
    __shared__ long long from_s[B];                        // where a token's block is in the pool: -1 none
    __shared__ int2 place_s[B];                            // its place there, and that of its values' first scale in the block's
    __shared__ int part[GA_WARPS];
    const PagesView &p = a.p;
    int4 *pair = reinterpret_cast<int4 *>(dyn);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, head = blockIdx.y, layer = blockIdx.z;
    await_previous();
    int pages = 0;
    for (int i0 = 0; i0 < a.n; i0 += GA_THREADS) {
        const int i = i0 + tid, keep = i < a.n ? a.keeps[i] : 0, w = (keep + p.P - 1) / p.P;
        int s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(FULL, s, o);
            if (lane >= o) s += t;
        }
        if (lane == 31) part[warp] = s;
        __syncthreads();
        int before = pages;
#pragma unroll
        for (int k = 0; k < GA_WARPS; k++) {
            if (k < warp) before += part[k];
            pages += part[k];
        }
        if (i < a.n) pair[i] = make_int4(a.src[i], a.dst[i], keep, before + s - w);
        __syncthreads();
    }
    const long long at_layer = static_cast<long long>(layer) * p.max_seqs, pool = static_cast<long long>(layer) * p.n_pages;
    auto scores_of = [&](int row) { return a.scores + ((at_layer + row) * p.Hkv + head) * a.cap; };
    const int shift = 31 - __clz(p.P);  // (a power of two)
    struct Step {
        int x, src, dst, keep, ord, b0;  // page of all pairs' pages; its pair; its ordinal; the block's first token in it
    };
    auto seek = [&](Step &s) {
        if (s.x >= pages) return;
        int lo = 0, hi = a.n - 1;
        while (lo < hi) {  // the last pair that begins at or before x
            const int mid = (lo + hi + 1) >> 1;
            if (pair[mid].w <= s.x) lo = mid;
            else hi = mid - 1;
        }
        const int4 q = pair[lo];
        s.src = q.x;
        s.dst = q.y;
        s.keep = q.z;
        s.ord = s.x - q.w;
        s.b0 = 0;
    };
    auto tokens = [&](const Step &s) {  // from the block's first token to the page's end
        const int left = s.keep - (s.ord << shift);
        return (left < p.P ? left : p.P) - s.b0;
    };
    auto step = [&](Step &s) {
        if (tokens(s) > B) {
            s.b0 += B;
        } else {
            s.x += gridDim.x;
            seek(s);
        }
    };
    auto position = [&](const Step &s) {  // of this thread's token
        return s.x < pages && tid < B && tid < tokens(s) ? __float_as_int(scores_of(s.dst)[(s.ord << shift) + s.b0 + tid]) : -1;
    };
    struct Found {
        int id, refs, page, place;
        float score;
    };
    auto look = [&](const Step &s, int j, int page, Found &f) {
        f.id = -1;
        f.refs = 0;
        f.page = page;
        f.place = 0;
        if (s.x >= pages) return;
        if (j >= 0 && j < p.M * p.P && j < a.cap) {  // (it is what choose_kernel wrote)
            f.id = p.table[static_cast<long long>(s.src) * p.M + (j >> shift)];
            f.place = j & (p.P - 1);
            f.score = scores_of(s.src)[j];
            if (f.id < 0 || f.id >= p.n_pages) f.id = -2;
        }
        if (page >= 0 && page < p.n_pages) f.refs = p.refs[page];
    };
    auto number = [&](const Step &s) { return s.x < pages ? p.table[static_cast<long long>(s.dst) * p.M + s.ord] : -1; };

    constexpr int PAIRS = B / 2 * C, KEYS = B * (D / 32), SCALES = B * (D / 64);  // pieces of values and keys, words of scales
    constexpr int NV = (PAIRS + GA_THREADS - 1) / GA_THREADS, NK = (KEYS + GA_THREADS - 1) / GA_THREADS;
    static_assert(SCALES <= GA_THREADS, "a thread a word");
    // summary: a warp's COLS columns of 8 channels, each over every 32 / COLS-th token
    constexpr int COLS = D / 8 / GA_WARPS;
    const int col = warp * COLS + lane % COLS;
    uint32_t top[4], low[4];
    Step now, next;
    now.x = blockIdx.x;
    seek(now);
    Found f;
    look(now, position(now), number(now), f);
    next = now;
    if (now.x < pages) step(next);
    int j = position(next), page_next = number(next);
    while (now.x < pages) {
        const int left = tokens(now), n = left < B ? left : B;
        int page = f.page;
        if (page < 0 || page >= p.n_pages || f.refs != 1) {
            if (tid == 0) atomicOr(p.status, page < 0 || page >= p.n_pages ? PST_TABLE : PST_SHARED);
            page = -1;
        }
        if (now.b0 == 0) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                top[i] = 0xfc00fc00u;
                low[i] = 0x7c007c00u;
            }
        }
        uint8_t *blk = page < 0 ? nullptr : p.pages + ((pool + page) * p.Hkv + head) * p.page_bytes + now.b0 / B * L::size(B);
        if (tid < B) {
            if (f.id == -2) atomicOr(p.status, PST_TABLE);
            from_s[tid] = f.id < 0 ? -1 : ((pool + f.id) * p.Hkv + head) * p.page_bytes + f.place / B * L::size(B);
            const int t = f.place % B;
            place_s[tid] = make_int2(t, L::vscale(t, 0));
            if (f.id != -1) scores_of(now.dst)[(now.ord << shift) + now.b0 + tid] = f.score;
        }
        __syncthreads();
        // everything that the block needs is loaded before anything is stored
        uint4 v[NV], w[NV], k[NK];
        uint32_t s0[NV], s1[NV], ks = 0;
#pragma unroll
        for (int e = 0; e < NV; e++) {  // values: (8 tokens, scale block, pair) in the order of the bytes
            const int i = tid + e * GA_THREADS, in = i % (4 * C), c = in >> 2, pr = 4 * (i / (4 * C)) + (in & 3);
            v[e] = w[e] = make_uint4(0, 0, 0, 0);
            s0[e] = s1[e] = 0;
            if (i >= PAIRS) continue;
            const long long f0 = from_s[2 * pr], f1 = from_s[2 * pr + 1];
            // (a scale block further on is 8 scales and 4 x 16 bytes of codes)
            if (f0 >= 0) {
                const int at = place_s[2 * pr].y;
                v[e] = *reinterpret_cast<const uint4 *>(p.pages + f0 + (L::vc(B) + (at >> 1) * 16 + c * 64));
                s0[e] = p.pages[f0 + (L::vs(B) + at + c * 8)];
            }
            if (f1 >= 0) {
                const int at = place_s[2 * pr + 1].y;
                w[e] = *reinterpret_cast<const uint4 *>(p.pages + f1 + (L::vc(B) + (at >> 1) * 16 + c * 64));
                s1[e] = p.pages[f1 + (L::vs(B) + at + c * 8)];
            }
        }
#pragma unroll
        for (int e = 0; e < NK; e++) {
            const int i = tid + e * GA_THREADS, u = i / (D / 32);
            k[e] = make_uint4(0, 0, 0, 0);
            if (i < KEYS && from_s[u] >= 0) k[e] = *reinterpret_cast<const uint4 *>(p.pages + from_s[u] + (place_s[u].x * (D / 2) + 16 * (i % (D / 32))));
        }
        if (tid < SCALES) {  // four scales
            const int u = tid / (D / 64);
            if (from_s[u] >= 0) ks = *reinterpret_cast<const uint32_t *>(p.pages + from_s[u] + (L::ks(B) + place_s[u].x * C + 4 * (tid % (D / 64))));
        }
        const bool last = left <= B;
        look(next, j, page_next, f);
        now = next;
        if (next.x < pages) step(next);
        j = position(next);
        page_next = number(next);
#pragma unroll
        for (int e = 0; e < NV; e++) {
            const int i = tid + e * GA_THREADS, pr = 4 * (i / (4 * C)) + (i & 3);
            if (i >= PAIRS || 2 * pr >= n || !blk) continue;
            // (the bytes' order is the items')
            uint4 *to = reinterpret_cast<uint4 *>(blk + L::vc(B)) + i;
            uint8_t *to_s = blk + L::vs(B) + 2 * i;
            int odd = place_s[2 * pr + 1].y & 1;
            if (2 * pr + 1 >= n) {  // the place behind the last token stays as it is
                w[e] = *to;
                s1[e] = to_s[1];
                odd = 1;
            }
            const int sv = 4 * (place_s[2 * pr].y & 1), sw = 4 * odd;
            auto both = [&](uint32_t x, uint32_t y) { return (x >> sv & 0x0f0f0f0fu) | (y >> sw & 0x0f0f0f0fu) << 4; };
            *to = make_uint4(both(v[e].x, w[e].x), both(v[e].y, w[e].y), both(v[e].z, w[e].z), both(v[e].w, w[e].w));
            *reinterpret_cast<uint16_t *>(to_s) = static_cast<uint16_t>(s0[e] | s1[e] << 8);
        }
#pragma unroll
        for (int e = 0; e < NK; e++) {
            const int i = tid + e * GA_THREADS;
            if (i >= n * (D / 32)) continue;
            reinterpret_cast<uint4 *>(img)[i] = k[e];
            if (blk) reinterpret_cast<uint4 *>(blk)[i] = k[e];
        }
        if (tid < n * (D / 64)) {
            reinterpret_cast<uint32_t *>(img + B * D / 2)[tid] = ks;
            if (blk) reinterpret_cast<uint32_t *>(blk + L::ks(B))[tid] = ks;
        }
        __syncthreads();
#pragma unroll 2
        for (int t = lane / COLS; t < n; t += 32 / COLS) {
            uint32_t h[4];
            e2m1x8_to_half(*reinterpret_cast<const uint32_t *>(img + t * (D / 2) + 4 * col), h);
            const uint32_t sc = e4m3x2_to_half2(img[B * D / 2 + t * C + (col >> 1)]), sc2 = __byte_perm(sc, sc, 0x1010);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                h[i] = hmul2(h[i], sc2);  // exact
                top[i] = hmax2(top[i], h[i]);
                low[i] = hmin2(low[i], h[i]);
            }
        }
        if (!last) {
            __syncthreads();  // (the next block's keys take the place of these)
            continue;
        }
        // the page's summary, as append has it
        float mx[8], mn[8], most = 0.f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
#pragma unroll
            for (int o = COLS; o < 32; o <<= 1) {
                top[i] = hmax2(top[i], __shfl_xor_sync(FULL, top[i], o));
                low[i] = hmin2(low[i], __shfl_xor_sync(FULL, low[i], o));
            }
            const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&top[i])), l = __half22float2(*reinterpret_cast<const __half2 *>(&low[i]));
            mx[2 * i] = h.x;
            mx[2 * i + 1] = h.y;
            mn[2 * i] = l.x;
            mn[2 * i + 1] = l.y;
            most = fmaxf(most, fmaxf(fmaxf(fabsf(h.x), fabsf(h.y)), fmaxf(fabsf(l.x), fabsf(l.y))));
        }
        most = warp_max(most);
        if (lane == 0) red[warp] = most;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < GA_WARPS; i++) most = fmaxf(most, red[i]);
        // (held keys are multiples of 2^-10 below 2^12)
        const int e = most > 0.f ? static_cast<int>(__float_as_uint(most) >> 23) - 126 - 7 : 0;
        if (page >= 0) {
            uint8_t *sum = p.summary + ((pool + page) * p.Hkv + head) * p.sum_bytes;
            if (lane < COLS) {
                const float unit = pow2i(-e);
                uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    b[i >> 2] |= (static_cast<uint32_t>(static_cast<int>(ceilf(mx[i] * unit))) & 0xffu) << (8 * (i & 3));
                    b[2 + (i >> 2)] |= (static_cast<uint32_t>(static_cast<int>(floorf(mn[i] * unit))) & 0xffu) << (8 * (i & 3));
                }
                *reinterpret_cast<uint2 *>(sum + 8 * col) = make_uint2(b[0], b[1]);
                *reinterpret_cast<uint2 *>(sum + D + 8 * col) = make_uint2(b[2], b[3]);
            }
            if (tid == 0) *reinterpret_cast<int *>(sum + 2 * D) = e;
        }
    }
}

template <int D, int B>
int launch_gather(const PagesEvictArgs &a, int num_sms, cudaStream_t st) {
    const long long units = static_cast<long long>(a.p.Hkv) * a.p.n_layers, room = static_cast<long long>(GA_CTAS) * num_sms;
    const dim3 grid(static_cast<unsigned>(units < room ? room / units : 1), a.p.Hkv, a.p.n_layers);
    return launch_overlapping(gather_kernel<D, B>, grid, GA_THREADS, a.n * 16, st, a);
}
template <int D>
int launch_gather_of(const PagesEvictArgs &a, int num_sms, cudaStream_t st) {
    return a.p.blk == 64 ? launch_gather<D, 64>(a, num_sms, st) : (a.p.blk == 32 ? launch_gather<D, 32>(a, num_sms, st) : launch_gather<D, 16>(a, num_sms, st));
}

template <int T>
int launch_choose(const PagesEvictArgs &a, cudaStream_t st) {
    const int held = a.cap < CH_HELD ? a.cap : CH_HELD, smem = static_cast<int>(sizeof(ChooseShared<T>));
    if (const int e = allow_shared<choose_kernel<T>>(smem + CH_HELD * 4)) return e;
    choose_kernel<T><<<dim3(a.n, a.p.Hkv, a.p.n_layers), T, smem + held * 4, st>>>(a, held);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_pages_evict(const PagesEvictArgs &a, int num_sms, void *stream) {
    auto st = static_cast<cudaStream_t>(stream);
    if (const int e = a.cap > CH_LONG ? launch_choose<1024>(a, st) : launch_choose<512>(a, st)) return e;
    return a.p.d == 128 ? launch_gather_of<128>(a, num_sms, st) : launch_gather_of<64>(a, num_sms, st);
}

}  // namespace dq
