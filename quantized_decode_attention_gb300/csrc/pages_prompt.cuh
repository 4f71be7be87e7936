// Paged cache: attention of many new tokens (a prompt's chunk) over 4-bit pages, on the
// 5th-generation tensor cores.
//
// Same mathematics as the kernel for few tokens: z = f q . k, p = exp2(z - m + LIFT),
// out = (sum p v) / (sum p).  4 D products and one exponential for each (query, key)
// pair: the kernel is bound by the tensor cores and, nearly as much, by the exponentials
// and their conversions.  2048 new tokens over 16384 (32 / 8 heads, head_dim 128) take
// 400 us, 1.29 PFLOP/s.
//
// Work.  A unit is 256 query rows (256 / G tokens with their G query heads) of one row and
// KV head, in two tiles of 128.  It walks the keys that its last token sees, 128 at a
// time.  Units stand on a line, each as long as its keys (causal: later blocks are longer),
// and the line is cut into equal shares, one for each CTA (one per SM); a unit that
// crosses a border leaves its parts in the workspace, and a second kernel adds them up in
// CTA order.
//
// Roles of the 16 warps.  Warps 0-3 and 4-7: softmax of tile 0 and 1, a thread a query
// row: scores come from tensor memory, weights go back there as binary16 in the place of
// the scores, the accumulator is rescaled in place when a logit passes the maximum by
// more than 2^8.  Warps 8-11: codes of 128 keys and values from the pages to binary16 operands in
// shared memory (exact), two stages deep.  Warp 12: one thread issues all products,
// S = Q K^T and O += P V (P from tensor memory), tile by tile in turn, so that one tile's
// softmax runs beside the other's products.
// Tensor memory: S0 S1 (128 columns each, P in the first 64), O0 O1 (D columns).
// Shared memory: operands in the 128-byte-swizzled K-major layout, values transposed
// (a page holds two tokens of a channel side by side, which is that layout's order).
#pragma once

#include <cuda_runtime.h>

#include "pages_tc.cuh"

namespace dq {
namespace {

constexpr float LN2 = 0.69314718055994530942f;
constexpr float LIFT = 7.f;       // log2 units: weights are 2^LIFT at a logit of m ...
constexpr float MOST = 32768.f;   // ... and may grow to 2^15 (a logit 2^8 over m) before m is raised
constexpr int TILE = 128, ROWS = 2 * TILE;   // query rows of a tile, of a unit
constexpr int KEYS = 128;                    // keys at a time
constexpr int UNIT_COST = 512, MIN_SHARE = 1024;  // tokens: of a unit's beginning and end; that make a CTA worth its parts
constexpr int MIN_SHARE_COMMON = 512;  // of pages in common, whose parts are joined in any case (64 rows over 8192 tokens: 4 % less than 1024)
constexpr int THREADS = 512;

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

// One query row's running softmax: m and the sum of weights in two halves.
struct RowState {
    float f, m;
    uint64_t l[2];
    __device__ __forceinline__ float mu() const { return m == -INFINITY ? 0.f : m - LIFT; }  // what a logit loses before exp2
    __device__ __forceinline__ float sum() const {
        const float2 a = both(l[0]), b = both(l[1]);
        return (a.x + a.y) + (b.x + b.y);
    }
    // A weight grew too large (in some row of the warp), z is the largest logit: raise m; the sums, the accumulator (n_o columns at o_at)
    // and this tile's weights so far (n_p columns of two at p_at) follow.
    template <int D>
    __device__ void raise(float z, bool has_o, uint32_t o_at, int n_p, uint32_t p_at) {
        const float mx = fmaxf(m, z), al = mx == -INFINITY ? 1.f : ex2(m - mx);
        m = mx;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float2 x = both(l[i]);
            l[i] = two(x.x * al, x.y * al);
        }
        tmem_wait_st();
        uint32_t s[16];
        if (has_o) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                tmem_ld16(o_at + c, s);
                tmem_wait_ld(s);
#pragma unroll
                for (int i = 0; i < 16; i++) s[i] = __float_as_uint(__uint_as_float(s[i]) * al);
                tmem_st16(o_at + c, s);
            }
        }
#pragma unroll 1
        for (int c = 0; c < n_p; c += 16) {
            tmem_ld16(p_at + c, s);
            tmem_wait_ld(s);
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&s[i]));
                s[i] = half2_of(x.x * al, x.y * al);
            }
            tmem_st16(p_at + c, s);
        }
    }
    // Scores of 32 keys -> weights, two a word, and their sums.
    __device__ __forceinline__ void weigh(const uint32_t (&s)[32], uint32_t (&w)[16], uint64_t (&c)[2]) const {
        const float lose = -mu();
        const uint64_t ff = two(f, f), mm = two(lose, lose);
        c[0] = c[1] = 0;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float2 e = both(fma2(two(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), ff, mm));
            const float a = ex2(e.x), b = ex2(e.y);
            c[i & 1] = add2(c[i & 1], two(a, b));
            w[i] = half2_of(a, b);
        }
    }
};
__device__ __forceinline__ float top_of(const uint32_t (&s)[32]) {
    float t[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        t[i] = fmaxf(__uint_as_float(s[8 * i]), __uint_as_float(s[8 * i + 1]));
#pragma unroll
        for (int j = 2; j < 8; j += 2) t[i] = fmaxf(t[i], fmaxf(__uint_as_float(s[8 * i + j]), __uint_as_float(s[8 * i + j + 1])));
    }
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

// A warp's 32 query rows of a block of tokens from tok0 on, as binary16 operands in shared memory: each by a power of two
// below 2^14 and with sm_scale's sign.  Returns this lane's row's logit unit.  A row is D / 8 lanes' 16 bytes, so that whole
// lines are read; two elements go at a time (where a CTA has few keys this is a good part of its time).
template <int D, bool BF16, class A>
__device__ __forceinline__ float put_queries(const A &a, const PageRow &r, int head, int tok0, int tb, uint8_t *to) {
    constexpr int LANES = D / 8, PER = 32 / LANES, DEEP = 4;
    const int G = a.p.G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, piece = lane % LANES, sub = lane / LANES, row0 = (warp & 7) * 32;
    const unsigned inv = 65536 / G + 1;  // i / G = i inv / 65536 for i below 256
    const uint16_t *src = a.q + (static_cast<long long>(r.q0) + tok0) * a.qt + head * G * a.qh + 8 * piece;
    float f = 0.f;
    // every line of the 32 rows is sent for at once, a row a lane, so that the loads below wait once for all
    {
        const unsigned i = row0 + lane, tk = i * inv >> 16, h = i - tk * G;
        if (static_cast<int>(tk) < tb && tok0 + static_cast<int>(tk) < r.n) {
            const uint16_t *at = src - 8 * piece + tk * a.qt + h * a.qh;
#pragma unroll
            for (int k = 0; k < D / 64; k++) {
                uint32_t x;
                asm volatile("ld.global.b32 %0, [%1];\n" : "=r"(x) : "l"(at + 64 * k));
            }
        }
    }
#pragma unroll 1
    for (int i0 = 0; i0 < 32; i0 += PER * DEEP) {
        uint4 w[DEEP];
#pragma unroll
        for (int k = 0; k < DEEP; k++) {
            const unsigned i = row0 + i0 + k * PER + sub, tk = i * inv >> 16, h = i - tk * G;
            const bool is = static_cast<int>(tk) < tb && tok0 + static_cast<int>(tk) < r.n;
            w[k] = is ? *reinterpret_cast<const uint4 *>(src + tk * a.qt + h * a.qh) : make_uint4(0, 0, 0, 0);
        }
        float top[DEEP];
#pragma unroll
        for (int k = 0; k < DEEP; k++) {
            const uint32_t m = max2_abs<BF16>(max2_abs<BF16>(w[k].x, w[k].y), max2_abs<BF16>(w[k].z, w[k].w));
            top[k] = fmaxf(from16(static_cast<uint16_t>(m & 0x7fffu), BF16), from16(static_cast<uint16_t>(m >> 16 & 0x7fffu), BF16));
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1)
#pragma unroll
            for (int k = 0; k < DEEP; k++) top[k] = fmaxf(top[k], __shfl_xor_sync(FULL, top[k], o));
#pragma unroll
        for (int k = 0; k < DEEP; k++) {
            int up = 13 - (static_cast<int>(__float_as_uint(top[k]) >> 23) - 127);
            up = top[k] > 0.f ? (up > 126 ? 126 : up) : 0;
            const float by = a.scale_log2 < 0.f ? -pow2i(up) : pow2i(up);
            const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float2 x = pair_to_float<BF16>(u[j]);
                h[j] = half2_of(x.x * by, x.y * by);
            }
            const int i = i0 + k * PER;
            *reinterpret_cast<uint4 *>(to + (piece >> 3) * (TILE * 128) + swizzled((warp & 3) * 32 + i + sub, piece & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
            const int mine = __shfl_sync(FULL, up, lane % PER * LANES);  // lane i + s has row i + s, whose lanes begin at s LANES
            if (lane >= i && lane < i + PER) f = fabsf(a.scale_log2) * pow2i(-mine);
        }
    }
    return f;
}

// ---- the line of units ---------------------------------------------------------------------
// Row i's units: blocks of `tb` tokens in order, KV heads within.  Block b is as long as
// the keys that a full block would see, plus UNIT_COST: base + (b + 1) tb.
struct Unit {
    PageRow r;
    int i, head, b;
    long long start, end;  // places
};

template <int D>
struct Shared {
    __align__(1024) uint8_t q[2][TILE * D * 2];
    __align__(1024) uint8_t k[2][KEYS * D * 2];
    __align__(1024) uint8_t v[2][KEYS * D * 2];  // panels of 64 keys, D rows
    long long first[DQ_PAGES_MAX_ROWS + 1];
    int row[DQ_PAGES_MAX_ROWS], keys[DQ_PAGES_MAX_ROWS];  // keys: tokens looked at
    long long part[THREADS / 32];
    uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], drained;
    uint32_t tmem;
};

__device__ __forceinline__ long long over(long long n, long long m) {  // n / m, both positive: 32 bits where they are enough
    return (n | m) >> 32 ? n / m : static_cast<unsigned>(n) / static_cast<unsigned>(m);
}
__device__ __forceinline__ long long blocks_before(long long base, int more, int b) {  // places of blocks 0 .. b - 1 of one head
    return b * (base + UNIT_COST) + static_cast<long long>(more) * b * (b + 1) / 2;
}
// Keys that every block of the row looks at, beside those that `more` a block add.
template <class A>
__device__ __forceinline__ long long base_of(const A &a, const PageRow &r) {
    const int seen = first_sees(a, r) + 1 - a.step;
    return (seen > 0 ? seen : 0) - r.from;
}
template <int D, class A>
__device__ Unit find_unit(const Shared<D> &sh, const A &a, int tb, long long x) {
    int lo = 0, hi = a.r.n_rows - 1;
    while (lo < hi) {  // the last row that begins at or before x
        const int mid = (lo + hi + 1) >> 1;
        if (sh.first[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    Unit u;
    u.i = lo;
    u.r = known_row(a, lo, sh.row[lo], sh.keys[lo]);
    const int more = tb * a.step;
    const long long base = base_of(a, u.r), in = x - sh.first[lo];
    int b0 = 0, b1 = (u.r.n - 1) / tb;
    while (b0 < b1) {
        const int mid = (b0 + b1 + 1) >> 1;
        if (a.p.Hkv * blocks_before(base, more, mid) <= in) b0 = mid;
        else b1 = mid - 1;
    }
    u.b = b0;
    const long long before = a.p.Hkv * blocks_before(base, more, b0), w = base + UNIT_COST + static_cast<long long>(b0 + 1) * more;
    u.head = static_cast<int>(over(in - before, w));
    u.start = sh.first[lo] + before + u.head * w;
    u.end = u.start + w;
    return u;
}
__device__ __forceinline__ long long share(long long n, int m, int k) {
    const long long q = over(n, m), rest = n - q * m;
    return k * q + (k < rest ? k : rest);
}
__device__ __forceinline__ int share_of(long long n, int m, long long x) {
    const long long q = over(n, m), rest = n - q * m, ahead = rest * (q + 1);
    return static_cast<int>(x < ahead ? over(x, q + 1) : rest + over(x - ahead, q));
}

// Maximum m and sum l of a part take another's in: the accumulators go by `keep` and `take`.
__device__ __forceinline__ void join_sums(float &m, float &l, float2 other, float &keep, float &take) {
    const float mx = fmaxf(m, other.x), mu = mx == -INFINITY ? 0.f : mx;
    keep = ex2(m - mu);  // 0 for a part that saw nothing
    take = ex2(other.x - mu);
    m = mx;
    l = l * keep + other.y * take;
}

// A segment: this CTA's part of a unit, key tiles [t0, t1).
struct Segment {
    Unit u;
    int t0, t1;
    bool begins, ends, two;  // two: the block has query rows in its second tile
};
template <int D, class A>
__device__ Segment find_segment(const Shared<D> &sh, const A &a, int tb, long long x, long long c1) {
    Segment s;
    s.u = find_unit<D>(sh, a, tb, x);
    s.begins = x <= s.u.start;
    s.ends = s.u.end <= c1;
    const int last = (s.u.b + 1) * tb < s.u.r.n ? (s.u.b + 1) * tb : s.u.r.n;
    const int seen = first_sees(a, s.u.r) + (a.step ? last : 1) - s.u.r.from;  // keys that the block's last token sees
    const int tiles = seen > 0 ? (seen + KEYS - 1) / KEYS : 0;
    auto tile_at = [&](long long at) {
        const long long t = (at - s.u.start - UNIT_COST + KEYS - 1) / KEYS;
        return at - s.u.start <= UNIT_COST ? 0 : (t < tiles ? static_cast<int>(t) : tiles);
    };
    s.two = (last - s.u.b * tb) * a.p.G > TILE;
    s.t0 = s.begins ? 0 : tile_at(x);
    s.t1 = s.ends ? tiles : tile_at(c1);
    return s;
}

// ---- the kernel --------------------------------------------------------------------------------
template <int D, int MODE>
__global__ void __launch_bounds__(THREADS, 1) attn_prompt(const InMode<MODE> a) {
    extern __shared__ uint8_t raw[];
    using S = Shared<D>;
    using B = PageBlock<D>;
    S &sh = *reinterpret_cast<S *>(raw + (-smem_u32(raw) & 1023u));
    const PagesView &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tb = ROWS / p.G;  // tokens of a block
    let_next_start();
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            mbar_init(&sh.q_full[i], 4);
            mbar_init(&sh.k_full[i], 4 + a.owed);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.v_full[i], 4);
            mbar_init(&sh.v_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.o_full[i], 1);
        }
        mbar_init(&sh.drained, 1);
        fence_mbar_init();
    }
    const long long own = own_places<THREADS>(a);
    // places before each row
    long long base = 0;
    for (int i0 = 0; i0 < a.r.n_rows; i0 += THREADS) {
        const int i = i0 + tid;
        long long w = 0;
        if (i < a.r.n_rows) {
            const PageRow r = attn_row(a, i);
            sh.row[i] = r.row;
            sh.keys[i] = r.len - r.from;
            if (r.len > 0 && takes(a, r)) w = p.Hkv * blocks_before(base_of(a, r), tb * a.step, (r.n + tb - 1) / tb);
        }
        long long s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(FULL, s, o);
            if (lane >= o) s += t;
        }
        if (lane == 31) sh.part[warp] = s;
        __syncthreads();
        long long before = base;
        for (int k = 0; k < THREADS / 32; k++) {
            const long long t = sh.part[k];
            if (k < warp) before += t;
            base += t;
        }
        if (i < a.r.n_rows) sh.first[i] = before + s - w;
        __syncthreads();
    }
    const long long N = base;
    if (tid == 0) sh.first[a.r.n_rows] = N;
    // rows that hold nothing: zeros
    for (int i = blockIdx.x; i < a.r.n_rows && a.mode != PAGES_COMMON; i += gridDim.x) {
        if (sh.keys[i] > 0) continue;
        const PageRow r = page_row(p, a.r, i);
        if (!takes(a, r)) continue;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + static_cast<long long>(r.q0) * p.Hq * D);
        for (long long k = tid; k < static_cast<long long>(r.n) * p.Hq * (D / 8); k += THREADS) o[k] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (long long k = tid; k < static_cast<long long>(r.n) * p.Hq; k += THREADS) a.lse[static_cast<long long>(r.q0) * p.Hq + k] = -INFINITY;
        if (a.mode == PAGES_OWN && a.plan[2 * i] > 0)
            for (long long k = tid; k < static_cast<long long>(r.n) * p.Hq; k += THREADS)
                reinterpret_cast<float2 *>(part_sums<D>(a))[static_cast<long long>(r.q0) * p.Hq + k] = make_float2(INFINITY, 0.f);
    }
    constexpr int worth = MODE == PAGES_COMMON ? MIN_SHARE_COMMON : MIN_SHARE;
    const int room = sms_left<THREADS>(a, own, sh.part);
    int ctas = static_cast<int>(N / worth < room ? N / worth : room);
    if (ctas < 1) ctas = 1;
    int4 *join = reinterpret_cast<int4 *>(a.joins) + blockIdx.x;
    if (N == 0 || static_cast<int>(blockIdx.x) >= ctas) {
        if (tid == 0) *join = make_int4(0, 0, 0, 0);
        if (a.mode == PAGES_COMMON) await_previous();
        return;
    }
    const long long c0 = share(N, ctas, blockIdx.x), c1 = share(N, ctas, blockIdx.x + 1);
    if (tid == 0) {  // the unit that begins here and goes on in other CTAs, if any
        const Unit u = find_unit<D>(sh, a, tb, c1 - 1);
        const bool on = u.start >= c0 && u.end > c1;
        const int t0 = u.b * tb, n = u.r.n - t0 < tb ? u.r.n - t0 : tb;
        *join = on ? make_int4(u.r.q0 + t0, u.head | (u.r.from > 0) << 16, n * p.G, share_of(N, ctas, u.end - 1) - static_cast<int>(blockIdx.x) + 1)
                   : make_int4(0, 0, 0, 0);
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // After a wait that ran out a thread waits no more: every role goes through its (finite)
    // loops, in step with its warp, and the status says that the outputs are not valid.  What it
    // did not wait for may still run: tensor memory is freed behind the last product (`drained`).
    bool late = false;
    auto wait = [&](uint64_t *bar, unsigned parity) {
        if (!late && !mbar_spin(bar, parity, a.wait_ns)) {
            late = true;
            atomicOr(p.status, PST_TIMEOUT);
        }
    };
    // registers move from the warps that need few (of 512 x 128: 384 x 144 + 128 x 80 = 65536)
    if (warp < 12) asm volatile("setmaxnreg.inc.sync.aligned.u32 144;\n");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
    constexpr int REC = ROWS * (D + 2);  // a part: accumulators [D / 4][ROWS][4], maxima [ROWS], sums [ROWS]

    if (warp < 8) {
        // ---- softmax: a thread a query row --------------------------------------------------
        const int t = warp >> 2, row = tid;  // tile, row of the unit
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes of tensor memory
        const uint32_t s_at = tmem + lanes + t * KEYS, o_at = tmem + lanes + 2 * KEYS + t * D;
        unsigned runs = 0, it = 0;
        for (long long x = c0; x < c1;) {
            const Segment g = find_segment<D>(sh, a, tb, x, c1);
            const PageRow &r = g.u.r;
            x = g.u.end;
            if (t == 1 && !g.two) continue;
            const int tok = g.u.b * tb + row / p.G, gq = row % p.G;
            const bool real = row < tb * p.G && tok < r.n;
            const int pos = real ? first_sees(a, r) + tok * a.step : 0x7fffffff;  // no row: nothing to mask
            // the query, by a power of two below 2^14 and with sm_scale's sign, as binary16
            RowState row_s{0.f, -INFINITY, {0, 0}};
            if (g.t0 < g.t1) {
                const float f = p.bf16 ? put_queries<D, true>(a, r, g.u.head, g.u.b * tb, tb, sh.q[t]) : put_queries<D, false>(a, r, g.u.head, g.u.b * tb, tb, sh.q[t]);
                // (never 0: a hidden key's -inf stays one)
                row_s.f = fmaxf(f, 1e-37f);
                fence_proxy_async();
                mbar_arrive(&sh.q_full[t]);
            }
            const int least = __reduce_min_sync(FULL, pos);
            for (int k = g.t0; k < g.t1; k++, it++) {
                wait(&sh.s_full[t], it & 1);
                tc_fence_after();
                const int key0 = r.from + k * KEYS;
                const bool tail = key0 + KEYS - 1 > least;
                if (tail) {  // hidden keys' scores become -inf
#pragma unroll 1
                    for (int c = 0; c < KEYS; c += 32) {
                        uint32_t s[32];
                        tmem_ld32(s_at + c, s);
                        tmem_wait_ld(s);
#pragma unroll
                        for (int i = 0; i < 32; i++) s[i] = key0 + c + i > pos ? 0xff800000u : s[i];
                        tmem_st32(s_at + c, s);
                    }
                    tmem_wait_st();
                }
                if (k == g.t0) {  // m from all of the first tile (a row that sees nothing of it sees nothing later)
                    float z = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < KEYS; c += 32) {
                        uint32_t s[32];
                        tmem_ld32(s_at + c, s);
                        tmem_wait_ld(s);
                        z = fmaxf(z, top_of(s));
                    }
                    row_s.m = z == -INFINITY ? -INFINITY : z * row_s.f;
                }
                // 32 keys at a time, the next 32 on their way; their weights take the place of scores that were read.
                // A load's registers hold nothing before its wait: load and wait stand in one straight piece of code,
                // with the weights of the 32 keys before between them and neither a branch nor the loop's end (so the
                // last 32 keys' load is of columns that nobody uses; unrolled without it 9 % slower).
                uint32_t sa[32], sb[32];
                auto chunk = [&](uint32_t (&s)[32], uint32_t (&coming)[32], int c) {
                    // Weights are positive: one over MOST shows in their sum, so that the maximum is
                    // only sought where the sum passes that (or, no harm, many smaller weights do).
                    uint32_t w[16];
                    uint64_t sum[2];
                    tmem_ld32(s_at + 32 * (c + 1) % KEYS, coming);
                    row_s.weigh(s, w, sum);
                    tmem_wait_ld(coming);
                    const float2 x0 = both(add2(sum[0], sum[1]));
                    if (__any_sync(FULL, x0.x + x0.y > MOST)) {
                        const float top = top_of(s);
                        row_s.raise<D>(top == -INFINITY ? -INFINITY : top * row_s.f, k > g.t0, o_at, 16 * c, s_at);
                        row_s.weigh(s, w, sum);
                    }
                    row_s.l[0] = add2(row_s.l[0], sum[0]);
                    row_s.l[1] = add2(row_s.l[1], sum[1]);
                    tmem_st16(s_at + 16 * c, w);
                };
                tmem_ld32(s_at, sa);
                tmem_wait_ld(sa);
#pragma unroll 1
                for (int c = 0; c < KEYS / 32; c += 2) {
                    chunk(sa, sb, c);
                    chunk(sb, sa, c + 1);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&sh.p_full[t]);
            }
            if (g.t0 < g.t1) {
                wait(&sh.o_full[t], runs & 1);
                runs++;
                tc_fence_after();
            }
            const long long o = (static_cast<long long>(r.q0) + tok) * p.Hq + g.u.head * p.G + gq;
            const bool whole = g.begins && g.ends;
            float *rec = a.records + (2LL * blockIdx.x + g.begins) * REC;
            float l = row_s.sum(), m = row_s.m, keep = 1.f, take = 0.f;
            if (a.mode == PAGES_COMMON && whole) {
                await_previous();
                if (real) {
                    const float2 own = reinterpret_cast<const float2 *>(part_sums<D>(a))[o];
                    if (own.x == INFINITY) l = 0.f;
                    else join_sums(m, l, own, keep, take);
                }
            }
            const float by = l == 0.f ? 0.f : a.out_scale / l;
#pragma unroll 1
            for (int c = 0; c < D / 32; c++) {
                uint32_t s[32];
                if (g.t0 < g.t1) {
                    tmem_ld32(o_at + 32 * c, s);
                    tmem_wait_ld(s);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i++) s[i] = 0;
                }
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        *reinterpret_cast<uint4 *>(rec + ((8 * c + i) * ROWS + row) * 4) = make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
                } else if (real && a.mode == PAGES_OWN && r.from > 0) {
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        *reinterpret_cast<uint4 *>(a.part + o * D + 32 * c + 4 * i) = make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
                } else if (real) {
                    if (a.mode == PAGES_COMMON) {
#pragma unroll
                        for (int i = 0; i < 32; i++) s[i] = __float_as_uint(__uint_as_float(s[i]) * keep + a.part[o * D + 32 * c + i] * take);
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        w[i] = l == 0.f ? 0u
                                        : pack2(to16(__uint_as_float(s[2 * i]) * by, p.bf16), to16(__uint_as_float(s[2 * i + 1]) * by, p.bf16));
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        *reinterpret_cast<uint4 *>(a.out + o * D + 32 * c + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                }
            }
            if (!whole) {
                rec[ROWS * D + row] = m;
                rec[ROWS * (D + 1) + row] = l;
            } else if (real && a.mode == PAGES_OWN && r.from > 0) {
                reinterpret_cast<float2 *>(part_sums<D>(a))[o] = make_float2(m, l);
            } else if (real && a.lse) {
                a.lse[o] = l == 0.f ? -INFINITY : (m - LIFT + log2f(l)) * LN2;
            }
            tc_fence_before();
        }
    } else if (warp < 12) {
        // ---- codes to operands: a thread a key, and a thread 8 tokens of 16 value channels --------
        const int dt = tid - 256, kg = dt & 15, c16 = dt >> 4;
        const bool has_v = c16 < D / 16;
        const int shift = 31 - __clz(p.P), in_page = p.P - 1, b = p.blk, b_shift = 31 - __clz(b), in_block = b - 1;  // powers of two
        // this thread's rows in the operands, the row's swizzle in place: piece c is at that address ^ 16 c
        const uint32_t k_row = smem_u32(sh.k[0]) + swizzled(dt, 0);
        uint32_t v_row[4];
#pragma unroll
        for (int c = 0; c < 4; c++) v_row[c] = smem_u32(sh.v[0]) + (kg >> 3) * (D * 128) + swizzled(c16 * 16 + c, kg & 7);
        auto store16 = [](uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
        };
        struct Packed {
            uint4 k[D / 32], v[4];
            uint2 ks, vs;
        };
        unsigned it = 0;
        for (long long x = c0; x < c1;) {
            const Segment g = find_segment<D>(sh, a, tb, x, c1);
            const PageRow &r = g.u.r;
            x = g.u.end;
            auto number = [&](int at) -> int {  // page of position `at`, or none
                if (at >= r.len || r.row < 0) return -1;
                return p.table[static_cast<long long>(r.row) * p.M + (at >> shift)];
            };
            auto checked = [&](int id, int at) -> int {
                if (at >= r.len || r.row < 0 || (id >= 0 && id < p.n_pages)) return id;
                atomicOr(p.status, PST_TABLE);
                return -1;
            };
            auto load = [&](Packed &w, int tile, int idk, int idv) {
                const int key = r.from + tile * KEYS + dt, tok = r.from + tile * KEYS + 8 * kg;
                idk = checked(idk, key);
                idv = checked(idv, tok);
#pragma unroll
                for (int i = 0; i < D / 32; i++) w.k[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; i++) w.v[i] = make_uint4(0, 0, 0, 0);
                w.ks = w.vs = make_uint2(0, 0);
                if (idk >= 0) {
                    const int u = key & in_page, ub = u & in_block;
                    const uint8_t *blk = page_ptr(p, idk, g.u.head) + (u >> b_shift) * B::size(b);
#pragma unroll
                    for (int i = 0; i < D / 32; i++) w.k[i] = *reinterpret_cast<const uint4 *>(blk + ub * (D / 2) + 16 * i);
                    if (D == 128) w.ks = *reinterpret_cast<const uint2 *>(blk + B::ks(b) + ub * (D / 16));
                    else w.ks.x = *reinterpret_cast<const uint32_t *>(blk + B::ks(b) + ub * (D / 16));
                }
                if (has_v && idv >= 0) {
                    const int u = tok & in_page, ub = u & in_block;
                    const uint8_t *blk = page_ptr(p, idv, g.u.head) + (u >> b_shift) * B::size(b);
#pragma unroll
                    for (int i = 0; i < 4; i++) w.v[i] = *reinterpret_cast<const uint4 *>(blk + B::vc(b) + B::vcode(ub, c16) + 16 * i);
                    w.vs = *reinterpret_cast<const uint2 *>(blk + B::vs(b) + B::vscale(ub, c16));
                }
            };
            // codes one tile ahead, page numbers two
            Packed cur, nxt;
            if (g.t0 < g.t1) load(cur, g.t0, number(r.from + g.t0 * KEYS + dt), number(r.from + g.t0 * KEYS + 8 * kg));
            int idk = number(r.from + (g.t0 + 1) * KEYS + dt), idv = number(r.from + (g.t0 + 1) * KEYS + 8 * kg);
            for (int k = g.t0; k < g.t1; k++, it++) {
                if (k + 1 < g.t1) {
                    load(nxt, k + 1, idk, idv);
                    idk = number(r.from + (k + 2) * KEYS + dt);
                    idv = number(r.from + (k + 2) * KEYS + 8 * kg);
                }
                const int st = it & 1;
                const unsigned free = ((it >> 1) + 1) & 1;
                if (it >= 2) wait(&sh.k_empty[st], free);
#pragma unroll
                for (int i = 0; i < D / 16; i++) {  // a scale block: two 16-byte pieces
                    const uint32_t sb = (i < 4 ? cur.ks.x : cur.ks.y) >> (8 * (i & 3)) & 0xffu;
                    const uint32_t s1 = e4m3x2_to_half2(static_cast<uint16_t>(sb)), s2 = __byte_perm(s1, s1, 0x1010);
                    const uint4 &q = cur.k[i >> 1];
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        uint32_t h[4];
                        e2m1x8_to_half(i & 1 ? (e ? q.w : q.z) : (e ? q.y : q.x), h);
                        const int c = 2 * i + e;
                        store16(((k_row + st * (KEYS * D * 2)) ^ ((c & 7) << 4)) + (c >> 3) * (KEYS * 128), hmul2(h[0], s2), hmul2(h[1], s2),
                                hmul2(h[2], s2), hmul2(h[3], s2));
                    }
                }
                fence_proxy_async();
                mbar_arrive(&sh.k_full[st]);
                if (it >= 2) wait(&sh.v_empty[st], free);
                if (has_v) {
                    uint32_t sv[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const uint32_t two = (e < 2 ? cur.vs.x : cur.vs.y) >> (16 * (e & 1)) & 0xffffu;
                        const int tok = r.from + k * KEYS + 8 * kg + 2 * e;  // tokens that are not there: 0, whatever their bytes say
                        sv[e] = e4m3x2_to_half2(static_cast<uint16_t>(two)) & ((tok < r.len ? 0x0000ffffu : 0u) | (tok + 1 < r.len ? 0xffff0000u : 0u));
                    }
#pragma unroll
                    for (int wd = 0; wd < 4; wd++) {
                        uint32_t h[4][4];  // [pair][channel]
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const uint4 &q = cur.v[e];
                            e2m1x8_to_half(wd == 0 ? q.x : (wd == 1 ? q.y : (wd == 2 ? q.z : q.w)), h[e]);
                        }
#pragma unroll
                        for (int c = 0; c < 4; c++)
                            // rows 4 wd + c: the swizzle goes by the row's last 3 bits, of which wd turns the highest
                            store16(((v_row[c] + st * (KEYS * D * 2)) ^ ((wd & 1) << 6)) + wd * 512, hmul2(h[0][c], sv[0]), hmul2(h[1][c], sv[1]),
                                    hmul2(h[2][c], sv[2]), hmul2(h[3][c], sv[3]));
                    }
                }
                fence_proxy_async();
                mbar_arrive(&sh.v_full[st]);
                cur = nxt;
            }
        }
    } else if (warp == 12) {
        // ---- products -----------------------------------------------------------------------------
        // The warp goes through them together and one lane issues them: a branch of one lane's own keeps the descriptors out
        // of the uniform registers that the instruction takes (2048 tokens over 16384: 404 us, so 433).
        unsigned runs[2] = {0, 0}, done[2] = {0, 0}, it = 0;  // of each tile: units, keys' tiles
        uint32_t q_at[2], s_at[2], o_at[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
            q_at[t] = operand(smem_u32(sh.q[t]));
            s_at[t] = tmem + t * KEYS;
            o_at[t] = tmem + 2 * KEYS + t * D;
        }
        const uint32_t k_at = operand(smem_u32(sh.k[0])), v_at = operand(smem_u32(sh.v[0]));
        constexpr uint32_t STAGE = KEYS * D * 2 / 16;
        auto commit = [](uint64_t *bar) {
            if (elect_one()) tc_commit(bar);
            __syncwarp();
        };
        auto scores = [&](int t, int st) {
            const uint32_t kb = k_at + st * STAGE;
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < D / 16; i++)
                    mma_smem(s_at[t], q_at[t] + (i >> 2) * (TILE * 8) + (i & 3) * 2, kb + (i >> 2) * (KEYS * 8) + (i & 3) * 2, product(KEYS), i > 0);
                tc_commit(&sh.s_full[t]);
            }
            __syncwarp();
        };
        for (long long x = c0; x < c1;) {
            const Segment g = find_segment<D>(sh, a, tb, x, c1);
            x = g.u.end;
            if (g.t0 >= g.t1) continue;
            wait(&sh.k_full[it & 1], it >> 1 & 1);
#pragma unroll
            for (int t = 0; t < 2; t++) {
                if (t == 1 && !g.two) break;
                wait(&sh.q_full[t], runs[t]++ & 1);
                tc_fence_after();
                scores(t, it & 1);
            }
            commit(&sh.k_empty[it & 1]);
            for (int k = g.t0; k < g.t1; k++, it++) {
                const int st = it & 1, next = (it + 1) & 1;
                const uint32_t vb = v_at + st * STAGE;
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    if (t == 1 && !g.two) break;
                    const bool last = t == 1 || !g.two;
                    wait(&sh.p_full[t], done[t]++ & 1);
                    if (t == 0) wait(&sh.v_full[st], it >> 1 & 1);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < KEYS / 16; i++)
                            mma_tmem(o_at[t], s_at[t] + 8 * i, vb + (i >> 2) * (D * 8) + (i & 3) * 2, product(D), k > g.t0 || i > 0);
                        if (last) tc_commit(&sh.v_empty[st]);
                    }
                    __syncwarp();
                    if (k + 1 < g.t1) {
                        if (t == 0) wait(&sh.k_full[next], (it + 1) >> 1 & 1);
                        if (t == 0) tc_fence_after();
                        scores(t, next);
                        if (last) commit(&sh.k_empty[next]);
                    } else {
                        commit(&sh.o_full[t]);
                    }
                }
            }
        }
        // (where no wait ran out, the softmax has waited for the same products)
        commit(&sh.drained);
        if (!mbar_spin(&sh.drained, 0, a.wait_ns)) atomicOr(p.status, PST_TIMEOUT);
    }
    if (a.mode == PAGES_COMMON) await_previous();
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
    }

}

// The units that crossed a share's border, where there may be many of a few parts each: CTA (c, y) adds up the parts of the
// unit that began in share c and went on, 8 channels of its 256 rows, in CTA order.
// (joins: first token, KV head and whether there are pages in common, query rows, parts)
template <int D, int MODE>
__global__ void __launch_bounds__(ROWS) join_many(const InMode<MODE> a) {
    let_next_start();
    await_previous();
    const int4 what = reinterpret_cast<const int4 *>(a.joins)[blockIdx.x];
    const PagesView &p = a.p;
    const int n = what.w, row = threadIdx.x, c = blockIdx.y, tok = row / p.G;
    if (n == 0 || row >= what.z) return;
    const long long o = (static_cast<long long>(what.x) + tok) * p.Hq + (what.y & 0xffff) * p.G + row - tok * p.G;
    constexpr int REC = ROWS * (D + 2);
    float2 own = make_float2(-INFINITY, 0.f);
    if (a.mode == PAGES_COMMON) own = reinterpret_cast<const float2 *>(part_sums<D>(a))[o];
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    auto add = [&](float mk, float lk, float4 xk, float4 yk) {
        float keep, take;
        join_sums(m, l, make_float2(mk, lk), keep, take);
        x = make_float4(x.x * keep + xk.x * take, x.y * keep + xk.y * take, x.z * keep + xk.z * take, x.w * keep + xk.w * take);
        y = make_float4(y.x * keep + yk.x * take, y.y * keep + yk.y * take, y.z * keep + yk.z * take, y.w * keep + yk.w * take);
    };
#pragma unroll 4
    for (int k = 0; k < n; k++) {
        const float *rec = a.records + (2LL * (blockIdx.x + k) + (k == 0)) * REC;
        const float4 *v = reinterpret_cast<const float4 *>(rec + (2 * c * ROWS + row) * 4);
        add(rec[ROWS * D + row], rec[ROWS * (D + 1) + row], v[0], v[ROWS]);
    }
    float4 *part = reinterpret_cast<float4 *>(a.part + o * D + 8 * c);
    if (a.mode == PAGES_OWN && what.y >> 16) {
        part[0] = x;
        part[1] = y;
        if (c == 0) reinterpret_cast<float2 *>(part_sums<D>(a))[o] = make_float2(m, l);
        return;
    }
    if (own.x == INFINITY) l = 0.f;  // the row holds nothing
    else if (a.mode == PAGES_COMMON) add(own.x, own.y, part[0], part[1]);
    const float by = l == 0.f ? 0.f : a.out_scale / l;
    *reinterpret_cast<uint4 *>(a.out + o * D + 8 * c) =
        make_uint4(pack2(to16(x.x * by, p.bf16), to16(x.y * by, p.bf16)), pack2(to16(x.z * by, p.bf16), to16(x.w * by, p.bf16)),
                   pack2(to16(y.x * by, p.bf16), to16(y.y * by, p.bf16)), pack2(to16(y.z * by, p.bf16), to16(y.w * by, p.bf16)));
    if (c == 0 && a.lse) a.lse[o] = l == 0.f ? -INFINITY : (m - LIFT + log2f(l)) * LN2;
}

// The same where there are few units of many parts (64 rows behind 8192 tokens: 8 of 11, 9 us; 12 with the kernel above): a CTA
// adds up 4 channels of 128 rows of a unit, a quarter of the parts in each quarter of its threads, so that all are on their
// way at once, always in the same order.
constexpr int JOIN_WAYS = 4, JOIN_THREADS = TILE * JOIN_WAYS, JOIN_FEW = 16;
template <int D, int MODE>
__global__ void __launch_bounds__(JOIN_THREADS) join_few(const InMode<MODE> a, int ctas) {
    __shared__ int4 todo[PAGES_MAX_CTAS];
    __shared__ int owner[PAGES_MAX_CTAS], n_todo;
    __shared__ float4 acc_s[JOIN_WAYS - 1][TILE];
    __shared__ float2 ml_s[JOIN_WAYS - 1][TILE];
    let_next_start();
    await_previous();
    const PagesView &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, way = tid / TILE;
    if (tid < 32) {
        int n = 0;
        int4 what[PAGES_MAX_CTAS / 32];
#pragma unroll
        for (int k = 0; k < PAGES_MAX_CTAS / 32; k++)
            what[k] = 32 * k + lane < ctas ? reinterpret_cast<const int4 *>(a.joins)[32 * k + lane] : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < PAGES_MAX_CTAS / 32; k++) {
            const unsigned some = __ballot_sync(FULL, what[k].w > 0);
            if (what[k].w > 0) {
                const int at = n + __popc(some & ((1u << lane) - 1u));
                todo[at] = what[k];
                owner[at] = 32 * k + lane;
            }
            n += __popc(some);
        }
        if (lane == 0) n_todo = n;
    }
    __syncthreads();
    constexpr int REC = ROWS * (D + 2), SLICES = D / 4 * 2, DEEP = 5;
    const int items = n_todo * SLICES;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int which = item / SLICES, c = item % (D / 4), row0 = item % SLICES / (D / 4) * TILE, row = row0 + tid % TILE;
        const int4 what = todo[which];
        if (row0 >= what.z) continue;  // no rows in the second tile
        const bool real = row < what.z, first = real && way == 0;
        const int tok = row / p.G;
        const long long o = (static_cast<long long>(what.x) + tok) * p.Hq + (what.y & 0xffff) * p.G + row - tok * p.G;
        float4 *part = reinterpret_cast<float4 *>(a.part + o * D + 4 * c);
        float2 own = make_float2(-INFINITY, 0.f);
        float4 own_acc = make_float4(0.f, 0.f, 0.f, 0.f), acc = own_acc;
        if (a.mode == PAGES_COMMON && first) {
            own = reinterpret_cast<const float2 *>(part_sums<D>(a))[o];
            own_acc = *part;
        }
        float m = -INFINITY, l = 0.f;
        auto add = [&](float mk, float lk, float4 x) {
            float keep, take;
            join_sums(m, l, make_float2(mk, lk), keep, take);
            acc = make_float4(acc.x * keep + x.x * take, acc.y * keep + x.y * take, acc.z * keep + x.z * take, acc.w * keep + x.w * take);
        };
        for (int k0 = way; k0 < what.w; k0 += DEEP * JOIN_WAYS) {
            float mk[DEEP], lk[DEEP];
            float4 x[DEEP];
#pragma unroll
            for (int e = 0; e < DEEP; e++) {
                const int k = k0 + e * JOIN_WAYS;
                mk[e] = -INFINITY;
                lk[e] = 0.f;
                x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k >= what.w || !real) continue;
                const float *rec = a.records + (2LL * (owner[which] + k) + (k == 0)) * REC;
                mk[e] = rec[ROWS * D + row];
                lk[e] = rec[ROWS * (D + 1) + row];
                x[e] = *reinterpret_cast<const float4 *>(rec + (c * ROWS + row) * 4);
            }
#pragma unroll
            for (int e = 0; e < DEEP; e++) add(mk[e], lk[e], x[e]);
        }
        if (way > 0) {
            acc_s[way - 1][tid % TILE] = acc;
            ml_s[way - 1][tid % TILE] = make_float2(m, l);
        }
        __syncthreads();
        if (first) {
#pragma unroll
            for (int w = 0; w < JOIN_WAYS - 1; w++) add(ml_s[w][tid].x, ml_s[w][tid].y, acc_s[w][tid]);
            if (a.mode == PAGES_OWN && what.y >> 16) {
                *part = acc;
                if (c == 0) reinterpret_cast<float2 *>(part_sums<D>(a))[o] = make_float2(m, l);
            } else {
                if (own.x == INFINITY) l = 0.f;
                else if (a.mode == PAGES_COMMON) add(own.x, own.y, own_acc);
                const float by = l == 0.f ? 0.f : a.out_scale / l;
                *reinterpret_cast<uint2 *>(a.out + o * D + 4 * c) =
                    make_uint2(pack2(to16(acc.x * by, p.bf16), to16(acc.y * by, p.bf16)), pack2(to16(acc.z * by, p.bf16), to16(acc.w * by, p.bf16)));
                if (c == 0 && a.lse) a.lse[o] = l == 0.f ? -INFINITY : (m - LIFT + log2f(l)) * LN2;
            }
        }
        __syncthreads();
    }
}

template <int D, int MODE>
int launch_as(const PagesAttnArgs &a, int grid, cudaStream_t st) {
    const int smem = static_cast<int>(sizeof(Shared<D>)) + 1024;  // room to put it on a 1024-byte boundary
    if (const int e = allow_shared<attn_prompt<D, MODE>>(smem)) return e;
    if (MODE == PAGES_COMMON && a.after_few) {
        if (const int e = launch_overlapping(attn_prompt<D, MODE>, dim3(grid), THREADS, smem, st, InMode<MODE>{a})) return e;
    } else {
        attn_prompt<D, MODE><<<grid, THREADS, smem, st>>>(InMode<MODE>{a});
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return static_cast<int>(e);
    }
    // (as many units at most: whole blocks of query rows, and one begun in each row)
    const long long units = (static_cast<long long>(a.r.n_tok) * a.p.G / ROWS + a.r.n_rows) * a.p.Hkv;
    if (units <= JOIN_FEW) return launch_overlapping(join_few<D, MODE>, dim3(3 * grid), JOIN_THREADS, 0, st, InMode<MODE>{a}, grid);
    return launch_overlapping(join_many<D, MODE>, dim3(grid, D / 8), ROWS, 0, st, InMode<MODE>{a});
}
template <int MODE>
int launch_many(const PagesAttnArgs &a, int grid, void *stream) {
    auto st = static_cast<cudaStream_t>(stream);
    return a.p.d == 128 ? launch_as<128, MODE>(a, grid, st) : launch_as<64, MODE>(a, grid, st);
}

}  // namespace
}  // namespace dq
