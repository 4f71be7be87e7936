// Paged cache: the attention weights of held tokens from many queries, on the 5th-generation
// tensor cores.
//
//   score_j (+)= sum_c exp2(f s_jc - less_c),  s = K Q^T,  f = sm_scale 2^k_exp log2(e),  less_c = lse_c log2(e)
// over the columns c, the query rows (token, query head of the group) that see key j.  2 D
// products and one exponential for each (query, key) pair: bound by the tensor cores and
// the exponentials alike.
//
// 2048 new tokens over 16384 (32 / 8 heads, head_dim 128) take 208 us, 1.24 PFLOP/s; the last 64 queries of
// four prompts of 9 to 16 k tokens 48 us.
//
// Keys are the rows of the product, so that a key's sum is one thread's: nothing is summed
// over lanes.  Their operand lies in tensor memory (a thread unpacks a key's codes and
// stores its lane), the queries' in shared memory as they come from memory: e2m1 times e4m3
// has 6 significant bits, so that keys are exact in the queries' own type, bf16 or binary16,
// and no query needs a conversion.
//
// Work.  A unit is 256 keys (two tiles of 128) of one row and KV head with all the row's
// query rows that see one of them, 128 / G tokens a block.  Units stand on a line, each as
// long as its tokens, and the line is cut into equal shares, one for each CTA (one per SM).
// Parts of a unit in several CTAs meet in the workspace, where the last CTA to arrive adds
// them up in CTA order.
//
// Roles of the 16 warps.  Warps 0-3 and 4-7: weights of tile 0 and 1, a thread a key.  Warps
// 8-11: a unit's keys into tensor memory, the next one's codes on their way.  Warps 12, 13 and 15: queries
// into shared memory, a block in turn, four deep.  Warp 14: one thread issues all products, tile by tile
// in turn, so that one tile's exponentials run beside the other's products.
// Tensor memory: two products (128 columns each), then two units' keys (2 tiles of D / 2 columns each).
#include <type_traits>

#include <cuda_runtime.h>

#include "pages_tc.cuh"
#include "pages_weigh.cuh"

namespace dq {
namespace {

constexpr int TILE = 128, KEYS = 2 * TILE;  // keys of a tile, of a unit
constexpr int COLS = 128;                   // query rows of a block, at most
constexpr int ST = 4;                       // blocks of queries in shared memory
constexpr int RING = 2, KB = 2;             // products and units' keys in tensor memory (three and one: 3 % slower at 2048 tokens)
constexpr int THREADS = 512;
constexpr int UNIT_COST = 32;               // tokens that a unit's beginning and end are worth
constexpr int MIN_SHARE = 64;               // tokens that make a CTA worth its parts

// A unit that this CTA shares with others: the one that its share begins within, and the one that goes on behind it.
struct Joint {
    int first, others;  // the CTA that it begins in, and how many more there are; others < 0: none
    int row, head, key0, len, old;
};
template <int D>
struct Shared {
    __align__(1024) uint8_t q[ST][COLS * D * 2];
    __align__(16) float less[ST][COLS];
    __align__(16) int pos[ST][COLS];
    long long at[COLS];  // where a block's row of queries is, behind its first token's
    long long first[DQ_PAGES_MAX_ROWS + 1];
    int row[DQ_PAGES_MAX_ROWS], keys[DQ_PAGES_MAX_ROWS];
    long long part[THREADS / 32];
    uint64_t q_full[ST], q_empty[ST], k_full[KB], k_empty[KB], s_full[RING], s_empty[RING], drained;
    uint32_t tmem;
    int last[2];
    Joint joint[2];
};

// Unit j of a row and KV head: places UNIT_COST + n - skipped(j); the tokens before that one see none of its keys.
__device__ __forceinline__ int skipped(const PageRow &r, int j) {
    const int s = j * KEYS - (r.len - r.n);
    return s > 0 ? s : 0;
}
__device__ __forceinline__ long long units_before(const PageRow &r, int j) {  // places of units 0 .. j - 1 of a head
    const long long old = r.len - r.n, j0 = old < 0 ? 0 : old / KEYS + 1, m = j > j0 ? j - j0 : 0;
    return j * static_cast<long long>(UNIT_COST + r.n) - (m * (j - 1 + j0) / 2 * KEYS - m * old);
}
__device__ __forceinline__ int units_of(const PageRow &r) { return (r.len + KEYS - 1) / KEYS; }

__device__ __forceinline__ long long over(long long n, long long m) {  // n / m, both positive: 32 bits where they are enough
    return (n | m) >> 32 ? n / m : static_cast<unsigned>(n) / static_cast<unsigned>(m);
}
__device__ __forceinline__ long long share(long long n, int m, int k) {
    const long long q = over(n, m), rest = n - q * m;
    return k * q + (k < rest ? k : rest);
}
__device__ __forceinline__ int share_of(long long n, int m, long long x) {
    const long long q = over(n, m), rest = n - q * m, ahead = rest * (q + 1);
    return static_cast<int>(x < ahead ? over(x, q + 1) : rest + over(x - ahead, q));
}

// A CTA's way along its share [c0, c1) of the line: unit by unit, with the blocks [b0, b1) of query rows that are its.
// The first unit is searched for, the next ones follow from it.
struct Walk {
    PageRow r;
    int i, head, j, units, b0, b1;
    uint32_t tb, inv;      // tokens of a block; x / tb is the high word of x inv (exact for x < 2^32 / tb: 2^25 at least)
    long long start, end;  // places of the unit
    __device__ explicit Walk(const PagesWeighArgs &a) : tb(COLS / a.p.G) { inv = 0xffffffffu / tb + 1u; }
    __device__ int blocks(int tokens) const { return __umulhi(tokens, inv); }
    bool begins, ends;
    template <int D>
    __device__ void find(const Shared<D> &sh, const PagesWeighArgs &a, long long x, long long c0, long long c1) {
        r = weigh_row_at(a, sh.row, sh.keys, sh.first, x, i);
        units = units_of(r);
        const long long all = units_before(r, units), in = x - sh.first[i];
        head = static_cast<int>(over(in, all));
        const long long at = in - head * all;
        int lo = 0, hi = units - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (units_before(r, mid) <= at) lo = mid;
            else hi = mid - 1;
        }
        j = lo;
        start = x - at + units_before(r, lo);
        here(a, c0, c1);
    }
    __device__ void here(const PagesWeighArgs &a, long long c0, long long c1) {
        const int skip = skipped(r, j);
        end = start + UNIT_COST + r.n - skip;
        begins = start >= c0;
        ends = end <= c1;
        auto block_at = [&](long long y) {
            const int t = static_cast<int>(y - start) - UNIT_COST;
            return blocks(skip + (t > 0 ? t : 0) + tb - 1);
        };
        b0 = begins ? blocks(skip) : block_at(c0);
        b1 = ends ? blocks(r.n + tb - 1) : block_at(c1);
    }
    template <int D>
    __device__ void next(const Shared<D> &sh, const PagesWeighArgs &a, long long c0, long long c1) {
        start = end;
        if (start >= c1) return;
        if (++j == units) {
            j = 0;
            if (++head == a.p.Hkv) {
                r = weigh_row_at(a, sh.row, sh.keys, sh.first, start, i);
                head = 0;
                units = units_of(r);
            }
        }
        here(a, c0, c1);
    }
};
// Two binary16 numbers of at most 8 significant bits -> bf16.
__device__ __forceinline__ uint32_t half2_to_bf16(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(f.y), "f"(f.x));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// 16 bytes from memory to shared memory, zeros where there is nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Arrive on `bar` when this thread's copies so far are there.
__device__ __forceinline__ void arrive_copied(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS, 1) weigh_many(const PagesWeighArgs a) {
    extern __shared__ uint8_t raw[];
    using S = Shared<D>;
    using B = PageBlock<D>;
    S &sh = *reinterpret_cast<S *>(raw + (-smem_u32(raw) & 1023u));
    const PagesView &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tb = COLS / p.G;
    if (tid == 0) {
        for (int i = 0; i < ST; i++) {
            mbar_init(&sh.q_full[i], 1 + 32);  // a warp's stores, 32 threads' copies
            mbar_init(&sh.q_empty[i], 9);
        }
        for (int i = 0; i < KB; i++) {
            mbar_init(&sh.k_full[i], 4 + a.owed);
            mbar_init(&sh.k_empty[i], 1);
        }
        for (int i = 0; i < RING; i++) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], 4);
        }
        mbar_init(&sh.drained, 1);
        fence_mbar_init();
    }
    if (tid < COLS) sh.at[tid] = tid / p.G * a.qt + tid % p.G * a.qh;
    const long long N = weigh_rows<THREADS>(a, sh.row, sh.keys, sh.first, sh.part, [&](const PageRow &r) {
        return units_before(r, units_of(r)) * p.Hkv;
    });
    int ctas = static_cast<int>(N / MIN_SHARE < gridDim.x ? N / MIN_SHARE : gridDim.x);
    if (ctas < 1) ctas = 1;
    if (N == 0 || static_cast<int>(blockIdx.x) >= ctas) return;
    const long long c0 = share(N, ctas, blockIdx.x), c1 = share(N, ctas, blockIdx.x + 1);
    if (warp == 14) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem, k_tmem = tmem + RING * COLS;
    // After a wait that ran out a thread waits no more: every role goes through its (finite) loops, and the
    // status says that the scores are not valid.  Tensor memory is freed behind the last product (`drained`).
    bool late = false;
    Walk g(a);
    auto wait = [&](uint64_t *bar, unsigned parity) {
        if (!late && !mbar_spin(bar, parity, a.wait_ns)) {
            late = true;
            atomicOr(p.status, PST_TIMEOUT);
        }
    };

    if (warp < 8) {
        // ---- weights: a thread a key ----------------------------------------------------------
        const int t = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const float f = a.scale_log2;
        const uint64_t ff = two(f, f);
        unsigned it = 0;
        for (g.find(sh, a, c0, c0, c1); g.start < c1; g.next(sh, a, c0, c1)) {
            const int key = g.j * KEYS + tid, old = g.r.len - g.r.n, last_key = g.j * KEYS + t * TILE + TILE - 1;
            float *score = scores_of(a, g.r.row, g.head) + key;
            const bool whole = g.begins && g.ends;
            const float was = whole && key < g.r.len && key < old ? *score : 0.f;
            float sum = 0.f;
            for (int b = g.b0; b < g.b1; b++, it++) {
                const int st = it % ST;
                wait(&sh.q_full[st], it / ST & 1);  // (what the queries lose)
                const bool tail = last_key > old + b * tb;  // some query of the block does not see some key of the tile
                uint64_t acc[2] = {0, 0};
                const unsigned n = 2 * it + t, buf = n % RING;
                const uint32_t s_at = tmem + lanes + buf * COLS;
                wait(&sh.s_full[buf], n / RING & 1);
                tc_fence_after();
                uint32_t sa[32], sb[32];
                // 32 columns at a time, the next 32 on their way: a load and its wait stand in one straight piece of code, with
                // the weights of the columns before between them
                auto chunk = [&](auto hide, uint32_t (&s)[32], uint32_t (&coming)[32], int c) {
                    if (c + 1 < COLS / 32) tmem_ld32(s_at + 32 * (c + 1), coming);
                    const float4 *less = reinterpret_cast<const float4 *>(sh.less[st] + 32 * c);
                    const int4 *pos = reinterpret_cast<const int4 *>(sh.pos[st] + 32 * c);
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const float4 l = less[i];
                        float2 u = both(fma2(two(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), ff, two(l.x, l.y)));
                        float2 v = both(fma2(two(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), ff, two(l.z, l.w)));
                        if (decltype(hide)::value) {
                            const int4 at = pos[i];
                            u.x = key > at.x ? -INFINITY : u.x;
                            u.y = key > at.y ? -INFINITY : u.y;
                            v.x = key > at.z ? -INFINITY : v.x;
                            v.y = key > at.w ? -INFINITY : v.y;
                        }
                        acc[0] = add2(acc[0], two(ex2(u.x), ex2(u.y)));
                        acc[1] = add2(acc[1], two(ex2(v.x), ex2(v.y)));
                    }
                    if (c + 1 < COLS / 32) tmem_wait_ld(coming);
                    if (c == COLS / 32 - 2) {  // all is read
                        tc_fence_before();
                        mbar_arrive(&sh.s_empty[buf]);
                    }
                };
                auto all = [&](auto hide) {
                    chunk(hide, sa, sb, 0);
                    chunk(hide, sb, sa, 1);
                    chunk(hide, sa, sb, 2);
                    chunk(hide, sb, sa, 3);
                };
                tmem_ld32(s_at, sa);
                tmem_wait_ld(sa);
                if (tail) all(std::true_type{});
                else all(std::false_type{});
                mbar_arrive(&sh.q_empty[st]);
                const float2 u = both(acc[0]), v = both(acc[1]);
                sum += (u.x + u.y) + (v.x + v.y);
            }
            if (whole) {
                if (key < g.r.len) *score = was + sum;
            } else {
                a.records[(2LL * blockIdx.x + g.begins) * KEYS + tid] = sum;
            }
        }
    } else if (warp < 12) {
        // ---- keys: codes to operands in tensor memory, a thread a lane ------------------------------
        const int dt = tid - 256;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const int shift = 31 - __clz(p.P), in_page = p.P - 1, blk = p.blk, b_shift = 31 - __clz(blk), in_block = blk - 1;
        unsigned units = 0;
        struct Packed {
            uint4 w[2][D / 32];
            uint2 ks[2];
        };
        auto numbers = [&](const Walk &g, int (&id)[2]) {
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const int key = g.j * KEYS + t * TILE + dt;
                id[t] = key < g.r.len ? p.table[static_cast<long long>(g.r.row) * p.M + (key >> shift)] : -1;
            }
        };
        auto load = [&](const Walk &g, const int (&id)[2], Packed &k) {
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const int key = g.j * KEYS + t * TILE + dt;
#pragma unroll
                for (int i = 0; i < D / 32; i++) k.w[t][i] = make_uint4(0, 0, 0, 0);
                k.ks[t] = make_uint2(0, 0);
                if (key >= g.r.len) continue;
                if (id[t] < 0 || id[t] >= p.n_pages) {
                    atomicOr(p.status, PST_TABLE);
                    continue;
                }
                const int u = key & in_page, ub = u & in_block;
                const uint8_t *at = page_ptr(p, id[t], g.head) + (u >> b_shift) * B::size(blk);
#pragma unroll
                for (int i = 0; i < D / 32; i++) k.w[t][i] = *reinterpret_cast<const uint4 *>(at + ub * (D / 2) + 16 * i);
                if (D == 128) k.ks[t] = *reinterpret_cast<const uint2 *>(at + B::ks(blk) + ub * (D / 16));
                else k.ks[t].x = *reinterpret_cast<const uint32_t *>(at + B::ks(blk) + ub * (D / 16));
            }
        };
        auto unpack = [&](const Packed &from) {
            const uint4 (&w)[2][D / 32] = from.w;
            const uint2 (&ks)[2] = from.ks;
            const int kb = units % KB;
            if (units >= KB) wait(&sh.k_empty[kb], (units / KB + 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const uint32_t to = k_tmem + lanes + (kb * 2 + t) * (D / 2);
#pragma unroll
                for (int i = 0; i < D / 32; i++) {  // 32 channels: two scale blocks, 16 words
                    uint32_t o[16];
                    const uint32_t c[4] = {w[t][i].x, w[t][i].y, w[t][i].z, w[t][i].w};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int sb = 2 * i + (e >> 1);
                        const uint32_t byte = (sb < 4 ? ks[t].x : ks[t].y) >> (8 * (sb & 3)) & 0xffu;
                        const uint32_t s1 = e4m3x2_to_half2(static_cast<uint16_t>(byte)), s2 = __byte_perm(s1, s1, 0x1010);
                        uint32_t h[4];
                        e2m1x8_to_half(c[e], h);
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const uint32_t v = hmul2(h[k], s2);
                            o[4 * e + k] = BF16 ? half2_to_bf16(v) : v;
                        }
                    }
                    tmem_st16(to + 16 * i, o);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.k_full[kb]);
            units++;
        };
        // codes one unit ahead, page numbers two
        Packed cur, nxt;
        int id[2];
        g.find(sh, a, c0, c0, c1);
        numbers(g, id);
        load(g, id, cur);
        bool some = g.b0 < g.b1;  // of this unit
        g.next(sh, a, c0, c1);
        if (g.start < c1) numbers(g, id);
        for (;;) {
            const bool more = g.start < c1, now = some;
            if (more) {
                load(g, id, nxt);
                some = g.b0 < g.b1;
                g.next(sh, a, c0, c1);
                if (g.start < c1) numbers(g, id);
            }
            if (now) unpack(cur);
            if (!more) break;
            cur = nxt;
        }
        if (dt < 2) {  // (here, where there is time for it)
            Walk h(a);
            h.find(sh, a, dt == 0 ? c0 : c1 - 1, c0, c1);
            const bool mine = dt == 0 ? h.start < c0 : h.start >= c0 && h.end > c1;
            const int first = share_of(N, ctas, h.start);
            sh.joint[dt] = Joint{first, mine ? share_of(N, ctas, h.end - 1) - first : -1, h.r.row, h.head, h.j * KEYS, h.r.len, h.r.len - h.r.n};
        }
    } else if (warp != 14) {
        // ---- queries: three warps take the blocks in turn ----------------------------------------------
        constexpr int PIECES = D / 8, PER = 32 / PIECES;  // 16-byte pieces of a row, rows of a copy
        const unsigned turn = warp == 15 ? 2 : warp - 12;
        const int piece = lane % PIECES, sub = lane / PIECES;
        const uint32_t q_at = smem_u32(sh.q[0]) + (piece >> 3) * (COLS * 128);
        unsigned it = 0;
        // this lane's rows of a block: token and query head, none behind the last token of the block
        int tok[COLS / 32], gq[COLS / 32];
#pragma unroll
        for (int h = 0; h < COLS / 32; h++) {
            const int mine = 32 * h + lane;
            tok[h] = mine / p.G;
            gq[h] = mine % p.G;
            if (mine >= tb * p.G) tok[h] = 1 << 30;
        }
        for (g.find(sh, a, c0, c0, c1); g.start < c1; g.next(sh, a, c0, c1)) {
            const int old = g.r.len - g.r.n;
            const float *lses = a.lse + static_cast<long long>(g.r.q0) * p.Hq + g.head * p.G;
            const uint16_t *qs = a.q + g.r.q0 * a.qt + g.head * p.G * a.qh + 8 * piece;
            float lse[COLS / 32];
            auto ask = [&](int b) {  // what the rows of block b lose is on its way
#pragma unroll
                for (int h = 0; h < COLS / 32; h++)
                    lse[h] = b < g.b1 && tok[h] < g.r.n - b * tb ? lses[static_cast<long long>(b * tb + tok[h]) * p.Hq + gq[h]] : -INFINITY;
            };
            int b = g.b0 + static_cast<int>((turn + 3 - it % 3) % 3);  // the first that is this warp's
            const unsigned to_next = it + (g.b1 - g.b0);
            it += b - g.b0;
            ask(b);
            for (; b < g.b1; b += 3, it += 3) {
                const int st = it % ST;
                if (it >= ST) wait(&sh.q_empty[st], (it / ST + 1) & 1);
                unsigned there[COLS / 32], all = FULL;
#pragma unroll
                for (int h = 0; h < COLS / 32; h++) {
                    const int mine = 32 * h + lane;
                    there[h] = __ballot_sync(FULL, lse[h] != -INFINITY);
                    all &= there[h];
                    sh.less[st][mine] = lse[h] == -INFINITY ? -INFINITY : -lse[h] * LOG2E;
                    sh.pos[st][mine] = old + b * tb + tok[h];
                }
                mbar_arrive(&sh.q_full[st]);
                ask(b + 3);
                const uint16_t *block = qs + static_cast<long long>(b) * tb * a.qt;
                const uint32_t to = q_at + st * (COLS * D * 2);
                if (all == FULL) {
#pragma unroll 16
                    for (int i = 0; i < COLS; i += PER) copy16(to + swizzled(i + sub, piece & 7), block + sh.at[i + sub], true);
                } else {
#pragma unroll
                    for (int h = 0; h < COLS / 32; h++)
#pragma unroll 4
                        for (int i = 0; i < 32; i += PER) {
                            const int k = 32 * h + i + sub;
                            const bool is = there[h] >> (i + sub) & 1u;
                            copy16(to + swizzled(k, piece & 7), is ? block + sh.at[k] : a.q, is);
                        }
                }
                arrive_copied(&sh.q_full[st]);
            }
            it = to_next;
        }
        asm volatile("cp.async.wait_all;\n" ::: "memory");
    } else {
        // ---- products: the warp goes through them together, one lane issues them ---------------------------
        const uint32_t q_at = operand(smem_u32(sh.q[0]));
        unsigned it = 0, units = 0;
        for (g.find(sh, a, c0, c0, c1); g.start < c1; g.next(sh, a, c0, c1)) {
            if (g.b0 >= g.b1) continue;
            const int kb = units % KB;
            wait(&sh.k_full[kb], units / KB & 1);
            for (int b = g.b0; b < g.b1; b++, it++) {
                const int st = it % ST;
                wait(&sh.q_full[st], it / ST & 1);
                fence_proxy_async();  // the copies are the threads' writes, the products read through another proxy
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    const unsigned n = 2 * it + t, buf = n % RING;
                    if (n >= RING) wait(&sh.s_empty[buf], (n / RING + 1) & 1);
                    tc_fence_after();
                    const uint32_t ka = k_tmem + (kb * 2 + t) * (D / 2), qb = q_at + st * (COLS * D * 2 / 16);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < D / 16; i++)
                            mma_tmem(tmem + buf * COLS, ka + 8 * i, qb + (i >> 2) * (COLS * 8) + (i & 3) * 2, product(COLS, BF16), i > 0);
                        tc_commit(&sh.s_full[buf]);
                    }
                    __syncwarp();
                }
                if (elect_one()) tc_commit(&sh.q_empty[st]);
                __syncwarp();
            }
            if (elect_one()) tc_commit(&sh.k_empty[kb]);
            __syncwarp();
            units++;
        }
        if (elect_one()) tc_commit(&sh.drained);
        __syncwarp();
        if (!mbar_spin(&sh.drained, 0, a.wait_ns)) atomicOr(p.status, PST_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 14) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
    }
    // Units that CTAs share: the last one to bring its part (the count releases and acquires the parts) adds all up.
    if (tid < 64 && lane == 0) {
        const Joint &u = sh.joint[tid >> 5];
        int all = 0;
        if (u.others >= 0) {
            all = atomic_add_acq_rel_gpu(a.tickets + u.first, 1) == u.others;
            if (all) a.tickets[u.first] = 0;  // for the next call
        }
        sh.last[tid >> 5] = all;
    }
    __syncthreads();
    for (int k = 0; k < 2; k++) {
        const Joint &u = sh.joint[k];
        const int key = u.key0 + tid;
        if (!sh.last[k] || tid >= KEYS || key >= u.len) continue;
        float sum = 0.f;
        for (int i = 0; i <= u.others; i++) sum += __ldcg(a.records + (2LL * (u.first + i) + (i == 0)) * KEYS + tid);
        float *score = scores_of(a, u.row, u.head) + key;
        *score = (key < u.old ? *score : 0.f) + sum;
    }
}

template <int D, bool BF16>
int launch_as(const PagesWeighArgs &a, int grid, cudaStream_t st) {
    const int smem = static_cast<int>(sizeof(Shared<D>)) + 1024;  // room to put it on a 1024-byte boundary
    if (const int e = allow_shared<weigh_many<D, BF16>>(smem)) return e;
    weigh_many<D, BF16><<<grid, THREADS, smem, st>>>(a);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_pages_weigh_many(const PagesWeighArgs &a, int grid, void *stream) {
    auto st = static_cast<cudaStream_t>(stream);
    if (a.p.d == 128) return a.p.bf16 ? launch_as<128, true>(a, grid, st) : launch_as<128, false>(a, grid, st);
    return a.p.bf16 ? launch_as<64, true>(a, grid, st) : launch_as<64, false>(a, grid, st);
}

}  // namespace dq
