// Paged cache: attention of many new tokens (a prompt's chunk) over 4-bit pages, on the
// 5th-generation tensor cores.
//
// Same mathematics as the kernel for few tokens: z = f q . k, p = exp2(z - m + LIFT),
// out = (sum p v) / (sum p).  4 D products and one exponential for each (query, key)
// pair: the kernel is bound by the tensor cores and, nearly as much, by the exponentials
// and their conversions.  2048 new tokens over 16384 (32 / 8 heads, head_dim 128) take
// 433 us, 1.19 PFLOP/s; over 131072, 3.3 ms, 1.32.
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
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr float LN2 = 0.69314718055994530942f;
constexpr float LIFT = 7.f;       // log2 units: weights are 2^LIFT at a logit of m ...
constexpr float MOST = 32768.f;   // ... and may grow to 2^15 (a logit 2^8 over m) before m is raised
constexpr int TILE = 128, ROWS = 2 * TILE;   // query rows of a tile, of a unit
constexpr int KEYS = 128;                    // keys at a time
constexpr int UNIT_COST = 512, MIN_SHARE = 1024;  // tokens: of a unit's beginning and end; that make a CTA worth its parts
constexpr int THREADS = 512;

// ---- tensor memory and tensor cores --------------------------------------------------------
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
        "%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
          "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
        "%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
        "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(addr), "r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
        "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Wait for the loads so far; nothing that uses r moves before it.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; i++) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
                   "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
// Arrive on `bar` when every product issued so far is done.
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
// The warp arrives, once for all its lanes' work before it.
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
// Wait for phase `parity` of an mbarrier, for `limit_ns` at most.  The hand-overs here are
// short and frequent: no hint to sleep long, and the clock is seldom looked at.
__device__ __forceinline__ bool mbar_spin(uint64_t *bar, unsigned parity, uint64_t limit_ns) {
    const uint32_t addr = smem_u32(bar);
    uint64_t t0 = 0;
    for (unsigned it = 0;; ++it) {
        uint32_t done;
        asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                     : "=r"(done)
                     : "r"(addr), "r"(parity)
                     : "memory");
        if (done) return true;
        if ((it & 1023u) == 0) {
            if (it == 0) t0 = global_ns();
            else if (global_ns() - t0 > limit_ns) return false;
        }
    }
}
// Descriptor of a K-major operand with 128-byte swizzle (8 rows of 128 bytes are 1024
// bytes): its low word holds the address in units of 16 bytes, so that an operand n bytes
// further on is n / 16 more.
__device__ __forceinline__ uint32_t operand(uint32_t addr) { return (addr >> 4 & 0x3fffu) | 1u << 16; }
constexpr uint32_t OPERAND_HIGH = 1024u >> 4 | 1u << 14 | 2u << 29;
// D += A B (D = A B where `add` is 0); descriptors by their low words.
__device__ __forceinline__ void mma_smem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 x, y;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(add), "r"(OPERAND_HIGH)
        : "memory");
}
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 y;\n mov.b64 y, {%2, %5};\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(add), "r"(OPERAND_HIGH)
        : "memory");
}
// Instruction descriptor: binary16 operands, both K-major, fp32 accumulators, M = 128.
__host__ __device__ constexpr uint32_t product(int n) { return 1u << 4 | static_cast<uint32_t>(n / 8) << 17 | (TILE / 16u) << 24; }
// Byte offset of 16-byte piece c (8 elements) of row r, in a panel of 64 elements a row.
__device__ __forceinline__ int swizzled(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

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

// Two fp32 numbers at a time.
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 both(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
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
    int row[DQ_PAGES_MAX_ROWS], len[DQ_PAGES_MAX_ROWS];
    long long part[THREADS / 32];
    uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], drained;
    uint32_t tmem;
};

__device__ __forceinline__ long long blocks_before(long long base, int tb, int b) {  // places of blocks 0 .. b - 1 of one head
    return b * (base + UNIT_COST) + static_cast<long long>(tb) * b * (b + 1) / 2;
}
__device__ __forceinline__ PageRow known_row(const int *row, const int *len, const PagesAttnArgs &a, int i) {
    PageRow r;
    r.row = row[i];
    r.len = len[i];
    r.q0 = a.r.cu ? a.r.cu[i] : i;
    r.n = a.r.cu ? a.r.cu[i + 1] - r.q0 : 1;
    return r;
}
template <int D>
__device__ Unit find_unit(const Shared<D> &sh, const PagesAttnArgs &a, int tb, long long x) {
    int lo = 0, hi = a.r.n_rows - 1;
    while (lo < hi) {  // the last row that begins at or before x
        const int mid = (lo + hi + 1) >> 1;
        if (sh.first[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    Unit u;
    u.i = lo;
    u.r = known_row(sh.row, sh.len, a, lo);
    const long long base = u.r.len > u.r.n ? u.r.len - u.r.n : 0, in = x - sh.first[lo];
    int b0 = 0, b1 = (u.r.n - 1) / tb;
    while (b0 < b1) {
        const int mid = (b0 + b1 + 1) >> 1;
        if (a.p.Hkv * blocks_before(base, tb, mid) <= in) b0 = mid;
        else b1 = mid - 1;
    }
    u.b = b0;
    const long long before = a.p.Hkv * blocks_before(base, tb, b0), w = base + UNIT_COST + static_cast<long long>(b0 + 1) * tb;
    u.head = static_cast<int>((in - before) / w);
    u.start = sh.first[lo] + before + u.head * w;
    u.end = u.start + w;
    return u;
}
__device__ __forceinline__ long long share(long long n, int m, int k) {
    const long long q = n / m, rest = n - q * m;
    return k * q + (k < rest ? k : rest);
}
__device__ __forceinline__ int share_of(long long n, int m, long long x) {
    const long long q = n / m, rest = n - q * m, ahead = rest * (q + 1);
    return static_cast<int>(x < ahead ? x / (q + 1) : rest + (x - ahead) / q);
}

// A segment: this CTA's part of a unit, key tiles [t0, t1).
struct Segment {
    Unit u;
    int t0, t1;
    bool begins, ends;
};
template <int D>
__device__ Segment find_segment(const Shared<D> &sh, const PagesAttnArgs &a, int tb, long long x, long long c1) {
    Segment s;
    s.u = find_unit<D>(sh, a, tb, x);
    s.begins = x <= s.u.start;
    s.ends = s.u.end <= c1;
    const int last = (s.u.b + 1) * tb < s.u.r.n ? (s.u.b + 1) * tb : s.u.r.n;
    const int seen = s.u.r.len - s.u.r.n + last;  // keys that the block's last token sees
    const int tiles = seen > 0 ? (seen + KEYS - 1) / KEYS : 0;
    auto tile_at = [&](long long at) {
        const long long t = (at - s.u.start - UNIT_COST + KEYS - 1) / KEYS;
        return at - s.u.start <= UNIT_COST ? 0 : (t < tiles ? static_cast<int>(t) : tiles);
    };
    s.t0 = s.begins ? 0 : tile_at(x);
    s.t1 = s.ends ? tiles : tile_at(c1);
    return s;
}

// ---- the kernel --------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(THREADS, 1) attn_prompt(PagesAttnArgs a) {
    extern __shared__ uint8_t raw[];
    using S = Shared<D>;
    using B = PageBlock<D>;
    S &sh = *reinterpret_cast<S *>(raw + (-smem_u32(raw) & 1023u));
    const PagesView &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tb = ROWS / p.G;  // tokens of a block
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
    // places before each row
    long long base = 0;
    for (int i0 = 0; i0 < a.r.n_rows; i0 += THREADS) {
        const int i = i0 + tid;
        long long w = 0;
        if (i < a.r.n_rows) {
            const PageRow r = page_row(p, a.r, i);
            sh.row[i] = r.row;
            sh.len[i] = r.len;
            if (r.len > 0 && takes(a, r)) w = p.Hkv * blocks_before(r.len > r.n ? r.len - r.n : 0, tb, (r.n + tb - 1) / tb);
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
    for (int i = blockIdx.x; i < a.r.n_rows; i += gridDim.x) {
        if (sh.len[i] > 0) continue;
        const PageRow r = page_row(p, a.r, i);
        if (!takes(a, r)) continue;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + static_cast<long long>(r.q0) * p.Hq * D);
        for (long long k = tid; k < static_cast<long long>(r.n) * p.Hq * (D / 8); k += THREADS) o[k] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (long long k = tid; k < static_cast<long long>(r.n) * p.Hq; k += THREADS) a.lse[static_cast<long long>(r.q0) * p.Hq + k] = -INFINITY;
    }
    int ctas = static_cast<int>(N / MIN_SHARE < gridDim.x ? N / MIN_SHARE : gridDim.x);
    if (ctas < 1) ctas = 1;
    int4 *join = reinterpret_cast<int4 *>(a.joins) + blockIdx.x;
    if (N == 0 || static_cast<int>(blockIdx.x) >= ctas) {
        if (tid == 0) *join = make_int4(0, 0, 0, 0);
        return;
    }
    const long long c0 = share(N, ctas, blockIdx.x), c1 = share(N, ctas, blockIdx.x + 1);
    if (tid == 0) {  // the unit that begins here and goes on in other CTAs, if any
        const Unit u = find_unit<D>(sh, a, tb, c1 - 1);
        const bool on = u.start >= c0 && u.end > c1;
        *join = on ? make_int4(u.i, u.head, u.b, share_of(N, ctas, u.end - 1) - static_cast<int>(blockIdx.x) + 1) : make_int4(0, 0, 0, 0);
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
        const int t = warp >> 2, mine = tid & (TILE - 1), row = tid;  // tile, row of the tile, row of the unit
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes of tensor memory
        const uint32_t s_at = tmem + lanes + t * KEYS, o_at = tmem + lanes + 2 * KEYS + t * D;
        unsigned runs = 0, it = 0;
        for (long long x = c0; x < c1;) {
            const Segment g = find_segment<D>(sh, a, tb, x, c1);
            const PageRow &r = g.u.r;
            x = g.u.end;
            const int tok = g.u.b * tb + row / p.G, gq = row % p.G;
            const bool real = row < tb * p.G && tok < r.n;
            const int pos = real ? r.len - r.n + tok : 0x7fffffff;  // no row: nothing to mask
            // the query, by a power of two below 2^14 and with sm_scale's sign, as binary16
            RowState row_s{0.f, -INFINITY, {0, 0}};
            if (g.t0 < g.t1) {
                const uint16_t *src = a.q + (static_cast<long long>(r.q0) + tok) * a.qt + (g.u.head * p.G + gq) * a.qh;
                uint4 w[D / 8];
#pragma unroll
                for (int i = 0; i < D / 8; i++) w[i] = real ? *reinterpret_cast<const uint4 *>(src + 8 * i) : make_uint4(0, 0, 0, 0);
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < D / 8; i++) {
                    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        top = fmaxf(top, fmaxf(fabsf(from16(static_cast<uint16_t>(u[j] & 0xffffu), p.bf16)), fabsf(from16(static_cast<uint16_t>(u[j] >> 16), p.bf16))));
                }
                int up = 13 - (static_cast<int>(__float_as_uint(top) >> 23) - 127);
                up = top > 0.f ? (up > 126 ? 126 : up) : 0;
                const float by = a.scale_log2 < 0.f ? -pow2i(up) : pow2i(up);
                // (never 0: a hidden key's -inf stays one)
                row_s.f = fmaxf(fabsf(a.scale_log2) * pow2i(-up), 1e-37f);
#pragma unroll
                for (int i = 0; i < D / 8; i++) {
                    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        h[j] = half2_of(from16(static_cast<uint16_t>(u[j] & 0xffffu), p.bf16) * by, from16(static_cast<uint16_t>(u[j] >> 16), p.bf16) * by);
                    *reinterpret_cast<uint4 *>(sh.q[t] + (i >> 3) * (TILE * 128) + swizzled(mine, i & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                fence_proxy_async();
                mbar_arrive(&sh.q_full[t]);
            }
            const int least = __reduce_min_sync(FULL, pos);
            for (int k = g.t0; k < g.t1; k++, it++) {
                wait(&sh.s_full[t], it & 1);
                tc_fence_after();
                const int key0 = k * KEYS;
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
                // last 32 keys' load is of columns that nobody uses; unrolled without it 468 us where this takes 430).
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
            const float l = row_s.sum(), m = row_s.m, by = l == 0.f ? 0.f : a.out_scale / l;
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
                } else if (real) {
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
                const int key = tile * KEYS + dt, tok = tile * KEYS + 8 * kg;
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
            if (g.t0 < g.t1) load(cur, g.t0, number(g.t0 * KEYS + dt), number(g.t0 * KEYS + 8 * kg));
            int idk = number((g.t0 + 1) * KEYS + dt), idv = number((g.t0 + 1) * KEYS + 8 * kg);
            for (int k = g.t0; k < g.t1; k++, it++) {
                if (k + 1 < g.t1) {
                    load(nxt, k + 1, idk, idv);
                    idk = number((k + 2) * KEYS + dt);
                    idv = number((k + 2) * KEYS + 8 * kg);
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
                        const int tok = k * KEYS + 8 * kg + 2 * e;  // tokens that are not there: 0, whatever their bytes say
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
    } else if (warp == 12 && lane == 0) {
        // ---- products -----------------------------------------------------------------------------
        unsigned runs = 0, it = 0;
        uint32_t q_at[2], s_at[2], o_at[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
            q_at[t] = operand(smem_u32(sh.q[t]));
            s_at[t] = tmem + t * KEYS;
            o_at[t] = tmem + 2 * KEYS + t * D;
        }
        const uint32_t k_at = operand(smem_u32(sh.k[0])), v_at = operand(smem_u32(sh.v[0]));
        constexpr uint32_t STAGE = KEYS * D * 2 / 16;
        auto scores = [&](int t, int st) {
            const uint32_t kb = k_at + st * STAGE;
#pragma unroll
            for (int i = 0; i < D / 16; i++)
                mma_smem(s_at[t], q_at[t] + (i >> 2) * (TILE * 8) + (i & 3) * 2, kb + (i >> 2) * (KEYS * 8) + (i & 3) * 2, product(KEYS), i > 0);
            tc_commit(&sh.s_full[t]);
        };
        for (long long x = c0; x < c1;) {
            const Segment g = find_segment<D>(sh, a, tb, x, c1);
            x = g.u.end;
            if (g.t0 >= g.t1) continue;
            wait(&sh.k_full[it & 1], it >> 1 & 1);
#pragma unroll
            for (int t = 0; t < 2; t++) {
                wait(&sh.q_full[t], runs & 1);
                tc_fence_after();
                scores(t, it & 1);
            }
            tc_commit(&sh.k_empty[it & 1]);
            runs++;
            for (int k = g.t0; k < g.t1; k++, it++) {
                const int st = it & 1, next = (it + 1) & 1;
                const uint32_t vb = v_at + st * STAGE;
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    wait(&sh.p_full[t], it & 1);
                    if (t == 0) wait(&sh.v_full[st], it >> 1 & 1);
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < KEYS / 16; i++)
                        mma_tmem(o_at[t], s_at[t] + 8 * i, vb + (i >> 2) * (D * 8) + (i & 3) * 2, product(D), k > g.t0 || i > 0);
                    if (t == 1) tc_commit(&sh.v_empty[st]);
                    if (k + 1 < g.t1) {
                        if (t == 0) wait(&sh.k_full[next], (it + 1) >> 1 & 1);
                        if (t == 0) tc_fence_after();
                        scores(t, next);
                        if (t == 1) tc_commit(&sh.k_empty[next]);
                    } else {
                        tc_commit(&sh.o_full[t]);
                    }
                }
            }
        }
        // (where no wait ran out, the softmax has waited for the same products)
        tc_commit(&sh.drained);
        if (!mbar_spin(&sh.drained, 0, a.wait_ns)) atomicOr(p.status, PST_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
    }

}

// The units that crossed a share's border: CTA (c, y) adds up the parts of the unit that
// began in share c and went on, 16 channels of its 256 rows, in CTA order.
template <int D>
__global__ void __launch_bounds__(ROWS) join_parts(PagesAttnArgs a) {
    const int4 what = reinterpret_cast<const int4 *>(a.joins)[blockIdx.x];  // row of the call, KV head, block, parts
    const int n = what.w, row = threadIdx.x, tb = ROWS / a.p.G, c = blockIdx.y;
    const PagesView &p = a.p;
    if (n == 0) return;
    const PageRow r = page_row(p, a.r, what.x);
    const int tok = what.z * tb + row / p.G;
    if (row >= tb * p.G || tok >= r.n) return;
    constexpr int REC = ROWS * (D + 2);
    float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
    for (int i = 0; i < 16; i++) acc[i] = 0.f;
#pragma unroll 2
    for (int j = 0; j < n; j++) {
        const float *rec = a.records + (2LL * (blockIdx.x + j) + (j == 0)) * REC;
        const float mk = rec[ROWS * D + row], lk = rec[ROWS * (D + 1) + row];
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = *reinterpret_cast<const float4 *>(rec + ((4 * c + i) * ROWS + row) * 4);
        const float mx = fmaxf(m, mk), mu = mx == -INFINITY ? 0.f : mx;
        const float wa = ex2(m - mu), wb = ex2(mk - mu);  // 0 for a part that saw nothing
        m = mx;
        l = l * wa + lk * wb;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            acc[4 * i] = acc[4 * i] * wa + v[i].x * wb;
            acc[4 * i + 1] = acc[4 * i + 1] * wa + v[i].y * wb;
            acc[4 * i + 2] = acc[4 * i + 2] * wa + v[i].z * wb;
            acc[4 * i + 3] = acc[4 * i + 3] * wa + v[i].w * wb;
        }
    }
    const long long o = (static_cast<long long>(r.q0) + tok) * p.Hq + what.y * p.G + row % p.G;
    const float by = l == 0.f ? 0.f : a.out_scale / l;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; i++) w[i] = pack2(to16(acc[2 * i] * by, p.bf16), to16(acc[2 * i + 1] * by, p.bf16));
    uint4 *dst = reinterpret_cast<uint4 *>(a.out + o * D + 16 * c);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (c == 0 && a.lse) a.lse[o] = l == 0.f ? -INFINITY : (m - LIFT + log2f(l)) * LN2;
}

template <int D>
int launch_as(const PagesAttnArgs &a, int grid, cudaStream_t st) {
    const int smem = static_cast<int>(sizeof(Shared<D>)) + 1024;  // room to put it on a 1024-byte boundary
    if (const int e = allow_shared<attn_prompt<D>>(smem)) return e;
    attn_prompt<D><<<grid, THREADS, smem, st>>>(a);
    const cudaError_t e1 = cudaGetLastError();
    if (e1 != cudaSuccess) return static_cast<int>(e1);
    join_parts<D><<<dim3(grid, D / 16), ROWS, 0, st>>>(a);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_pages_prompt(const PagesAttnArgs &a, int grid, void *stream) {
    return a.p.d == 128 ? launch_as<128>(a, grid, static_cast<cudaStream_t>(stream)) : launch_as<64>(a, grid, static_cast<cudaStream_t>(stream));
}

}  // namespace dq
