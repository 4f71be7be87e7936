// Paged cache: new tokens into pages (append) and back to 16 bits (read).
//
// A scale block is 16 channels of one token: top = max|x|, s = e4m3(top / 6 / 2^exp),
// codes e2m1(x / (2^exp s)), both as exact arithmetic would round them:
// - x / S is x (h + l) with h + l = 1 / S to 2^-44 in two fp32 numbers, h below 1 / S:
//   fma(x, h, x l) is on a border between two codes where the quotient is (the border has
//   3 bits), and elsewhere on its side, since x has at most 11 significant bits and a border
//   times S at most 7, so that no other quotient comes within 2^-12 of a border.  l >= 0
//   keeps the sign of a zero.
// - top / 6 is a product with a rounded 1 / 6 put on a grid of 17 bits; borders between
//   scales times 6 have at most 7 bits.
//
// 83 k tokens of 16 prompts (8 KV heads, head_dim 128; 437 MB) append in 100 us and read in 68.
// append: 14 instructions a value take 59 % of the issue slots and DRAM is busy for 51 %; 128
// registers a thread leave 16 warps an SM, which wait for loads and for one another's results:
// too little is in flight.  read: 8 instructions a value (54 % of the slots), DRAM 70 % busy.
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr int ST_THREADS = 128, ST_WARPS = ST_THREADS / 32;

// The larger magnitudes (with signs of no meaning), NaN where there is one.
template <bool BF16>
__device__ __forceinline__ uint32_t max2_abs(uint32_t a, uint32_t b) {
    uint32_t r;
    if (BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
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
template <bool BF16>
__device__ __forceinline__ float2 pair_to_float(uint32_t w) {
    if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// 16 channels of one token.
struct Block16 {
    uint32_t w[8];  // the values, two a word
    __device__ __forceinline__ void load(const uint16_t *x) {
        const uint4 a = *reinterpret_cast<const uint4 *>(x), b = *reinterpret_cast<const uint4 *>(x + 8);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = 0;
    }
    // The scale's byte, and 1 / S in two parts that turns values into codes (0 for S = 0).
    // `fine` is cleared where a value is not finite; the scale is then the largest one.
    template <bool BF16>
    __device__ __forceinline__ uint8_t scale(float sixth, float unit, float2 &r, bool &fine) const {
        uint32_t m = w[0];
#pragma unroll
        for (int i = 1; i < 8; i++) m = max2_abs<BF16>(m, w[i]);
        const uint32_t lo = m & 0x7fffu, hi = m >> 16 & 0x7fffu, inf = BF16 ? 0x7f80u : 0x7c00u;
        uint32_t top = lo > hi ? lo : hi;  // magnitudes order like their bits
        if (top >= inf) {
            top = inf;
            fine = false;
        }
        const float t = from16(static_cast<uint16_t>(top), BF16) * sixth;
        const uint8_t s = float_to_e4m3(__uint_as_float((__float_as_uint(t) + 0x40u) & ~0x7fu));
        const float S = e4m3_to_float(s) * unit;
        float h;
        asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(h) : "f"(S));
        h = __uint_as_float(__float_as_uint(h) - 2u);  // off by an ulp at most: below 1 / S now
        r = S > 0.f ? make_float2(h, fmaf(-S, h, 1.f) * h) : make_float2(0.f, 0.f);
        return s;
    }
};
__device__ __forceinline__ float quotient(float x, float2 r) { return fmaf(x, r.x, x * r.y); }

// One CTA per (row, touched page, KV head).  A block of B = min(P, 64) tokens at a time
// is put together in shared memory in the page's layout.  What a page holds already is
// read only where it is needed: its keys for the summary, and the groups of 8 tokens
// that the new ones share with others.  The page is one row's alone, so that no other
// CTA writes it.
template <int D, int B, bool BF16>
__global__ void __launch_bounds__(ST_THREADS) append_kernel(PagesStoreArgs a) {
    using L = PageBlock<D>;
    constexpr int C = D / 16;                                     // scale blocks of a token
    constexpr int KI = (B * C + ST_THREADS - 1) / ST_THREADS;     // (token, scale block) items of a thread
    constexpr int VI = (B / 2 * C + ST_THREADS - 1) / ST_THREADS; // (token pair, scale block) items
    __shared__ __align__(16) uint8_t img[L::size(B)];
    __shared__ float top_s[ST_WARPS][D], low_s[ST_WARPS][D], red[ST_WARPS];
    const PagesView &p = a.p;
    const PageRow r = page_row(p, a.r, blockIdx.y);
    const int head = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lo = r.len - r.n < 0 ? 0 : r.len - r.n;  // first position written
    const int j = lo / p.P + blockIdx.x;
    if (r.row < 0 || r.n == 0 || j * p.P >= r.len) return;
    // does the call bring tokens of this row a second time?  (two CTAs would write the same bytes)
    bool twice = false;
    if (a.r.rows)
        for (int i = tid; i < a.r.n_rows; i += ST_THREADS)
            twice |= a.r.rows[i] == r.row && i != static_cast<int>(blockIdx.y) && (!a.r.cu || a.r.cu[i + 1] > a.r.cu[i]);
    const int id = page_of(p, r.row, j);
    if (id < 0) return;
    const int t0 = lo > j * p.P ? lo - j * p.P : 0;  // new tokens of the page: [t0, t1)
    const int t1 = r.len - j * p.P < p.P ? r.len - j * p.P : p.P;
    const bool shared = p.refs[id] != 1;
    if (a.r.rows && __syncthreads_or(twice)) {
        if (tid == 0) atomicOr(p.status, PST_ARG);
        return;
    }
    if (shared) {
        if (tid == 0) atomicOr(p.status, PST_SHARED);
        return;
    }
    // the call's token at t = 0, k and v of this head there
    const long long first = r.q0 + (static_cast<long long>(j) * p.P - (r.len - r.n));
    const uint16_t *kp = a.k + first * a.kt + head * a.kh, *vp = a.v + first * a.vt + head * a.vh;
    const float ku = pow2i(p.k_exp), k6 = 0.16666667f * pow2i(-p.k_exp), vu = pow2i(p.v_exp), v6 = 0.16666667f * pow2i(-p.v_exp);
    bool fine = true;
    // summary: this thread's 8 channels over every (128 / (D / 8))-th token
    const int col = tid % (D / 8);
    uint32_t top[4], low[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        top[i] = 0xfc00fc00u;
        low[i] = 0x7c007c00u;
    }
    for (int b0 = 0; b0 < t1; b0 += B) {  // the page's blocks
        uint8_t *blk = page_ptr(p, id, head) + b0 / B * L::size(B);
        const int n0 = t0 > b0 ? t0 - b0 : 0, n1 = t1 - b0 < B ? t1 - b0 : B;  // the block's new tokens, if n0 < n1
        const bool some = n0 < n1;
        Block16 kx[KI], vx[VI][2];
        if (some) {  // the new tokens are on their way first
            const int tk = n0 + tid / C, tv = (n0 & ~1) + 2 * (tid / C);
            const uint16_t *kq = kp + (b0 + tk) * a.kt + 16 * (tid % C), *vq = vp + (b0 + tv) * a.vt + 16 * (tid % C);
#pragma unroll
            for (int i = 0; i < KI; i++)
                if (tk + i * (ST_THREADS / C) < n1) kx[i].load(kq + i * (ST_THREADS / C * a.kt));
#pragma unroll
            for (int i = 0; i < VI; i++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int t = tv + i * (2 * ST_THREADS / C) + e;
                    if (t >= n0 && t < n1) vx[i][e].load(vq + i * (2 * ST_THREADS / C * a.vt) + e * a.vt);
                    else vx[i][e].clear();
                }
        }
        const int g0 = some ? n0 / 8 : B / 8, g1 = (n1 + 7) / 8;  // 8-token groups written: [g0, g1)
        if (b0) __syncthreads();
        if (!some || n0 > 0 || (n1 & 7)) {  // old keys, for the summary and beside new ones in a group
            for (int i = tid; i < g1 * (D / 4); i += ST_THREADS) reinterpret_cast<uint4 *>(img)[i] = reinterpret_cast<const uint4 *>(blk)[i];
            for (int i = tid; i < g1 * (D / 32); i += ST_THREADS)
                reinterpret_cast<uint4 *>(img + L::ks(B))[i] = reinterpret_cast<const uint4 *>(blk + L::ks(B))[i];
        }
        for (int g = g0; g < g1; g++) {  // old values beside new ones in a group
            if (8 * g >= n0 && 8 * g + 8 <= n1) continue;
            for (int i = tid; i < D / 4 + D / 32; i += ST_THREADS) {
                const int at = i < D / 4 ? L::vc(B) + g * 4 * D + 16 * i : L::vs(B) + g * (D / 2) + 16 * (i - D / 4);
                *reinterpret_cast<uint4 *>(img + at) = *reinterpret_cast<const uint4 *>(blk + at);
            }
        }
        __syncthreads();
        if (some) {
#pragma unroll
            for (int i = 0; i < KI; i++) {
                const int u = tid + i * ST_THREADS, t = n0 + u / C, c = u % C;
                if (t >= n1) break;
                float2 rc;
                img[L::ks(B) + t * C + c] = kx[i].template scale<BF16>(k6, ku, rc, fine);
                uint32_t code[2];
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float2 f = pair_to_float<BF16>(kx[i].w[4 * k + e]);
                        x[2 * e] = quotient(f.x, rc);
                        x[2 * e + 1] = quotient(f.y, rc);
                    }
                    code[k] = float8_to_e2m1(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
                }
                *reinterpret_cast<uint2 *>(img + t * (D / 2) + 8 * c) = make_uint2(code[0], code[1]);
            }
#pragma unroll
            for (int i = 0; i < VI; i++) {
                const int u = tid + i * ST_THREADS, t = (n0 & ~1) + 2 * (u / C), c = u % C;
                if (t >= n1) break;
                const bool e0 = t >= n0, e1 = t + 1 < n1;
                float2 r0 = make_float2(0.f, 0.f), r1 = r0;
                uint8_t *cp = img + L::vc(B) + L::vcode(t, c), *sp = img + L::vs(B) + L::vscale(t, c);
                if (e0) sp[0] = vx[i][0].template scale<BF16>(v6, vu, r0, fine);
                if (e1) sp[1] = vx[i][1].template scale<BF16>(v6, vu, r1, fine);
                uint32_t code[4];  // a byte is a channel: even token low, odd token high
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float2 x = pair_to_float<BF16>(vx[i][0].w[2 * k]), y = pair_to_float<BF16>(vx[i][1].w[2 * k]);
                    const float2 z = pair_to_float<BF16>(vx[i][0].w[2 * k + 1]), w = pair_to_float<BF16>(vx[i][1].w[2 * k + 1]);
                    code[k] = float8_to_e2m1(quotient(x.x, r0), quotient(y.x, r1), quotient(x.y, r0), quotient(y.y, r1), quotient(z.x, r0),
                                             quotient(w.x, r1), quotient(z.y, r0), quotient(w.y, r1));
                }
                uint4 *dst = reinterpret_cast<uint4 *>(cp);
                if (!e0 || !e1) {  // one of the two is new
                    const uint32_t m = e0 ? 0x0f0f0f0fu : 0xf0f0f0f0u;
                    const uint4 old = *dst;
                    code[0] = (code[0] & m) | (old.x & ~m);
                    code[1] = (code[1] & m) | (old.y & ~m);
                    code[2] = (code[2] & m) | (old.z & ~m);
                    code[3] = (code[3] & m) | (old.w & ~m);
                }
                *dst = make_uint4(code[0], code[1], code[2], code[3]);
            }
        }
        __syncthreads();
        // the groups with new tokens go back
        const int n = g1 - g0;
        for (int i = tid; i < n * (D / 4); i += ST_THREADS) {
            const int at = g0 * 4 * D + 16 * i;
            *reinterpret_cast<uint4 *>(blk + at) = *reinterpret_cast<const uint4 *>(img + at);
            *reinterpret_cast<uint4 *>(blk + L::vc(B) + at) = *reinterpret_cast<const uint4 *>(img + L::vc(B) + at);
        }
        for (int i = tid; i < n * (D / 32); i += ST_THREADS) {
            const int at = g0 * (D / 2) + 16 * i;
            *reinterpret_cast<uint4 *>(blk + L::ks(B) + at) = *reinterpret_cast<const uint4 *>(img + L::ks(B) + at);
            *reinterpret_cast<uint4 *>(blk + L::vs(B) + at) = *reinterpret_cast<const uint4 *>(img + L::vs(B) + at);
        }
        for (int t = tid / (D / 8); t < n1; t += ST_THREADS / (D / 8)) {
            uint32_t h[4];
            e2m1x8_to_half(*reinterpret_cast<const uint32_t *>(img + t * (D / 2) + 4 * col), h);
            const uint32_t s = e4m3x2_to_half2(img[L::ks(B) + t * C + (col >> 1)]), s2 = __byte_perm(s, s, 0x1010);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                h[i] = hmul2(h[i], s2);  // exact
                top[i] = hmax2(top[i], h[i]);
                low[i] = hmin2(low[i], h[i]);
            }
        }
    }
    if (!fine) atomicOr(p.status, PST_NONFINITE);
    // the threads with the same channels: within the warp, then over the warps
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
        for (int i = 0; i < ST_WARPS; i++) {
            mx = fmaxf(mx, top_s[i][tid]);
            mn = fminf(mn, low_s[i][tid]);
        }
    const float w = warp_max(tid < D ? fmaxf(fabsf(mx), fabsf(mn)) : 0.f);
    if (lane == 0) red[warp] = w;
    __syncthreads();
    float most = red[0];
#pragma unroll
    for (int i = 1; i < ST_WARPS; i++) most = fmaxf(most, red[i]);
    // held keys are multiples of 2^-10 below 2^12 of at most 6 bits: most = m 2^E, E from the exponent field
    const int e = most > 0.f ? static_cast<int>(__float_as_uint(most) >> 23) - 126 - 7 : 0;
    uint8_t *sum = summary_ptr(p, id, head);
    if (tid < D) {
        const float unit = pow2i(-e);
        reinterpret_cast<int8_t *>(sum)[tid] = static_cast<int8_t>(ceilf(mx * unit));
        reinterpret_cast<int8_t *>(sum)[D + tid] = static_cast<int8_t>(floorf(mn * unit));
    }
    if (tid == 0) *reinterpret_cast<int *>(sum + 2 * D) = e;
}

// A half2 of held values (in units of 2^exp) -> 16-bit words.
template <bool BF16>
__device__ __forceinline__ uint32_t held_to_16(uint32_t h, float unit) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    uint32_t r;
    if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(f.y * unit), "f"(f.x * unit));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(f.y * unit), "f"(f.x * unit));
    return r;
}

// One thread per (group of 8 positions, KV head, 8 channels): a group is in one page.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) read_kernel(PagesReadArgs a) {
    const PagesView &p = a.p;
    const PageRow r = page_row(p, a.r, blockIdx.y);
    using B = PageBlock<D>;
    constexpr int C8 = D / 8;
    const int pos0 = r.len - r.n;  // the first token's position
    const int group0 = pos0 >> 3, groups = r.n ? ((r.len - 1) >> 3) - group0 + 1 : 0;
    const float ku = pow2i(p.k_exp), vu = pow2i(p.v_exp);
    const int c8 = threadIdx.x % C8, units = groups * p.Hkv;
    for (int u = blockIdx.x * (256 / C8) + threadIdx.x / C8; u < units; u += gridDim.x * (256 / C8)) {
        const int gr = u / p.Hkv, head = u - gr * p.Hkv, pos = 8 * (group0 + gr);
        int id = -1;
        if (pos >= 0 && r.row >= 0 && pos < r.len) id = page_of(p, r.row, pos / p.P);
        uint32_t kw[8], ks[8], vs[4];
        uint2 vw[4];
        if (id >= 0) {
            const int t = pos % p.P, tb = t % p.blk, b = p.blk;
            const uint8_t *blk = page_ptr(p, id, head) + t / b * B::size(b);
            const uint8_t *kc = blk + tb * (D / 2) + 4 * c8, *kb = blk + B::ks(b) + tb * (D / 16) + (c8 >> 1);
            const uint8_t *vc = blk + B::vc(b) + B::vcode(tb, c8 >> 1) + 8 * (c8 & 1), *vb = blk + B::vs(b) + B::vscale(tb, c8 >> 1);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                kw[e] = *reinterpret_cast<const uint32_t *>(kc + e * (D / 2));
                ks[e] = kb[e * (D / 16)];
            }
#pragma unroll
            for (int e = 0; e < 4; e++) {
                vw[e] = *reinterpret_cast<const uint2 *>(vc + 16 * e);
                vs[e] = *reinterpret_cast<const uint16_t *>(vb + 2 * e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) kw[e] = ks[e] = 0;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                vw[e] = make_uint2(0, 0);
                vs[e] = 0;
            }
        }
        const long long o = ((static_cast<long long>(r.q0) + pos - pos0) * p.Hkv + head) * D + 8 * c8;
        uint16_t *ko = a.k + o, *vo = a.v + o;
        const int stride = p.Hkv * D;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            if (pos + e < pos0 || pos + e >= r.len) continue;
            uint32_t h[4];
            e2m1x8_to_half(kw[e], h);
            const uint32_t s = e4m3x2_to_half2(static_cast<uint16_t>(ks[e])), s2 = __byte_perm(s, s, 0x1010);
#pragma unroll
            for (int x = 0; x < 4; x++) h[x] = held_to_16<BF16>(hmul2(h[x], s2), ku);
            *reinterpret_cast<uint4 *>(ko + e * stride) = make_uint4(h[0], h[1], h[2], h[3]);
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
            uint32_t x[4], y[4], w[2][4];  // a half2 is the two tokens of a channel
            e2m1x8_to_half(vw[e].x, x);
            e2m1x8_to_half(vw[e].y, y);
            const uint32_t s = e4m3x2_to_half2(static_cast<uint16_t>(vs[e]));
#pragma unroll
            for (int i = 0; i < 4; i++) {
                x[i] = hmul2(x[i], s);
                y[i] = hmul2(y[i], s);
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                w[0][i] = held_to_16<BF16>(__byte_perm(x[2 * i], x[2 * i + 1], 0x5410), vu);
                w[1][i] = held_to_16<BF16>(__byte_perm(x[2 * i], x[2 * i + 1], 0x7632), vu);
                w[0][i + 2] = held_to_16<BF16>(__byte_perm(y[2 * i], y[2 * i + 1], 0x5410), vu);
                w[1][i + 2] = held_to_16<BF16>(__byte_perm(y[2 * i], y[2 * i + 1], 0x7632), vu);
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int at = pos + 2 * e + i;
                if (at < pos0 || at >= r.len) continue;
                *reinterpret_cast<uint4 *>(vo + (2 * e + i) * stride) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            }
        }
    }
}

template <int D, int B>
void append_of(const PagesStoreArgs &a, dim3 grid, cudaStream_t st) {
    if (a.p.bf16) append_kernel<D, B, true><<<grid, ST_THREADS, 0, st>>>(a);
    else append_kernel<D, B, false><<<grid, ST_THREADS, 0, st>>>(a);
}
template <int D>
void read_of(const PagesReadArgs &a, dim3 grid, cudaStream_t st) {
    if (a.p.bf16) read_kernel<D, true><<<grid, 256, 0, st>>>(a);
    else read_kernel<D, false><<<grid, 256, 0, st>>>(a);
}
template <int D>
void append_as(const PagesStoreArgs &a, dim3 grid, cudaStream_t st) {
    if (a.p.blk == 64) append_of<D, 64>(a, grid, st);
    else if (a.p.blk == 32) append_of<D, 32>(a, grid, st);
    else append_of<D, 16>(a, grid, st);
}

}  // namespace

int launch_pages_append(const PagesStoreArgs &a, void *stream) {
    // a row's new tokens touch at most this many pages
    const int most = (a.r.max_new + a.p.P - 2) / a.p.P + 1;
    const dim3 grid(most < a.p.M ? most : a.p.M, a.r.n_rows, a.p.Hkv);
    auto st = static_cast<cudaStream_t>(stream);
    if (a.p.d == 128) append_as<128>(a, grid, st);
    else append_as<64>(a, grid, st);
    return static_cast<int>(cudaGetLastError());
}

int launch_pages_read(const PagesReadArgs &a, void *stream) {
    const long long per = static_cast<long long>((a.r.max_new + 6) / 8 + 1) * a.p.Hkv * (a.p.d / 8);
    const long long want = (per + 255) / 256;
    const dim3 grid(static_cast<unsigned>(want < 4096 ? want : 4096), a.r.n_rows);
    auto st = static_cast<cudaStream_t>(stream);
    if (a.p.d == 128) read_of<128>(a, grid, st);
    else read_of<64>(a, grid, st);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace dq
