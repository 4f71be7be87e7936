// Paged cache: attention of each row's newest tokens over its 4-bit pages.
//
// For a query at position x, with z_j = sm_scale q . k_j over the visible keys j <= x:
//   m = max z_j, l = sum exp(z_j - m), out = sum exp(z_j - m) v_j / l, lse = m + log l
// in one pass over the pages.
//
// Work.  A unit is 8 NT query rows (token, query head of the group) of one row and KV
// head; it walks the row's tokens in chunks of 32.  All units' chunks, in order, are cut
// into equal shares, one for each warp of one CTA per SM, so that ragged lengths and
// small batches fill the card alike.  A warp that holds all of a unit writes its output;
// parts of a unit meet in shared memory, and parts in several CTAs in the workspace,
// where the last CTA to arrive adds them up in CTA order (so that the result does not
// depend on timing; nobody waits).
//
// A chunk.  Each warp has a ring of its own in shared memory, filled by bulk copies (four
// a chunk: codes and scales of keys and of values; eight where a page is 16 tokens) that
// run ahead of it, so that no warp waits for another and 16 warps x 1.5 chunks keep
// 110 KB in flight per SM.  The page layout is made for the product: a lane's 16 bytes
// are its own operands, without bank conflicts.  Codes become binary16 by one
// conversion and one multiplication by the scale, both exact (2 + 4 significant bits,
// multiples of 2^-10 below 2^12).  Both products run on mma.sync m16n8k16 with
// the cache as the 16-row operand: K [16 tokens x 16 channels] . Q^T and
// V^T [16 channels x 16 tokens] . P, in which 8 query rows fill the n of 8.
// Lane (g, t) = (lane / 4, lane % 4) holds, of D / 4 channels at t D / 4, tokens g and
// g + 8 of K; of D / 8 channels at g D / 8, token pairs t and t + 4 of V.
//
// Rounding.  Queries are scaled by a power of two to at most 2^14 and are exact in
// binary16 down to 2^-38 of their row's largest.  Weights exp2(z - m + 7) are rounded to
// binary16 for P . V (11 bits; 8 bits of slack for m, which is raised only when a logit
// passes it by 2^8, and 7 bits up so that weights below binary16's normal range are
// those under 2^-21); sums, logits and accumulators are fp32.
#pragma once

#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr float LN2 = 0.69314718055994530942f;
constexpr float SLACK = 8.f, LIFT = 7.f;   // log2 units
constexpr int CHUNK = 32;                  // tokens
constexpr int UNIT_COST = FEW_UNIT_COST;   // (40 ragged rows: 76 us, with 0 94)
// Places of a unit that CTAs do not share; of common pages, which few units have, fewer (8 rows behind 2000 tokens, which are shared
// only where the caller asks for it always, four layers: 77 us, with 64 93; 8 groups of 8 behind 2048 37.7 / 36.1, 20 of 3 behind 2560
// 45.2 / 41.2; with 8 places 16 groups of 8 behind 1024 40.1 for 33.2).
constexpr int SHORT_ROWS = 64, SHORT_COMMON = 24;
constexpr int MIN_PLACES = 16;             // places that make a CTA worth its merge (1 row of 500: 8.4 us, with 64 13.4)

__device__ __forceinline__ void mbar_expect(uint32_t bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, unsigned bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// ---- a chunk in shared memory: a block of 32 tokens in the page's own layout ---------------
template <int N>
__device__ __forceinline__ void ld_words(const uint8_t *p, uint32_t (&w)[N]) {
    if (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[N > 2 ? 2 : 0] = v.z;
        w[N > 3 ? 3 : 0] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    }
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// ---- a warp's state over a unit: lane (g, t) holds query rows 2t and 2t + 1 of each n tile ----
template <int D, int NT>
struct State {
    uint32_t q[NT][D / 16][2];
    float f[NT][2];            // logit units: sm_scale log2(e) 2^k_exp, and the row's power of two
    int pos[NT][2];            // positions of the rows
    float m[NT][2], l[NT][2];  // m the same in every lane of a row; l this lane's part
    float acc[NT][D / 16][4];  // [channel g D/8 + 2 mi (+ 1: 2, 3)][row 2t (+ 1: 1, 3)]

    // what a logit loses before the exponential
    __device__ __forceinline__ float mu(int n, int e) const { return m[n][e] == -INFINITY ? 0.f : m[n][e] - LIFT; }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int n = 0; n < NT; n++) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; i++) acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.f;
        }
    }

    // Queries of rows row0 .. row0 + 8 NT of the unit's (token, head) rows: the loads first,
    // so that they are on their way while the first chunks are sent for.
    template <class A>
    __device__ __forceinline__ static void fetch_q(uint4 (&w)[NT][D / 32], const A &a, const PageRow &r, int head, int row0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; n++) {
            const int row = row0 + 8 * n + g, tok = row / a.p.G;
            const uint16_t *src = a.q + (static_cast<long long>(r.q0) + tok) * a.qt + (head * a.p.G + row - tok * a.p.G) * a.qh + t * (D / 4);
#pragma unroll
            for (int i = 0; i < D / 32; i++)
                w[n][i] = row < r.n * a.p.G ? *reinterpret_cast<const uint4 *>(src + 8 * i) : make_uint4(0, 0, 0, 0);
        }
    }
    template <class A>
    __device__ __forceinline__ void load_q(const uint4 (&w)[NT][D / 32], const A &a, const PageRow &r, int row0) {
        const int lane = threadIdx.x & 31, t = lane & 3;
        const int rows = r.n * a.p.G;
#pragma unroll
        for (int n = 0; n < NT; n++) {
            float x[D / 4], top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; i++) {
                const uint32_t u[4] = {w[n][i].x, w[n][i].y, w[n][i].z, w[n][i].w};
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
            // top < 2^(e + 1) -> scaled below 2^14
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
                const int other = __shfl_sync(FULL, up, 4 * (2 * t + e));
                const int rw = row0 + 8 * n + 2 * t + e;
                f[n][e] = a.scale_log2 * pow2i(-other);
                pos[n][e] = rw < rows ? first_sees(a, r) + rw / a.p.G * a.step : 0x7fffffff;  // no row: nothing to mask
            }
        }
    }

    // One chunk at `c`: tokens at positions pa .. pa + 15 and pb .. pb + 15 (negative: not there).
    __device__ __forceinline__ void step(const uint8_t *c, int pa, int pb, int len, int least) {
        using B = PageBlock<D>;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        float s[NT][8];  // tokens g, g + 8, g + 16, g + 24, rows 2t and 2t + 1 of each
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int i = 0; i < 8; i++) s[n][i] = 0.f;
        const uint8_t *kc = c + g * (D / 2) + t * (D / 8), *ks = c + B::ks(CHUNK) + g * (D / 16) + t * (D / 64);
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t ka[D / 32], kb[D / 32], sa[2], sb[2];
            ld_words(kc + h * 16 * (D / 2), ka);
            ld_words(kc + (h * 16 + 8) * (D / 2), kb);
            // scales of tokens g, g + 8: both halves of a register each
            const uint8_t *s0 = ks + h * D, *s1 = s0 + D / 2;
            const uint32_t two0 = e4m3x2_to_half2(D == 128 ? *reinterpret_cast<const uint16_t *>(s0) : *s0);
            const uint32_t two1 = e4m3x2_to_half2(D == 128 ? *reinterpret_cast<const uint16_t *>(s1) : *s1);
            sa[0] = __byte_perm(two0, two0, 0x1010);
            sb[0] = __byte_perm(two1, two1, 0x1010);
            sa[1] = D == 128 ? __byte_perm(two0, two0, 0x3232) : sa[0];
            sb[1] = D == 128 ? __byte_perm(two1, two1, 0x3232) : sb[0];
#pragma unroll
            for (int w = 0; w < D / 32; w++) {
                uint32_t a[4], b[4];
                e2m1x8_to_half(ka[w], a);
                e2m1x8_to_half(kb[w], b);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    a[i] = hmul2(a[i], sa[w >> 1]);
                    b[i] = hmul2(b[i], sb[w >> 1]);
                }
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    float(&d)[4] = *reinterpret_cast<float(*)[4]>(&s[n][4 * h]);
                    mma_f16(d, a[0], b[0], a[1], b[1], q[n][2 * w][0], q[n][2 * w][1]);
                    mma_f16(d, a[2], b[2], a[3], b[3], q[n][2 * w + 1][0], q[n][2 * w + 1][1]);
                }
            }
        }
        // exponents z - m + LIFT
        bool grow = false;
        const bool tail = pa < 0 || pb < 0 || pa + 15 > least || pb + 15 > least;  // a token that some row does not see
#pragma unroll
        for (int n = 0; n < NT; n++) {
#pragma unroll
            for (int i = 0; i < 8; i++) s[n][i] = fmaf(s[n][i], f[n][i & 1], -mu(n, i & 1));
            if (tail) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int at = i < 4 ? pa : pb;
                    if (at < 0 || at + g + 8 * ((i >> 1) & 1) > pos[n][i & 1]) s[n][i] = -INFINITY;
                }
            }
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float top = fmaxf(fmaxf(s[n][e], s[n][e + 2]), fmaxf(s[n][e + 4], s[n][e + 6]));
                grow |= top > (m[n][e] == -INFINITY ? -INFINITY : SLACK + LIFT);  // also the first finite logit
            }
        }
        if (__any_sync(FULL, grow)) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float top = fmaxf(fmaxf(s[n][e], s[n][e + 2]), fmaxf(s[n][e + 4], s[n][e + 6]));
                    top = fmaxf(top, __shfl_xor_sync(FULL, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(FULL, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(FULL, top, 16));
                    const float old = mu(n, e);
                    const float mx = fmaxf(top + old, m[n][e]);  // top is z - old
                    const float al = mx == -INFINITY ? 1.f : ex2(m[n][e] - mx);
                    m[n][e] = mx;
                    const float by = old - mu(n, e);
#pragma unroll
                    for (int i = e; i < 8; i += 2) s[n][i] += by;
                    l[n][e] *= al;
#pragma unroll
                    for (int i = 0; i < D / 16; i++) {
                        acc[n][i][e] *= al;
                        acc[n][i][e + 2] *= al;
                    }
                }
        }
        uint32_t p[NT][4];
#pragma unroll
        for (int n = 0; n < NT; n++) {
#pragma unroll
            for (int i = 0; i < 8; i++) s[n][i] = ex2(s[n][i]);
            l[n][0] += (s[n][0] + s[n][2]) + (s[n][4] + s[n][6]);
            l[n][1] += (s[n][1] + s[n][3]) + (s[n][5] + s[n][7]);
#pragma unroll
            for (int i = 0; i < 4; i++) p[n][i] = transpose8(half2_of(s[n][2 * i], s[n][2 * i + 1]));
        }
        const uint8_t *vc = c + B::vc(CHUNK) + ((D == 128 ? g : g >> 1) * 4 + t) * 16 + (D == 128 ? 0 : (g & 1) * 8);
        const uint8_t *vs = c + B::vs(CHUNK) + ((D == 128 ? g : g >> 1) * 4 + t) * 2;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t va[D / 32], vb[D / 32];
            ld_words(vc + (2 * h) * 4 * D, va);
            ld_words(vc + (2 * h + 1) * 4 * D, vb);
            uint32_t v0 = e4m3x2_to_half2(*reinterpret_cast<const uint16_t *>(vs + (2 * h) * (D / 2)));
            uint32_t v1 = e4m3x2_to_half2(*reinterpret_cast<const uint16_t *>(vs + (2 * h + 1) * (D / 2)));
            if (tail) {  // tokens that are not there may hold anything, NaN scales too: 0 . NaN must not count
                const int at = h ? pb : pa;
                const int n = at < 0 ? 0 : len - at;
                v0 &= (2 * t < n ? 0x0000ffffu : 0u) | (2 * t + 1 < n ? 0xffff0000u : 0u);
                v1 &= (2 * t + 8 < n ? 0x0000ffffu : 0u) | (2 * t + 9 < n ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int w = 0; w < D / 32; w++) {
                uint32_t a[4], b[4];
                e2m1x8_to_half(va[w], a);
                e2m1x8_to_half(vb[w], b);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    a[i] = hmul2(a[i], v0);
                    b[i] = hmul2(b[i], v1);
                }
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    mma_f16(acc[n][2 * w], a[0], a[1], b[0], b[1], p[n][2 * h], p[n][2 * h + 1]);
                    mma_f16(acc[n][2 * w + 1], a[2], a[3], b[2], b[3], p[n][2 * h], p[n][2 * h + 1]);
                }
            }
        }
    }

    // What the launch over the rows' own pages left for the unit's rows, beside this state.
    template <class A>
    __device__ __forceinline__ void take_in(const A &a, const PageRow &r, int head, int row0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int row = row0 + 8 * n + 2 * t + e;
                if (row >= r.n * a.p.G) continue;
                const long long o = query_of(a, r, head, row);
                const float2 ml = reinterpret_cast<const float2 *>(part_sums<D>(a))[o];
                if (ml.x == INFINITY) continue;  // (its output is 0)
                const float mx = fmaxf(m[n][e], ml.x), by = mx == -INFINITY ? 0.f : mx;
                const float keep = ex2(m[n][e] - by), take = ex2(ml.x - by);  // 0 for a part that saw nothing
                m[n][e] = mx;
                l[n][e] = l[n][e] * keep + (g == 0 ? ml.y * take : 0.f);
#pragma unroll
                for (int i = 0; i < D / 16; i++) {
                    const float2 x = *reinterpret_cast<const float2 *>(a.part + o * D + g * (D / 8) + 2 * i);
                    acc[n][i][e] = acc[n][i][e] * keep + x.x * take;
                    acc[n][i][e + 2] = acc[n][i][e + 2] * keep + x.y * take;
                }
            }
    }

    __device__ __forceinline__ void sum_l() {
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                l[n][e] += __shfl_xor_sync(FULL, l[n][e], 4);
                l[n][e] += __shfl_xor_sync(FULL, l[n][e], 8);
                l[n][e] += __shfl_xor_sync(FULL, l[n][e], 16);
            }
    }

    // A part of a unit: [8 NT][D] accumulators, then m, then l of each row.
    __device__ __forceinline__ void to_record(float *rec) {
        sum_l();
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int row = 8 * n + 2 * t + e;
#pragma unroll
                for (int i = 0; i < D / 16; i++)
                    *reinterpret_cast<float2 *>(rec + row * D + g * (D / 8) + 2 * i) = make_float2(acc[n][i][e], acc[n][i][e + 2]);
                if (g == 0) {
                    rec[8 * NT * D + row] = m[n][e];
                    rec[8 * NT * (D + 1) + row] = l[n][e];
                }
            }
    }

    // A whole unit: the rows' outputs.
    template <class A>
    __device__ __forceinline__ void to_output(const A &a, const PageRow &r, int head, int row0) {
        sum_l();
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int rows = r.n * a.p.G;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int row = row0 + 8 * n + 2 * t + e;
                if (row >= rows) continue;
                const long long o = query_of(a, r, head, row);
                if (a.mode == PAGES_OWN && r.from > 0) {
#pragma unroll
                    for (int i = 0; i < D / 16; i++)
                        *reinterpret_cast<float2 *>(a.part + o * D + g * (D / 8) + 2 * i) = make_float2(acc[n][i][e], acc[n][i][e + 2]);
                    if (g == 0) reinterpret_cast<float2 *>(part_sums<D>(a))[o] = make_float2(m[n][e], l[n][e]);
                    continue;
                }
                if (a.mode == PAGES_COMMON && reinterpret_cast<const float2 *>(part_sums<D>(a))[o].x == INFINITY) l[n][e] = 0.f;
                const float w = l[n][e] == 0.f ? 0.f : a.out_scale / l[n][e];
                uint32_t u[D / 16];
#pragma unroll
                for (int i = 0; i < D / 16; i++)
                    u[i] = pack2(to16(acc[n][i][e] * w, a.p.bf16), to16(acc[n][i][e + 2] * w, a.p.bf16));
                uint4 *dst = reinterpret_cast<uint4 *>(a.out + o * D + g * (D / 8));
#pragma unroll
                for (int i = 0; i < D / 64; i++) dst[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
                if (a.lse && g == 0) a.lse[o] = l[n][e] == 0.f ? -INFINITY : (m[n][e] - LIFT + log2f(l[n][e])) * LN2;
            }
    }
};

// ---- the call's units --------------------------------------------------------------------
// Units stand one after the other on a line, rows in order, KV heads, then query blocks
// within: UNIT_COST places for what a unit costs beside its chunks, then its chunks.
struct Unit {
    int i, head, row0;
    int first, chunks;  // place of its first chunk, and their number
};

template <int D, int NT, int NW>
struct Shared {
    static constexpr int REC = 8 * NT * (D + 2);   // floats of a record
    static constexpr int ST = 32 / NW;             // chunks of a warp's ring
    static constexpr int CB = CHUNK * D * 9 / 8;   // bytes of a chunk
    // each warp's ring, and its part of a unit begun before it; its part of a unit that
    // goes on after it takes the ring's place, which is done by then
    __align__(128) uint8_t ring[NW][ST][CB];
    __align__(16) float rec[NW][REC];
    uint64_t full[NW][ST];
    int2 pos[NW][ST];                  // positions of a chunk's two halves
    int first[DQ_PAGES_MAX_ROWS + 1];  // places before row i
    int row[DQ_PAGES_MAX_ROWS], keys[DQ_PAGES_MAX_ROWS];  // keys: tokens looked at
    long long part[NW];
    int unit[2 * NW];                  // the unit that each record is a part of, by its first chunk's place; -1: none
    int last[2];
    __device__ const float *record(int k) const { return k & 1 ? reinterpret_cast<const float *>(ring[k >> 1]) : rec[k >> 1]; }
    __device__ float *record(int k) { return k & 1 ? reinterpret_cast<float *>(ring[k >> 1]) : rec[k >> 1]; }
};

template <class A>
__device__ __forceinline__ int row_chunks(const A &a, int keys) {
    return (a.sel ? a.n_sel * a.p.P + CHUNK - 1 : keys + CHUNK - 1) / CHUNK;
}

// The unit at place x (the same for the whole warp).
template <int D, int NT, int NW, class A>
__device__ __forceinline__ Unit find_unit(const Shared<D, NT, NW> &sh, const A &a, int x) {
    // the last row that begins at or before x (rows without a place begin where the next one does)
    const int lane = threadIdx.x & 31, n = a.r.n_rows;
    int lo = 0;
    if (n > 32) lo = 32 * (__popc(__ballot_sync(FULL, 32 * lane < n && sh.first[32 * lane] <= x)) - 1);
    lo += __popc(__ballot_sync(FULL, lo + lane < n && sh.first[lo + lane] <= x)) - 1;
    Unit u;
    u.i = lo;
    u.chunks = row_chunks(a, sh.keys[lo]);
    const unsigned places = u.chunks + UNIT_COST, unit = static_cast<unsigned>(x - sh.first[lo]) / places;
    u.first = sh.first[lo] + unit * places + UNIT_COST;
    if (a.r.max_new * a.p.G <= 8 * NT) {
        u.head = unit;
        u.row0 = 0;
    } else {
        const unsigned blocks = static_cast<unsigned>(sh.first[lo + 1] - sh.first[lo]) / (places * a.p.Hkv);
        u.head = unit / blocks;
        u.row0 = (unit - u.head * blocks) * 8 * NT;
    }
    return u;
}

// Row i of the launch, which the prefix found to be in order.
template <int D, int NT, int NW, class A>
__device__ __forceinline__ PageRow known_row(const Shared<D, NT, NW> &sh, const A &a, int i) {
    return known_row(a, i, sh.row[i], sh.keys[i]);
}

// Share k of n places among m: [share(k), share(k + 1)).
__device__ __forceinline__ int share(int n, int m, int k) {
    const unsigned q = static_cast<unsigned>(n) / m, rest = n - q * m;
    return k * q + (k < static_cast<int>(rest) ? k : rest);
}
// The share that place x is in (m <= n).
__device__ __forceinline__ int share_of(int n, int m, int x) {
    const unsigned q = static_cast<unsigned>(n) / m, rest = n - q * m, ahead = rest * (q + 1);
    return static_cast<unsigned>(x) < ahead ? x / (q + 1) : rest + (x - ahead) / q;
}

// Four channels of a part beside those of others.
__device__ __forceinline__ void join(float (&acc)[4], float &m, float &l, float mk, float lk, float4 x) {
    const float mx = fmaxf(m, mk), mu = mx == -INFINITY ? 0.f : mx;
    const float wa = ex2(m - mu), wb = ex2(mk - mu);  // 0 for a part that saw nothing
    m = mx;
    l = l * wa + lk * wb;
    acc[0] = acc[0] * wa + x.x * wb;
    acc[1] = acc[1] * wa + x.y * wb;
    acc[2] = acc[2] * wa + x.z * wb;
    acc[3] = acc[3] * wa + x.w * wb;
}

// One thread's 4 channels at c of row `row` over n records, added up in order.
template <int D, int NT, class F>
__device__ __forceinline__ void add_records(int n, int row, int c, F rec_of, float (&acc)[4], float &m, float &l) {
    m = -INFINITY;
    l = 0.f;
    acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll 4
    for (int k = 0; k < n; k++) {
        const float *r = rec_of(k);
        const float mk = r[8 * NT * D + row], lk = r[8 * NT * (D + 1) + row];
        join(acc, m, l, mk, lk, *reinterpret_cast<const float4 *>(r + row * D + c));
    }
}

template <int D, class A>
__device__ __forceinline__ void write4(const A &a, const PageRow &r, int head, int row, int c, float (&acc)[4], float m, float l) {
    if (row >= r.n * a.p.G) return;
    const long long o = query_of(a, r, head, row);
    if (a.mode == PAGES_OWN && r.from > 0) {
        *reinterpret_cast<float4 *>(a.part + o * D + c) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (c == 0) reinterpret_cast<float2 *>(part_sums<D>(a))[o] = make_float2(m, l);
        return;
    }
    if (a.mode == PAGES_COMMON) {  // what the launch over the rows' own pages left
        const float2 own = reinterpret_cast<const float2 *>(part_sums<D>(a))[o];
        const float4 x = *reinterpret_cast<const float4 *>(a.part + o * D + c);
        if (own.x == INFINITY) l = 0.f;
        else join(acc, m, l, own.x, own.y, x);
    }
    const float w = l == 0.f ? 0.f : a.out_scale / l;
    *reinterpret_cast<uint2 *>(a.out + o * D + c) =
        make_uint2(pack2(to16(acc[0] * w, a.p.bf16), to16(acc[1] * w, a.p.bf16)), pack2(to16(acc[2] * w, a.p.bf16), to16(acc[3] * w, a.p.bf16)));
    if (a.lse && c == 0) a.lse[o] = l == 0.f ? -INFINITY : (m - LIFT + log2f(l)) * LN2;
}

template <int D, int NT, int NW, bool TWO, int MODE>
__global__ void __launch_bounds__(32 * NW, 1) attn_chunks(const InMode<MODE> a) {
    extern __shared__ __align__(128) uint8_t raw[];
    using S = Shared<D, NT, NW>;
    S &sh = *reinterpret_cast<S *>(raw);
    const PagesView &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int ST = S::ST;
    if (a.mode == PAGES_OWN) let_next_start();
    int *tickets = a.mode == PAGES_OWN ? a.own_tickets : a.tickets;
    float *records = a.mode == PAGES_OWN ? a.own_records : a.records;
    if (lane < ST) mbar_init(&sh.full[warp][lane], 1 + a.owed);
    fence_mbar_init();
    const long long own = own_places<32 * NW>(a);
    // places before each row: a prefix over the rows, 32 NW at a time
    long long base = 0;
    for (int i0 = 0; i0 < a.r.n_rows; i0 += 32 * NW) {
        const int i = i0 + tid;
        long long w = 0;
        if (i < a.r.n_rows) {
            const PageRow r = attn_row(a, i);
            sh.row[i] = r.row;
            sh.keys[i] = r.len - r.from;
            if (r.len > 0 && takes(a, r))
                w = static_cast<long long>((r.n * p.G + 8 * NT - 1) / (8 * NT)) * p.Hkv * (row_chunks(a, r.len - r.from) + UNIT_COST);
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
#pragma unroll
        for (int k = 0; k < NW; k++) {
            const long long t = sh.part[k];
            if (k < warp) before += t;
            base += t;
        }
        if (i < a.r.n_rows) sh.first[i] = static_cast<int>(before + s - w);
        if (i0 + 32 * NW < a.r.n_rows) __syncthreads();
    }
    if (base > 0x7fffffff) {  // more places than int counts
        if (tid == 0) atomicOr(p.status, PST_ARG);
        if (a.mode == PAGES_COMMON) await_previous();
        return;
    }
    const int N = static_cast<int>(base);
    if (tid == 0) sh.first[a.r.n_rows] = N;
    if (tid < 2 * NW) sh.unit[tid] = -1;
    __syncthreads();
    // rows that hold nothing: zeros
    for (int i = blockIdx.x; i < a.r.n_rows && a.mode != PAGES_COMMON; i += gridDim.x) {
        if (sh.keys[i] > 0) continue;
        const PageRow r = page_row(p, a.r, i);
        if (!takes(a, r)) continue;
        uint4 *o = reinterpret_cast<uint4 *>(a.out + static_cast<long long>(r.q0) * p.Hq * D);
        for (long long k = tid; k < static_cast<long long>(r.n) * p.Hq * (D / 8); k += 32 * NW) o[k] = make_uint4(0, 0, 0, 0);
        if (a.mode == PAGES_OWN && a.plan[2 * i] > 0)
            for (long long k = tid; k < static_cast<long long>(r.n) * p.Hq; k += 32 * NW)
                reinterpret_cast<float2 *>(part_sums<D>(a))[static_cast<long long>(r.q0) * p.Hq + k] = make_float2(INFINITY, 0.f);
        if (a.lse)
            for (long long k = tid; k < static_cast<long long>(r.n) * p.Hq; k += 32 * NW) a.lse[static_cast<long long>(r.q0) * p.Hq + k] = -INFINITY;
    }
    // this CTA's places [c0, c1), this warp's [w0, w1)
    // (the compiler's schedule of the loop below hangs on this: with one bound for all kinds of launch 8 rows of 4 to 8 tokens
    // over 32768 take 5 % longer)
    int ctas = N / MIN_PLACES;
    ctas = ctas < 1 ? 1 : (ctas > static_cast<int>(gridDim.x) ? gridDim.x : ctas);
    if (a.mode == PAGES_OWN || a.mode == PAGES_COMMON) {
        int room = a.mode == PAGES_OWN ? own_ctas(N, gridDim.x) : sms_left<32 * NW>(a, own, sh.part);
        if (a.mode == PAGES_OWN) {
            // nothing in common: all SMs (16 rows of 1364 tokens 21.4 -> 16.8 us, 32 of 664 22.4 -> 17.0).  Each warp looks for
            // itself: with a barrier's vote the loop below spills (64 rows of 8256 113 -> 115)
            bool shares = false;
            for (int i = lane; i < a.r.n_rows; i += 32) shares |= a.plan[2 * i] > 0;
            if (!__any_sync(FULL, shares)) room = gridDim.x;
        }
        ctas = ctas > room ? room : ctas;
    }
    if (N == 0 || static_cast<int>(blockIdx.x) >= ctas) {
        if (a.mode == PAGES_COMMON) await_previous();
        return;
    }
    // (a border inside a short unit goes to its beginning: the wait for the longer share is less than the 4 us
    // that CTAs take to join a unit; up to 128 places where that share is not much over the others.  16 rows of
    // 1024 tokens 14.9 -> 11.9 us, of 2048 19.0 -> 16.0)
    auto border = [&](int k) {
        const int x = share(N, ctas, k);
        if (x <= 0 || x >= N) return x;
        const Unit u = find_unit<D, NT, NW>(sh, a, x);
        const int places = u.chunks + UNIT_COST;
        constexpr int SHORT = MODE == PAGES_COMMON ? SHORT_COMMON : SHORT_ROWS;
        return places <= SHORT || (places <= 2 * SHORT && 4LL * places * ctas <= 5LL * N) ? u.first - UNIT_COST : x;
    };
    const int c0 = border(blockIdx.x), c1 = border(blockIdx.x + 1);
    const int w0 = c0 + share(c1 - c0, NW, warp), w1 = c0 + share(c1 - c0, NW, warp + 1);

    // chunks of a page, a power of two (TWO: 2 pages of 16 tokens make a chunk)
    const int shift = TWO ? 0 : 31 - __clz(p.P / CHUNK), mask = (1 << shift) - 1;
    // what this lane copies: part 0 .. 3 (of the second page in lanes 4 .. 7) of `bytes` bytes
    using B = PageBlock<D>;
    constexpr int HB = 16 * D * 9 / 8;
    const int b = TWO ? 16 : p.blk, part = lane & 3, half = TWO ? lane >> 2 & 1 : 0;
    const int line = part & 1 ? D / 16 : D / 2;  // bytes of a token
    const unsigned bytes = (TWO ? 16 : CHUNK) * line;
    const int from = part == 0 ? 0 : (part == 1 ? B::ks(b) : (part == 2 ? B::vc(b) : B::vs(b)));
    const int to = (part == 0 ? 0 : (part == 1 ? B::ks(CHUNK) : (part == 2 ? B::vc(CHUNK) : B::vs(CHUNK)))) + half * 16 * line;
    const unsigned page_stride = static_cast<unsigned>(p.Hkv) * p.page_bytes;
    const uint32_t ring = smem_u32(sh.ring[warp][0]), lane_to = ring + to, bars = smem_u32(sh.full[warp]);
    State<D, NT> st;
    unsigned sent = 0, done = 0;  // chunks of this warp's ring
    // After a wait that ran out this warp waits for no copy more, but it goes through its units, leaves its
    // parts and has them counted, so that the workspace is as every other call leaves it; the status says
    // that the outputs are not valid.
    bool late = false;
    for (int x = w0; x < w1;) {
        const Unit u = find_unit<D, NT, NW>(sh, a, x);
        const int t0 = x > u.first ? x - u.first : 0;
        const int t1 = u.first + u.chunks < w1 ? u.chunks : w1 - u.first;
        x = u.first + u.chunks;
        if (t1 <= t0) continue;  // none of its chunks
        const PageRow r = known_row<D, NT, NW>(sh, a, u.i);
        // the rows' least and greatest position: tokens past the greatest are nobody's
        const int rows = r.n * p.G;
        const int end = u.row0 + 8 * NT < rows ? u.row0 + 8 * NT : rows;
        const int least = first_sees(a, r) + u.row0 / p.G * a.step, most = first_sees(a, r) + (end - 1) / p.G * a.step;
        uint4 qw[NT][D / 32];
        st.fetch_q(qw, a, r, u.head, u.row0);
        // page numbers of 32 entries at a time, one a lane, the next 32 on their way
        const int first_page = r.from / p.P;
        const int *sel = a.sel ? a.sel + (static_cast<long long>(u.i) * p.Hkv + u.head) * a.n_sel : nullptr;
        auto entry = [&](int e, int &id, int &at) {  // at: position of the page's first token, -1: no page
            id = at = -1;
            int ord = e + first_page;
            if (sel) ord = e < a.n_sel ? sel[e] : -1;
            if (r.row < 0 || ord < 0 || ord >= p.M || ord * p.P >= r.len) return;
            at = ord * p.P;
            id = p.table[static_cast<long long>(r.row) * p.M + ord];
        };
        auto checked = [&](int id, int at) {
            if (at < 0 || (id >= 0 && id < p.n_pages)) return id;
            atomicOr(p.status, PST_TABLE);
            return -1;
        };
        int e0 = TWO ? 2 * t0 : t0 >> shift, id0, at0, id1, at1;
        entry(e0 + lane, id0, at0);
        entry(e0 + 32 + lane, id1, at1);
        id0 = checked(id0, at0);
        int next = t0;
        const uint8_t *lane_from = p.pages + static_cast<long long>(u.head) * p.page_bytes + from;
        // copy the next chunk that holds something into the ring
        auto send = [&]() {
            while (next < t1 && !late) {
                const int c = next++;
                int e = (TWO ? 2 * c : c >> shift) - e0;
                if (e >= 32) {
                    e -= 32;
                    e0 += 32;
                    id0 = checked(id1, at1);
                    at0 = at1;
                    entry(e0 + 32 + lane, id1, at1);
                }
                const unsigned k = sent % ST;
                const uint32_t bar = bars + 8 * k, dst = lane_to + k * S::CB;
                if (TWO) {
                    const int ia = __shfl_sync(FULL, id0, e), ib = __shfl_sync(FULL, id0, e + 1);
                    int pa = __shfl_sync(FULL, at0, e), pb = __shfl_sync(FULL, at0, e + 1);
                    if (ia < 0 || pa > most) pa = -1;
                    if (ib < 0 || pb > most) pb = -1;
                    if ((pa & pb) < 0) continue;
                    if (lane == 0) {
                        sh.pos[warp][k] = make_int2(pa, pb);
                        mbar_expect(bar, (pa < 0 ? 0 : HB) + (pb < 0 ? 0 : HB));
                    }
                    __syncwarp();
                    if (lane < 8 && (half ? pb : pa) >= 0)
                        bulk_copy(dst, lane_from + static_cast<unsigned long long>(half ? ib : ia) * page_stride, bytes, bar);
                } else {
                    const int id = __shfl_sync(FULL, id0, e), j = c & mask, pa = __shfl_sync(FULL, at0, e) + j * CHUNK;
                    if (id < 0 || pa > most) continue;
                    if (lane == 0) {
                        sh.pos[warp][k] = make_int2(pa, pa + 16 > most ? -1 : pa + 16);
                        mbar_expect(bar, 2 * HB);
                    }
                    __syncwarp();
                    if (lane < 4)
                        bulk_copy(dst, lane_from + static_cast<unsigned long long>(id) * page_stride + ((j >> 1) * B::size(64) + (j & 1) * CHUNK * line),
                                  bytes, bar);
                }
                sent++;
                return;
            }
        };
#pragma unroll
        for (int k = 0; k < ST; k++) send();
        st.load_q(qw, a, r, u.row0);
        st.reset();
        while (done != sent) {
            const int k = done % ST;
            if (!__all_sync(FULL, mbar_wait(&sh.full[warp][k], done / ST & 1, a.wait_ns))) {
                if (lane == 0) atomicOr(p.status, PST_TIMEOUT);
                late = true;
                while (++done != sent) mbar_wait(&sh.full[warp][done % ST], done / ST & 1, a.wait_ns);  // what is in flight has its limit too
                __syncwarp();
                break;
            }
            const int2 at = sh.pos[warp][k];
            st.step(sh.ring[warp][k], at.x, at.y, r.len, least);
            done++;
            __syncwarp();
            send();
        }
        if (a.mode == PAGES_COMMON && t0 == 0 && t1 == u.chunks) {
            await_previous();
            st.take_in(a, r, u.head, u.row0);
        }
        if (t0 == 0 && t1 == u.chunks) st.to_output(a, r, u.head, u.row0);
        else {
            __syncwarp();
            st.to_record(sh.record(2 * warp + (t0 == 0)));
            if (lane == 0) sh.unit[2 * warp + (t0 == 0)] = u.first;
        }
    }
    if (a.mode == PAGES_COMMON) await_previous();
    __syncthreads();

    // The records that warps left, in order: a unit's are neighbours (a run), the first of
    // them odd where the unit begins in its warp, then one for each warp.  Groups of
    // warps take the runs in turn: a unit that is all here is written, a part of one goes
    // to the workspace (at most two: of the unit that began before this CTA, and of the
    // one that goes on after it).
    constexpr int REC = S::REC, ITEMS = 8 * NT * (D / 4);
    constexpr int GROUPS = 32 * NW > ITEMS ? 32 * NW / ITEMS : 1, TH = 32 * NW / GROUPS;
    const int mine_is = lane < 2 * NW ? sh.unit[lane] : -1;
    int front = -1, back = -1, turn = 0;
    for (unsigned left = __ballot_sync(FULL, mine_is >= 0); left; turn++) {
        const int k0 = __ffs(left) - 1, first = __shfl_sync(FULL, mine_is, k0);
        const unsigned run = __ballot_sync(FULL, mine_is == first);
        left &= ~run;
        const Unit u = find_unit<D, NT, NW>(sh, a, first);
        const bool begins = first >= c0, ends = first + u.chunks <= c1;
        if (!begins) front = first;
        else if (!ends) back = first;
        if (turn % GROUPS != tid / TH) continue;
        const PageRow r = known_row<D, NT, NW>(sh, a, u.i);
        const int n = __popc(run), even = (k0 + 1) & ~1, odd = k0 & 1;
        auto part_of = [&](int k) -> const float * { return k < odd ? sh.record(k0) : sh.rec[(even >> 1) + k - odd]; };
        float *to = records + (2LL * blockIdx.x + begins) * REC;
        for (int i = tid % TH; i < ITEMS; i += TH) {
            float acc[4], m, l;
            const int row = i / (D / 4), c = i % (D / 4) * 4;
            add_records<D, NT>(n, row, c, part_of, acc, m, l);
            if (begins && ends) {
                write4<D>(a, r, u.head, u.row0 + row, c, acc, m, l);
            } else {
                *reinterpret_cast<float4 *>(to + row * D + c) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                if (c == 0) {
                    to[8 * NT * D + row] = m;
                    to[8 * NT * (D + 1) + row] = l;
                }
            }
        }
    }
    if (front < 0 && back < 0) return;
    // The last of a unit's CTAs to bring its part adds all parts up.  The count releases the
    // block's writes (which the barrier put before it) and acquires the others'.
    __syncthreads();
    if (warp < 2) {
        const int first = warp == 0 ? front : back;
        int all = 0;
        if (first >= 0) {
            const Unit u = find_unit<D, NT, NW>(sh, a, first);
            const int cf = share_of(N, ctas, first), others = share_of(N, ctas, first + u.chunks - 1) - cf;
            if (lane == 0) {
                all = atomic_add_acq_rel_gpu(tickets + cf, 1) == others;
                if (all) tickets[cf] = 0;  // for the next call
            }
        }
        if (lane == 0) sh.last[warp] = all;
    }
    __syncthreads();
#pragma unroll 1
    for (int s = 0; s < 2; s++) {
        if (!sh.last[s]) continue;
        const int first = s == 0 ? front : back;
        const Unit u = find_unit<D, NT, NW>(sh, a, first);
        const PageRow r = known_row<D, NT, NW>(sh, a, u.i);
        const int cf = share_of(N, ctas, first), n = share_of(N, ctas, first + u.chunks - 1) - cf + 1;
        auto cta_of = [&](int k) -> const float * { return records + (2LL * (cf + k) + (k == 0)) * REC; };
        for (int i = tid; i < ITEMS; i += 32 * NW) {
            float acc[4], m, l;
            const int row = i / (D / 4), c = i % (D / 4) * 4;
            add_records<D, NT>(n, row, c, cta_of, acc, m, l);
            write4<D>(a, r, u.head, u.row0 + row, c, acc, m, l);
        }
    }
}

template <int D, int NT, int NW, bool TWO, int MODE>
int launch_as(const PagesAttnArgs &a, int grid, cudaStream_t st) {
    const int smem = static_cast<int>(sizeof(Shared<D, NT, NW>));
    if (const int e = allow_shared<attn_chunks<D, NT, NW, TWO, MODE>>(smem)) return e;
    if (MODE == PAGES_COMMON && a.after_few) return launch_overlapping(attn_chunks<D, NT, NW, TWO, MODE>, dim3(grid), 32 * NW, smem, st, InMode<MODE>{a});
    attn_chunks<D, NT, NW, TWO, MODE><<<grid, 32 * NW, smem, st>>>(InMode<MODE>{a});
    return static_cast<int>(cudaGetLastError());
}
template <int D, int NT, int NW, int MODE>
int launch_chunks(const PagesAttnArgs &a, int grid, cudaStream_t st) {
    return a.p.P < CHUNK ? launch_as<D, NT, NW, true, MODE>(a, grid, st) : launch_as<D, NT, NW, false, MODE>(a, grid, st);
}
// 8 query rows fill one n tile; more share the conversions of two, with fewer warps for their
// registers (8 x 4 tokens over 32768 at head_dim 64: 69 us with 8 warps, 59 with 12; the
// same 86 with either at 128, where mma.sync itself is the limit)
template <int MODE>
int launch_few(const PagesAttnArgs &a, int grid, void *stream) {
    auto st = static_cast<cudaStream_t>(stream);
    if (a.r.max_new * a.p.G <= 8) return a.p.d == 128 ? launch_chunks<128, 1, 16, MODE>(a, grid, st) : launch_chunks<64, 1, 16, MODE>(a, grid, st);
    return a.p.d == 128 ? launch_chunks<128, 2, 8, MODE>(a, grid, st) : launch_chunks<64, 2, 12, MODE>(a, grid, st);
}

}  // namespace
}  // namespace dq
