// Paged cache: new tokens into pages (append) and back to 16 bits (read).
//
// A scale block is 16 channels of one token: top = max|x|, s = e4m3(top / 6 / 2^exp),
// codes e2m1(x / (2^exp s)).  The quotient is IEEE-rounded: for 16-bit x no quotient
// lies within half an fp32 step of a rounding border without being on it, so that
// the codes are those of exact arithmetic.
#include <cuda_runtime.h>

#include "pages.cuh"

namespace dq {
namespace {

constexpr int ST_THREADS = 128;

// 16 values at x (a block of one token) -> 8 bytes of code pairs (channel order) and
// the scale.  Returns false if a value is not finite.
__device__ __forceinline__ bool quantise16(const uint16_t *x, bool bf16, float inv_unit, float unit, uint32_t (&code)[2],
                                           uint8_t &scale) {
    const uint4 a = *reinterpret_cast<const uint4 *>(x), b = *reinterpret_cast<const uint4 *>(x + 8);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float f[16], top = 0.f, nan = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        f[2 * i] = from16(static_cast<uint16_t>(w[i] & 0xffffu), bf16);
        f[2 * i + 1] = from16(static_cast<uint16_t>(w[i] >> 16), bf16);
    }
#pragma unroll
    for (int i = 0; i < 16; i++) {
        top = fmaxf(top, fabsf(f[i]));
        nan += f[i] * 0.f;
    }
    float S;
    scale = block_scale(top, inv_unit, unit, S);
    code[0] = code[1] = 0;
    if (S > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            code[i >> 2] |= float2_to_e2m1(__fdiv_rn(f[2 * i], S), __fdiv_rn(f[2 * i + 1], S)) << (8 * (i & 3));
    } else {  // every code 0, signs kept
#pragma unroll
        for (int i = 0; i < 16; i++) code[i >> 3] |= (__float_as_uint(f[i]) >> 31) << (4 * (i & 7) + 3);
    }
    return nan == 0.f;
}

// One CTA per (row, touched page, KV head): the page's bytes come to shared memory,
// the new tokens' codes go in, the summary is taken over all tokens, and the bytes go
// back.  The page is one row's alone, so no other CTA writes it.
template <int D>
__global__ void __launch_bounds__(ST_THREADS) append_kernel(PagesStoreArgs a) {
    extern __shared__ __align__(16) uint8_t img[];
    __shared__ float red[ST_THREADS / 32];
    const PagesView &p = a.p;
    const PageRow r = page_row(p, a.r, blockIdx.y);
    const int head = blockIdx.z, tid = threadIdx.x;
    const int lo = r.len - r.n < 0 ? 0 : r.len - r.n;  // first position written
    const int j = lo / p.P + blockIdx.x;
    if (r.row < 0 || r.n == 0 || j * p.P >= r.len) return;
    const int id = page_of(p, r.row, j);
    if (id < 0) return;
    if (p.refs[id] != 1) {
        if (tid == 0) atomicOr(p.status, PST_SHARED);
        return;
    }
    using B = PageBlock<D>;
    uint4 *page = reinterpret_cast<uint4 *>(page_ptr(p, id, head));
    for (int i = tid; i < p.page_bytes / 16; i += ST_THREADS) reinterpret_cast<uint4 *>(img)[i] = page[i];
    __syncthreads();
    const int t0 = lo > j * p.P ? lo - j * p.P : 0;                        // new tokens of the page: [t0, t1)
    const int t1 = r.len - j * p.P < p.P ? r.len - j * p.P : p.P;
    const long long first = r.q0 + (static_cast<long long>(j) * p.P - (r.len - r.n));  // the call's token at t = 0
    const float ku = pow2i(p.k_exp), ki = pow2i(-p.k_exp), vu = pow2i(p.v_exp), vi = pow2i(-p.v_exp);
    bool fine = true;
    // keys: a thread takes a (token, scale block)
    for (int i = tid; i < (t1 - t0) * (D / 16); i += ST_THREADS) {
        const int t = t0 + i / (D / 16), c = i % (D / 16);
        uint8_t *blk = img + (t / p.blk) * B::size(p.blk);
        uint32_t code[2];
        uint8_t s;
        fine &= quantise16(a.k + (first + t) * a.kt + head * a.kh + 16 * c, p.bf16, ki, ku, code, s);
        *reinterpret_cast<uint2 *>(blk + (t % p.blk) * (D / 2) + 8 * c) = make_uint2(code[0], code[1]);
        blk[B::ks(p.blk) + (t % p.blk) * (D / 16) + c] = s;
    }
    // values: a thread takes a (token pair, scale block) and puts the new tokens' halves in
    for (int i = tid; i < ((t1 + 1) / 2 - t0 / 2) * (D / 16); i += ST_THREADS) {
        const int t = 2 * (t0 / 2 + i / (D / 16)), c = i % (D / 16);
        uint8_t *blk = img + (t / p.blk) * B::size(p.blk);
        uint8_t *cp = blk + B::vc(p.blk) + B::vcode(t % p.blk, c), *sp = blk + B::vs(p.blk) + B::vscale(t % p.blk, c);
        for (int e = 0; e < 2; e++) {
            if (t + e < t0 || t + e >= t1) continue;
            uint32_t code[2];
            uint8_t s;
            fine &= quantise16(a.v + (first + t + e) * a.vt + head * a.vh + 16 * c, p.bf16, vi, vu, code, s);
            sp[e] = s;
            for (int ch = 0; ch < 16; ch++) {
                const uint32_t m = (code[ch >> 3] >> (4 * (ch & 7))) & 15u;
                cp[ch] = static_cast<uint8_t>(e ? ((cp[ch] & 0x0fu) | (m << 4)) : ((cp[ch] & 0xf0u) | m));
            }
        }
    }
    if (!fine) atomicOr(p.status, PST_NONFINITE);
    __syncthreads();
    for (int i = tid; i < p.page_bytes / 16; i += ST_THREADS) page[i] = reinterpret_cast<uint4 *>(img)[i];
    // summary: thread c takes channel c over tokens [0, t1)
    float mx = -INFINITY, mn = INFINITY;
    if (tid < D) {
        for (int t = 0; t < t1; t++) {
            const uint8_t *blk = img + (t / p.blk) * B::size(p.blk);
            const uint32_t byte = blk[(t % p.blk) * (D / 2) + (tid >> 1)];
            const float x = e2m1_to_float((byte >> (4 * (tid & 1))) & 15u) *
                            e4m3_to_float(blk[B::ks(p.blk) + (t % p.blk) * (D / 16) + (tid >> 4)]);
            mx = fmaxf(mx, x);
            mn = fminf(mn, x);
        }
    }
    const float w = warp_max(tid < D ? fmaxf(fabsf(mx), fabsf(mn)) : 0.f);
    if ((tid & 31) == 0) red[tid >> 5] = w;
    __syncthreads();
    float top = red[0];
    for (int i = 1; i < ST_THREADS / 32; i++) top = fmaxf(top, red[i]);
    // held keys are multiples of 2^-10 below 2^12: top = m 2^E with E from the exponent field
    const int e = top > 0.f ? static_cast<int>(__float_as_uint(top) >> 23) - 126 - 7 : 0;
    uint8_t *sum = summary_ptr(p, id, head);
    if (tid < D) {
        const float unit = pow2i(-e);
        reinterpret_cast<int8_t *>(sum)[tid] = static_cast<int8_t>(ceilf(mx * unit));
        reinterpret_cast<int8_t *>(sum)[D + tid] = static_cast<int8_t>(floorf(mn * unit));
    }
    if (tid == 0) *reinterpret_cast<int *>(sum + 2 * D) = e;
}

// One thread per (token, KV head, scale block).
template <int D>
__global__ void __launch_bounds__(256) read_kernel(PagesReadArgs a) {
    const PagesView &p = a.p;
    const PageRow r = page_row(p, a.r, blockIdx.y);
    const int per = p.Hkv * (D / 16);
    using B = PageBlock<D>;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < static_cast<long long>(r.n) * per; i += gridDim.x * 256LL) {
        const int n = static_cast<int>(i / per), u = static_cast<int>(i % per), head = u / (D / 16), c = u % (D / 16);
        const int pos = r.len - r.n + n;
        uint16_t *ko = a.k + ((static_cast<long long>(r.q0) + n) * p.Hkv + head) * D + 16 * c;
        uint16_t *vo = a.v + ((static_cast<long long>(r.q0) + n) * p.Hkv + head) * D + 16 * c;
        const int id = pos >= 0 && r.row >= 0 ? page_of(p, r.row, pos / p.P) : -1;
        float kx[16], vx[16];
#pragma unroll
        for (int ch = 0; ch < 16; ch++) kx[ch] = vx[ch] = 0.f;
        if (id >= 0) {
            const int t = pos % p.P, tb = t % p.blk;
            const uint8_t *blk = page_ptr(p, id, head) + (t / p.blk) * B::size(p.blk);
            const float ks = e4m3_to_float(blk[B::ks(p.blk) + tb * (D / 16) + c]) * pow2i(p.k_exp);
            const float vs = e4m3_to_float(blk[B::vs(p.blk) + B::vscale(tb, c)]) * pow2i(p.v_exp);
            const uint8_t *kc = blk + tb * (D / 2) + 8 * c, *vc = blk + B::vc(p.blk) + B::vcode(tb, c);
#pragma unroll
            for (int ch = 0; ch < 16; ch++) {
                kx[ch] = e2m1_to_float((kc[ch >> 1] >> (4 * (ch & 1))) & 15u) * ks;
                vx[ch] = e2m1_to_float((vc[ch] >> (4 * (t & 1))) & 15u) * vs;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
            uint32_t kw[4], vw[4];
#pragma unroll
            for (int i4 = 0; i4 < 4; i4++) {
                kw[i4] = pack2(to16(kx[8 * h + 2 * i4], p.bf16), to16(kx[8 * h + 2 * i4 + 1], p.bf16));
                vw[i4] = pack2(to16(vx[8 * h + 2 * i4], p.bf16), to16(vx[8 * h + 2 * i4 + 1], p.bf16));
            }
            reinterpret_cast<uint4 *>(ko)[h] = make_uint4(kw[0], kw[1], kw[2], kw[3]);
            reinterpret_cast<uint4 *>(vo)[h] = make_uint4(vw[0], vw[1], vw[2], vw[3]);
        }
    }
}

}  // namespace

int launch_pages_append(const PagesStoreArgs &a, void *stream) {
    // a row's new tokens touch at most this many pages
    const int most = (a.r.max_new + a.p.P - 2) / a.p.P + 1;
    const dim3 grid(most < a.p.M ? most : a.p.M, a.r.n_rows, a.p.Hkv);
    auto st = static_cast<cudaStream_t>(stream);
    if (a.p.d == 128) append_kernel<128><<<grid, ST_THREADS, a.p.page_bytes, st>>>(a);
    else append_kernel<64><<<grid, ST_THREADS, a.p.page_bytes, st>>>(a);
    return static_cast<int>(cudaGetLastError());
}

int launch_pages_read(const PagesReadArgs &a, void *stream) {
    const long long per = static_cast<long long>(a.r.max_new) * a.p.Hkv * (a.p.d / 16);
    const long long want = (per + 255) / 256;
    const dim3 grid(static_cast<unsigned>(want < 4096 ? want : 4096), a.r.n_rows);
    auto st = static_cast<cudaStream_t>(stream);
    if (a.p.d == 128) read_kernel<128><<<grid, 256, 0, st>>>(a);
    else read_kernel<64><<<grid, 256, 0, st>>>(a);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace dq
