// paged_cache.cu -- writing K and V rows into the pages of a cache and reading them back.
//
// A bf16 cache holds the rows as they come.  An e4m3 cache holds, per row x of d elements,
//     s = 2^e,  e = max(-120, the least e with max|x| <= 448 * 2^e),   code = e4m3(x / s)
// (448 is the largest e4m3 number; round to nearest even).  A power of two costs nothing
// against an arbitrary scale, because the format is a floating-point one, and makes both
// directions exact: x / s and code * s are products with a power of two, and code * s has 4
// significant bits and an exponent that bf16 has (2^-129 at least), so that reading back
// rounds nothing.  e comes from the bits of max|x|: no logarithm, no division.
// A row with an infinity or a NaN has no scale: it is stored as zeros with the scale NaN,
// which every reader turns into a row of NaN.
//
// Both kernels move d / 8 threads a row, 8 elements (16 bytes of bf16) a thread, K and V in one
// thread, and are bound by HBM once there is enough to move.  The place of a token hangs on four
// loads one after the other (its sequence, that one's rows and length, the page), so:
//   * small calls: a thread a piece, which finds its place itself while its rows are on their
//     way; a decoding step of 64 tokens (8 heads, d = 128, e4m3) takes 2.8 us, 17.5k tokens of d = 64
//     13.8 us (5.2 TB/s); with a block's shared list of places 3.9 and 17 us.
//   * large calls (more than eight waves of full SMs): a block finds the places of its tokens
//     once, in shared memory, and every thread moves four pieces with all loads in flight: 32k
//     tokens into e4m3 37 us (5.5 TB/s; a piece a thread 45 us), 131072 out of it 127 us
//     (6.4 TB/s; 143 us).
#include <cuda_bf16.h>

#include "paged.h"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kCuShared = 1024;  // batches up to this keep cu in shared memory for the searches
constexpr int kMaxTokens = 64;   // of a block

__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Data read once: not kept in L1.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 x;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
    return x;
}
__device__ __forceinline__ uint2 ld_stream(const uint2* p) {
    uint2 x;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
    return x;
}

// Largest |x| of 8 bf16 each of a K and a V row held by LPR neighbouring lanes: K's in the low half, V's in
// the high one, so that one chain of shuffles does for both (32k tokens 38.0 us with two, 37.1 so).  (|x| orders like the bits without the sign.)
template <int LPR>
__device__ __forceinline__ uint32_t row_maxima(uint4 k, uint4 v) {
    const uint32_t a = __vmaxu2(__vmaxu2(k.x & 0x7fff7fffu, k.y & 0x7fff7fffu), __vmaxu2(k.z & 0x7fff7fffu, k.w & 0x7fff7fffu));
    const uint32_t b = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    uint32_t m = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
    for (int o = 1; o < LPR; o *= 2) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// 8 bf16 of a row whose largest |x| has the bits m -> their codes and the row's scale.
__device__ __forceinline__ uint2 quantise8(uint4 x, uint32_t m, float& scale) {
    if (m >= 0x7f80u) {
        scale = __uint_as_float(0x7fc00000u);
        return make_uint2(0u, 0u);
    }
    // max|x| = 1.f * 2^(E - 127) <= 1.75 * 2^(8 + e)
    int e = static_cast<int>(m >> 7) - 127 - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0);
    e = max(e, -120);
    scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint2 r;
    r.x = cvt_e4m3x2(bf_lo(x.x) * inv, bf_hi(x.x) * inv) | (cvt_e4m3x2(bf_lo(x.y) * inv, bf_hi(x.y) * inv) << 16);
    r.y = cvt_e4m3x2(bf_lo(x.z) * inv, bf_hi(x.z) * inv) | (cvt_e4m3x2(bf_lo(x.w) * inv, bf_hi(x.w) * inv) << 16);
    return r;
}

// 2 e4m3 codes (exact in fp16) times s, as packed bf16.
__device__ __forceinline__ uint32_t dequant2(uint32_t codes, float s) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi * s), "f"(lo * s));
    return r;
}
__device__ __forceinline__ uint4 dequant8(uint2 c, float s) {
    return make_uint4(dequant2(c.x & 0xffffu, s), dequant2(c.x >> 16, s), dequant2(c.y & 0xffffu, s),
                      dequant2(c.y >> 16, s));
}

// Where token t is kept: page (-1: nowhere) and row in the page; false if it belongs to no sequence.
__device__ __forceinline__ bool find_place(const PagedKV& kv, const int* cu, int t, int& pg, int& row) {
    const int b = paged_find(cu, kv.batch, t);
    pg = -1;
    row = 0;
    if (b < 0) return false;
    const PagedSeq s = paged_seq(kv, b);
    const int pos = s.base + (t - s.q0);
    if (pos >= 0 && pos < s.L) pg = paged_page(kv, b, pos, row);
    return true;
}

// cu for the searches: in shared memory when it fits.
__device__ __forceinline__ const int* stage_cu(const PagedKV& kv, int* sm) {
    if (kv.batch > kCuShared) return kv.cu;
    for (int i = threadIdx.x; i <= kv.batch; i += kThreads) sm[i] = __ldg(kv.cu + i);
    __syncthreads();
    return sm;
}

// Where a block's tokens are kept: page (-1: nowhere) and row in the page.
struct Places {
    int page[kMaxTokens], row[kMaxTokens];
    bool known[kMaxTokens];  // the token belongs to a sequence
};

// The places of tokens [t0, t0 + n).
__device__ __forceinline__ void find_places(const PagedKV& kv, int t0, int n, Places& w, int* sm) {
    const int* cu = stage_cu(kv, sm);
    if (threadIdx.x < n)
        w.known[threadIdx.x] = find_place(kv, cu, t0 + threadIdx.x, w.page[threadIdx.x], w.row[threadIdx.x]);
    __syncthreads();
}

template <int LPR, bool E4M3, int kUnroll>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ PagedCopyParams p) {
    __shared__ int sm[kCuShared + 1];
    __shared__ Places w;
    constexpr int kRowsAtOnce = kThreads / LPR;
    const PagedKV& kv = p.kv;
    const int t0 = blockIdx.x * p.tokens, n = min(p.tokens, kv.total - t0), rows = n * kv.hkv;
    const int part = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
    const int* cu = nullptr;
    for (int base = 0; base < rows; base += kRowsAtOnce * kUnroll) {
        uint4 xk[kUnroll], xv[kUnroll];
        int tl[kUnroll], h[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            // a row behind the last runs along with its warp, which shuffles, and stores nothing
            const int r = min(base + u * kRowsAtOnce + r0, rows - 1);
            tl[u] = static_cast<int>(fdiv(static_cast<unsigned>(r), p.by_heads));
            h[u] = r - tl[u] * kv.hkv;
            const long long t = t0 + tl[u];
            xk[u] = xv[u] = make_uint4(0, 0, 0, 0);
            if (!RA_CHECKED(paged_row_ok(kv, kv.hkv, t, h[u]), p.err, kSitePagedToken)) continue;
            xk[u] = ld_stream(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k_in) + t * p.k_ts + h[u] * p.k_hs) + part);
            xv[u] = ld_stream(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v_in) + t * p.v_ts + h[u] * p.v_hs) + part);
        }
        // (with the first rows on their way)
        if (kUnroll == 1) cu = cu ? cu : stage_cu(kv, sm);
        else if (base == 0) find_places(kv, t0, n, w, sm);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            int pg = -1, row = 0;
            if (base + u * kRowsAtOnce + r0 < rows) {
                if (kUnroll == 1) {
                    find_place(kv, cu, t0 + tl[u], pg, row);
                } else {
                    pg = w.page[tl[u]];
                    row = w.row[tl[u]];
                }
            }
            if (pg >= 0 && !RA_CHECKED(paged_place_ok(kv, pg, h[u], row), p.err, kSitePagedPlace)) pg = -1;
            const long long at = static_cast<long long>(h[u]) * kv.page + row;  // row inside the page
            if (E4M3) {
                float sk, sv;
                const uint32_t m = row_maxima<LPR>(xk[u], xv[u]);
                const uint2 ck = quantise8(xk[u], m & 0xffffu, sk), cv = quantise8(xv[u], m >> 16, sv);
                if (pg < 0) continue;
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(kv.k) + pg * kv.k_ps + at * (8 * LPR))[part] = ck;
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(kv.v) + pg * kv.v_ps + at * (8 * LPR))[part] = cv;
                if (part == 0) {
                    kv.k_scale[pg * kv.ks_ps + at] = sk;
                    kv.v_scale[pg * kv.vs_ps + at] = sv;
                }
            } else {
                if (pg < 0) continue;
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv.k) + pg * kv.k_ps + at * (8 * LPR))[part] = xk[u];
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv.v) + pg * kv.v_ps + at * (8 * LPR))[part] = xv[u];
            }
        }
    }
}

template <int LPR, bool E4M3, int kUnroll>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ PagedCopyParams p) {
    __shared__ int sm[kCuShared + 1];
    __shared__ Places w;
    constexpr int kRowsAtOnce = kThreads / LPR;
    const PagedKV& kv = p.kv;
    // a piece a thread: the whole output in its own order, so that neighbouring blocks read and
    // write on (18.2 us against 20.3 for 23k tokens of d = 64 with four tokens of all heads a block)
    const int t0 = kUnroll == 1 ? 0 : blockIdx.x * p.tokens, n = min(p.tokens, kv.total - t0), rows = n * kv.hkv;
    const int begin = kUnroll == 1 ? blockIdx.x * kRowsAtOnce : 0, end = kUnroll == 1 ? begin + 1 : rows;
    const int part = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
    const int* cu = nullptr;
    if (kUnroll == 1) cu = stage_cu(kv, sm);
    else find_places(kv, t0, n, w, sm);
    for (int base = begin; base < end; base += kRowsAtOnce * kUnroll) {
        uint4 xk[kUnroll], xv[kUnroll];
        uint2 ck[kUnroll], cv[kUnroll];
        float sk[kUnroll], sv[kUnroll];
        long long to[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = base + u * kRowsAtOnce + r0;  // head-major inside the block, as the pages and the output are
            const int h = n == p.tokens ? static_cast<int>(fdiv(static_cast<unsigned>(r), p.by_tokens)) : r / n, tl = r - h * n;
            to[u] = -1;
            xk[u] = xv[u] = make_uint4(0, 0, 0, 0);  // a position that no page holds reads as zeros
            ck[u] = cv[u] = make_uint2(0, 0);
            sk[u] = sv[u] = 0.f;
            if (r >= rows) continue;
            int pg, row;
            if (kUnroll == 1) {
                if (!find_place(kv, cu, t0 + tl, pg, row)) continue;
            } else {
                if (!w.known[tl]) continue;
                pg = w.page[tl];
                row = w.row[tl];
            }
            if (!RA_CHECKED(paged_row_ok(kv, kv.hkv, t0 + tl, h), p.err, kSitePagedToken)) continue;
            to[u] = (static_cast<long long>(h) * kv.total + t0 + tl) * LPR + part;
            if (pg < 0 || !RA_CHECKED(paged_place_ok(kv, pg, h, row), p.err, kSitePagedPlace)) continue;
            const long long at = static_cast<long long>(h) * kv.page + row;
            if (E4M3) {
                ck[u] = ld_stream(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(kv.k) + pg * kv.k_ps + at * (8 * LPR)) + part);
                cv[u] = ld_stream(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(kv.v) + pg * kv.v_ps + at * (8 * LPR)) + part);
                sk[u] = __ldg(kv.k_scale + pg * kv.ks_ps + at);
                sv[u] = __ldg(kv.v_scale + pg * kv.vs_ps + at);
            } else {
                xk[u] = ld_stream(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(kv.k) + pg * kv.k_ps + at * (8 * LPR)) + part);
                xv[u] = ld_stream(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(kv.v) + pg * kv.v_ps + at * (8 * LPR)) + part);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (to[u] < 0) continue;
            if (E4M3) {
                xk[u] = dequant8(ck[u], sk[u]);
                xv[u] = dequant8(cv[u], sv[u]);
            }
            reinterpret_cast<uint4*>(p.k_out)[to[u]] = xk[u];
            reinterpret_cast<uint4*>(p.v_out)[to[u]] = xv[u];
        }
    }
}

template <template <int, bool> class Launch>
int dispatch(PagedCopyParams p, bool whole, int sms, cudaStream_t stream) {
    // (the two sides of the rule, with times, are at the top)
    const long long per_token = static_cast<long long>(p.kv.hkv) * (p.kv.d / 8);  // threads' worth of rows
    const int unroll = per_token * p.kv.total > 8LL * 2048 * sms ? 4 : 1;
    p.tokens = static_cast<int>(kThreads * unroll / per_token);
    if (p.tokens > kMaxTokens) p.tokens = kMaxTokens;
    if (p.tokens < 1) p.tokens = 1;
    unsigned grid = static_cast<unsigned>((p.kv.total + p.tokens - 1) / p.tokens);
    if (whole && unroll == 1) {
        p.tokens = p.kv.total;
        grid = static_cast<unsigned>((per_token * p.kv.total + kThreads - 1) / kThreads);
    }
    p.by_heads = make_fastdiv(static_cast<unsigned>(p.kv.hkv));
    p.by_tokens = make_fastdiv(static_cast<unsigned>(p.tokens));
    if (p.kv.d == 128) {
        if (p.kv.e4m3) Launch<16, true>::go(p, grid, unroll, stream);
        else Launch<16, false>::go(p, grid, unroll, stream);
    } else {
        if (p.kv.e4m3) Launch<8, true>::go(p, grid, unroll, stream);
        else Launch<8, false>::go(p, grid, unroll, stream);
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <int LPR, bool E4M3>
struct Append {
    static void go(const PagedCopyParams& p, unsigned grid, int unroll, cudaStream_t s) {
        if (unroll == 4) append_kernel<LPR, E4M3, 4><<<grid, kThreads, 0, s>>>(p);
        else append_kernel<LPR, E4M3, 1><<<grid, kThreads, 0, s>>>(p);
    }
};
template <int LPR, bool E4M3>
struct Read {
    static void go(const PagedCopyParams& p, unsigned grid, int unroll, cudaStream_t s) {
        if (unroll == 4) read_kernel<LPR, E4M3, 4><<<grid, kThreads, 0, s>>>(p);
        else read_kernel<LPR, E4M3, 1><<<grid, kThreads, 0, s>>>(p);
    }
};

}  // namespace

int launch_cache_append(const PagedCopyParams& p, int sms, cudaStream_t stream) { return dispatch<Append>(p, false, sms, stream); }
int launch_cache_read(const PagedCopyParams& p, int sms, cudaStream_t stream) { return dispatch<Read>(p, true, sms, stream); }

}  // namespace ra
