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
// thread so that two loads are in flight; they are bound by HBM.
#include <cuda_bf16.h>

#include "paged.h"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kCuShared = 1024;  // batches up to this keep cu in shared memory for the searches

__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 8 bf16 of a row held by LPR neighbouring lanes -> their codes and the row's scale.
template <int LPR>
__device__ __forceinline__ uint2 quantise8(uint4 x, float& scale) {
    // |x| of bf16 values orders like their bits without the sign
    uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                          __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int o = 1; o < LPR; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
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

// cu in shared memory when it fits
__device__ __forceinline__ const int* stage_cu(const PagedKV& kv, int* sm) {
    if (kv.batch > kCuShared) return kv.cu;
    for (int i = threadIdx.x; i <= kv.batch; i += kThreads) sm[i] = __ldg(kv.cu + i);
    __syncthreads();
    return sm;
}

template <int LPR, bool E4M3>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ PagedCopyParams p) {
    __shared__ int sm[kCuShared + 1];
    const PagedKV& kv = p.kv;
    const int* cu = stage_cu(kv, sm);
    const int part = threadIdx.x % LPR;
    const long long rows = static_cast<long long>(kv.total) * kv.hkv;
    const long long row0 = static_cast<long long>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
    // a row behind the last runs along with its warp, which shuffles, and stores nothing
    const int row = static_cast<int>(row0 < rows ? row0 : rows - 1);
    const int t = static_cast<int>(fdiv(static_cast<unsigned>(row), p.by_heads));
    const int h = row - t * kv.hkv;
    const uint4 xk = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k_in) + t * p.k_ts + h * p.k_hs) + part);
    const uint4 xv = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v_in) + t * p.v_ts + h * p.v_hs) + part);
    const int b = paged_find(cu, kv.batch, t);
    int pg = -1, off = 0;
    if (b >= 0 && row0 < rows) {
        const PagedSeq s = paged_seq(kv, b);
        const int pos = s.base + (t - s.q0);
        if (pos >= 0 && pos < s.L) pg = paged_page(kv, b, pos, off);
    }
    const long long at = static_cast<long long>(h) * kv.page + off;  // row inside the page
    if (E4M3) {
        float sk, sv;
        const uint2 ck = quantise8<LPR>(xk, sk), cv = quantise8<LPR>(xv, sv);
        if (pg < 0) return;
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(kv.k) + pg * kv.k_ps + at * (8 * LPR))[part] = ck;
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(kv.v) + pg * kv.v_ps + at * (8 * LPR))[part] = cv;
        if (part == 0) {
            kv.k_scale[pg * kv.ks_ps + at] = sk;
            kv.v_scale[pg * kv.vs_ps + at] = sv;
        }
    } else {
        if (pg < 0) return;
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv.k) + pg * kv.k_ps + at * (8 * LPR))[part] = xk;
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(kv.v) + pg * kv.v_ps + at * (8 * LPR))[part] = xv;
    }
}

template <int LPR, bool E4M3>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ PagedCopyParams p) {
    __shared__ int sm[kCuShared + 1];
    const PagedKV& kv = p.kv;
    const int* cu = stage_cu(kv, sm);
    const int part = threadIdx.x % LPR;
    const long long rows = static_cast<long long>(kv.total) * kv.hkv;
    const long long row0 = static_cast<long long>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
    if (row0 >= rows) return;
    const int row = static_cast<int>(row0);  // h * total + t: the output's order
    const int h = static_cast<int>(fdiv(static_cast<unsigned>(row), p.by_heads));
    const int t = row - h * kv.total;
    const int b = paged_find(cu, kv.batch, t);
    if (b < 0) return;
    const PagedSeq s = paged_seq(kv, b);
    const int pos = s.base + (t - s.q0);
    int off = 0;
    const int pg = (pos >= 0 && pos < s.L) ? paged_page(kv, b, pos, off) : -1;
    const long long at = static_cast<long long>(h) * kv.page + off;
    uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;  // a position that no page holds reads as zeros
    if (pg >= 0) {
        if (E4M3) {
            const uint2 ck = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(kv.k) + pg * kv.k_ps + at * (8 * LPR)) + part);
            const uint2 cv = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(kv.v) + pg * kv.v_ps + at * (8 * LPR)) + part);
            const float sk = __ldg(kv.k_scale + pg * kv.ks_ps + at), sv = __ldg(kv.v_scale + pg * kv.vs_ps + at);
            xk = dequant8(ck, sk);
            xv = dequant8(cv, sv);
        } else {
            xk = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(kv.k) + pg * kv.k_ps + at * (8 * LPR)) + part);
            xv = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(kv.v) + pg * kv.v_ps + at * (8 * LPR)) + part);
        }
    }
    reinterpret_cast<uint4*>(p.k_out)[row0 * LPR + part] = xk;
    reinterpret_cast<uint4*>(p.v_out)[row0 * LPR + part] = xv;
}

template <template <int, bool> class Launch>
int dispatch(const PagedCopyParams& p, cudaStream_t stream) {
    const long long rows = static_cast<long long>(p.kv.total) * p.kv.hkv;
    const int per = kThreads / (p.kv.d / 8);
    const unsigned grid = static_cast<unsigned>((rows + per - 1) / per);
    if (p.kv.d == 128) {
        if (p.kv.e4m3) Launch<16, true>::go(p, grid, stream);
        else Launch<16, false>::go(p, grid, stream);
    } else {
        if (p.kv.e4m3) Launch<8, true>::go(p, grid, stream);
        else Launch<8, false>::go(p, grid, stream);
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <int LPR, bool E4M3>
struct Append {
    static void go(const PagedCopyParams& p, unsigned grid, cudaStream_t s) { append_kernel<LPR, E4M3><<<grid, kThreads, 0, s>>>(p); }
};
template <int LPR, bool E4M3>
struct Read {
    static void go(const PagedCopyParams& p, unsigned grid, cudaStream_t s) { read_kernel<LPR, E4M3><<<grid, kThreads, 0, s>>>(p); }
};

}  // namespace

int launch_cache_append(const PagedCopyParams& p, cudaStream_t stream) { return dispatch<Append>(p, stream); }
int launch_cache_read(const PagedCopyParams& p, cudaStream_t stream) { return dispatch<Read>(p, stream); }

}  // namespace ra
