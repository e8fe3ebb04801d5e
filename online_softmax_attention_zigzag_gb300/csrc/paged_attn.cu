// paged_attn.cu -- attention of new tokens over a paged K/V cache, the plain kernel: a warp per
// (row, query head) walks the visible keys one by one with an online softmax in fp32, each lane
// holding d / 32 elements.  Bound by the latency of its one key after the other.
#include <cuda_bf16.h>

#include "paged.h"

namespace ra {
namespace {

template <int N, bool E4M3>
__device__ __forceinline__ void load_row(const void* base, long long at, float s, int lane, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (E4M3) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h)
                : "h"(static_cast<uint16_t>(__ldg(static_cast<const uint8_t*>(base) + at + lane * N + i))));
            float f;
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(h));
            x[i] = f * s;
        } else {
            x[i] = __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(base) + at + lane * N + i)) << 16);
        }
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(256) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    constexpr int N = D / 32;
    const PagedKV& kv = p.kv;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32;
    if (w >= static_cast<long long>(kv.total) * p.hq) return;
    const int t = static_cast<int>(w / p.hq), hq = static_cast<int>(w % p.hq), h = hq / p.g;
    const int b = paged_find(kv.cu, kv.batch, t);
    if (b < 0) return;
    const PagedSeq s = paged_seq(kv, b);
    if (t - s.q0 >= p.max_q) return;
    const int i = s.base + (t - s.q0);
    const int hi = p.causal ? i + 1 : s.L;
    const int lo = p.window > 0 ? max(0, i - p.window + 1) : 0;
    float q[N], o[N] = {}, m = -INFINITY, l = 0.f;
    load_row<N, false>(p.q, t * p.q_ts + hq * p.q_hs, 1.f, lane, q);
    for (int j = 0; j < hi; ++j) {
        if (j < lo && j >= p.sinks) j = lo;
        int off;
        const int pg = paged_page(kv, b, j, off);
        float k[N] = {}, v[N] = {};
        if (pg >= 0) {
            const long long at = static_cast<long long>(h) * kv.page + off;
            load_row<N, E4M3>(kv.k, pg * kv.k_ps + at * D, E4M3 ? __ldg(kv.k_scale + pg * kv.ks_ps + at) : 1.f, lane, k);
            load_row<N, E4M3>(kv.v, pg * kv.v_ps + at * D, E4M3 ? __ldg(kv.v_scale + pg * kv.vs_ps + at) : 1.f, lane, v);
        }
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) x += q[e] * k[e];
#pragma unroll
        for (int e = 16; e; e >>= 1) x += __shfl_xor_sync(0xffffffffu, x, e);
        const float mn = fmaxf(m, x);
        const float f = (m == -INFINITY) ? 0.f : expf(m - mn), w1 = (x == -INFINITY) ? 0.f : expf(x - mn);
        l = l * f + w1;
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = o[e] * f + w1 * v[e];
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const long long at = t * p.o_ts + hq * p.o_hs + lane * N + e;
        if (p.out_f32) static_cast<float*>(p.out)[at] = o[e] * inv;
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(o[e] * inv);
    }
    if (lane == 0) p.lse[t * p.l_ts + hq * p.l_hs] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

int launch_paged_attn(const PagedAttnParams& p, cudaStream_t stream) {
    const long long warps = static_cast<long long>(p.kv.total) * p.hq;
    const unsigned grid = static_cast<unsigned>((warps + 7) / 8);
    if (p.kv.d == 128) {
        if (p.kv.e4m3) paged_attn_kernel<128, true><<<grid, 256, 0, stream>>>(p);
        else paged_attn_kernel<128, false><<<grid, 256, 0, stream>>>(p);
    } else {
        if (p.kv.e4m3) paged_attn_kernel<64, true><<<grid, 256, 0, stream>>>(p);
        else paged_attn_kernel<64, false><<<grid, 256, 0, stream>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace ra
