// qk_norm.cu -- what comes between the projections and attention: every head's q and k row x normed by its root mean
// square, weighted and turned by its position, in one pass, and the gradients of that.
//
//     r = 1 / sqrt(mean(x^2) + eps),  y = w x r,  z = R(position) y s          (s: q's scale; 1 for k)
// where R turns every pair (a, b) of the first `rot` elements: (a cos - b sin, b cos + a sin).  With dz given:
//     g = s R^T dz,  dw = sum over rows of g x r,  u = w g,  dx = r (u - x r^2 mean(u x)).
// All of it in fp32, rounded once where a row is stored in bf16.
//
// Both are bound by HBM: 4 bytes an element forward, 8 backward with fp32 gradients (32k tokens, 64 query and 8 KV heads, d = 128,
// head-major results: 202 us, 6.1 TB/s; 394 us, 6.2 TB/s).  A row is held by d / 8
// neighbouring lanes, two pieces of 4 elements each: where pairs lie rot / 2 apart, the piece and the one that it is
// paired with, so that a pair never crosses lanes and the only shuffles are those of the row's sums.  A lane's four rows
// are heads of one token, all loads in flight at once, and share its cosines and sines.  Hints that keep the rows out of the
// caches made it slower (loads: 211 us and 408).
#include <cuda_bf16.h>

#include "qk_norm.h"
#include "ptx_paged.cuh"

namespace ra {
namespace {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The elements of a lane's two pieces: of d / 8 lanes, those below rot / 8 hold what is turned.
struct Pieces {
    int at[2];
    bool turned;
};
__device__ __forceinline__ Pieces pieces(int lane, int rot, int d) {
    const int n = rot / 8;
    Pieces s;
    s.turned = lane < n;
    s.at[0] = s.turned ? 4 * lane : rot + 4 * (lane - n);
    s.at[1] = s.at[0] + (s.turned ? rot / 2 : (d - rot) / 2);
    return s;
}

// Four elements as fp32.
__device__ __forceinline__ void unpack4(uint2 w, float* x) {
    x[0] = bf_lo(w.x);
    x[1] = bf_hi(w.x);
    x[2] = bf_lo(w.y);
    x[3] = bf_hi(w.y);
}
__device__ __forceinline__ void unpack4(float4 w, float* x) {
    x[0] = w.x;
    x[1] = w.y;
    x[2] = w.z;
    x[3] = w.w;
}
__device__ __forceinline__ void pack4(const float* x, uint2& w) { w = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])); }
__device__ __forceinline__ void pack4(const float* x, float4& w) { w = make_float4(x[0], x[1], x[2], x[3]); }

// Storage of four elements.  (Plain loads: a row may be written where it was read.)
template <bool F32>
struct Quad {
    using T = uint2;
    using E = uint16_t;
};
template <>
struct Quad<true> {
    using T = float4;
    using E = float;
};

// Cosines and sines of a lane's eight elements: z_i = c_i x_i + s_i x_pair(i), where the pair of element i is
// element i + 4 of the lane's eight (halves) or its neighbour (interleaved).  Elements that are not turned: 1 and 0.
template <bool INTER>
__device__ __forceinline__ void load_turn(const NormParams& p, int pos, const Pieces& at, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
    }
    if (!at.turned || !RA_CHECKED(pos >= 0 && pos < p.n_pos && at.at[1] + 4 <= p.rot, p.err, kSiteNormTable)) return;
    const float* row = p.cos_sin + static_cast<long long>(pos) * p.rot;
    if (INTER) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 a = __ldg(reinterpret_cast<const float2*>(row + at.at[k] / 2));
            const float2 b = __ldg(reinterpret_cast<const float2*>(row + p.rot / 2 + at.at[k] / 2));
            c[4 * k] = c[4 * k + 1] = a.x;
            c[4 * k + 2] = c[4 * k + 3] = a.y;
            s[4 * k] = -b.x;
            s[4 * k + 1] = b.x;
            s[4 * k + 2] = -b.y;
            s[4 * k + 3] = b.y;
        }
    } else {
        const float4 a = __ldg(reinterpret_cast<const float4*>(row + at.at[0]));
        const float4 b = __ldg(reinterpret_cast<const float4*>(row + p.rot / 2 + at.at[0]));
        float x[4], y[4];
        unpack4(a, x);
        unpack4(b, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = c[i + 4] = x[i];
            s[i] = -y[i];
            s[i + 4] = y[i];
        }
    }
}

template <bool INTER>
__device__ __forceinline__ constexpr int pair_of(int i) {
    return INTER ? i ^ 1 : i ^ 4;
}

__device__ __forceinline__ void load_weights(const NormParams& p, int kind, const Pieces& at, float (&w)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!p.w[kind]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * k + i] = 1.f;
        } else if (p.w_f32) {
            unpack4(__ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.w[kind]) + at.at[k])), w + 4 * k);
        } else {
            unpack4(__ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.w[kind]) + at.at[k])), w + 4 * k);
        }
    }
}

// Sum over a row's lanes.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 1; o < LPR; o *= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Rows whose mean(x^2) + eps is out of 2^-60 .. 2^60 (or NaN): their squares, or the sum of them, may leave fp32's normal numbers.  They are
// left for a second look (FAR), in kernels of their own for an eps so small that it does not cover rows whose squares vanish: the look
// costs the backward pass 8 to 11 us of 32k tokens' 346 to 458 (64 query and 8 KV heads, d = 128), the forward pass 2 of 203.
constexpr float kFar = 0x1p-60f;
__device__ __forceinline__ bool far_out(float mean) { return !(mean >= kFar && mean <= 0x1p60f); }
// Such a row's x times a power of two `a` that brings the larger of its largest element and sqrt(eps) to about 1, and
// 1 / sqrt(mean + eps) of that, so that x r is what it was.  A warp's lanes run together.
template <int LPR>
__device__ __forceinline__ float bring_in(float (&x)[8], float eps, float& a) {
    uint32_t top = eps > 0.f ? ((__float_as_uint(eps) >> 23) + 127u) >> 1 : 0u;  // a biased exponent
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t e = __float_as_uint(x[i]) >> 23 & 0xffu;
        top = max(top, e == 0xffu ? 0u : e);
    }
#pragma unroll
    for (int o = 1; o < LPR; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    a = __uint_as_float(max(254u - top, 1u) << 23);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] *= a;
        ss = fmaf(x[i], x[i], ss);
    }
    return rsqrtf(fmaf(row_sum<LPR>(ss), 1.f / (8 * LPR), eps * a * a));
}

// What a block's threads do: blockIdx.y is a group of heads of q or of k, and a row's lanes take tokens
// blocks_x * kNormThreads / LPR apart.
struct Part {
    int kind, h0, heads;  // heads h0 .. h0 + heads of q (0) or k (1)
};
__device__ __forceinline__ Part block_part(const NormParams& p) {
    Part s;
    s.kind = static_cast<int>(blockIdx.y) >= p.groups[0];
    s.h0 = (static_cast<int>(blockIdx.y) - (s.kind ? p.groups[0] : 0)) * kNormHeads;
    s.heads = min(kNormHeads, p.heads[s.kind] - s.h0);
    return s;
}

template <int LPR, bool INTER, bool FAR>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const __grid_constant__ NormParams p) {
    constexpr int kTokens = kNormThreads / LPR;
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const Part part = block_part(p);
    const Pieces at = pieces(lane, p.rot, 8 * LPR);
    const float inv_d = 1.f / (8 * LPR);
    float w[8];
    load_weights(p, part.kind, at, w);
    // (a warp's lanes all run the same number of times: they shuffle)
    for (int t0 = blockIdx.x * kTokens; t0 < p.total; t0 += p.blocks_x * kTokens) {
        const int t = min(t0 + slot, p.total - 1);
        uint2 raw[kNormHeads][2];
        const uint16_t* src = static_cast<const uint16_t*>(p.x.p[part.kind]) + t * p.x.ts[part.kind] + part.h0 * p.x.hs[part.kind];
#pragma unroll
        for (int h = 0; h < kNormHeads; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                raw[h][k] = make_uint2(0, 0);
                if (h < part.heads && RA_CHECKED(t >= 0 && part.h0 + h < p.heads[part.kind], p.err, kSiteNormRow))
                    raw[h][k] = *reinterpret_cast<const uint2*>(src + h * p.x.hs[part.kind] + at.at[k]);
            }
        const int pos = __ldg(p.position + t);
        const bool on = t0 + slot < p.total && pos >= 0 && pos < p.n_pos;
        float c[8], s[8];
        load_turn<INTER>(p, on ? pos : 0, at, c, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // (the weight and the scale go with the cosines and sines)
            s[i] *= w[pair_of<INTER>(i)] * p.scale[part.kind];
            c[i] *= w[i] * p.scale[part.kind];
        }
        uint16_t* dst = static_cast<uint16_t*>(p.y.p[part.kind]) + t * p.y.ts[part.kind] + part.h0 * p.y.hs[part.kind];
        auto store = [&](int h, const float (&x)[8], float r) {
            float z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = r * fmaf(x[i], c[i], at.turned ? x[pair_of<INTER>(i)] * s[i] : 0.f);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint2 o;
                pack4(z + 4 * k, o);
                *reinterpret_cast<uint2*>(dst + h * p.y.hs[part.kind] + at.at[k]) = o;
            }
        };
        uint32_t later = 0;  // heads whose rows are far out
#pragma unroll
        for (int h = 0; h < kNormHeads; ++h) {
            float x[8], ss = 0.f;
            unpack4(raw[h][0], x);
            unpack4(raw[h][1], x + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            const float mean = fmaf(row_sum<LPR>(ss), inv_d, p.eps);
            if (!on || h >= part.heads || !RA_CHECKED(part.h0 + h < p.heads[part.kind], p.err, kSiteNormRow)) continue;
            if (FAR && far_out(mean)) later |= 1u << h;
            else store(h, x, rsqrtf(mean));
        }
        if (FAR && __any_sync(0xffffffffu, later != 0u)) {
#pragma unroll 1
            for (int h = 0; h < part.heads; ++h) {
                const bool mine = later >> h & 1u;
                float x[8] = {}, a;
                if (mine) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) unpack4(*reinterpret_cast<const uint2*>(src + h * p.x.hs[part.kind] + at.at[k]), x + 4 * k);
                }
                const float r = bring_in<LPR>(x, p.eps, a);
                if (mine) store(h, x, r);
            }
        }
    }
}

template <int LPR, bool INTER, bool DY32, bool DX32, bool FAR>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_kernel(const __grid_constant__ NormParams p) {
    using QY = typename Quad<DY32>::T;
    using QX = typename Quad<DX32>::T;
    constexpr int kTokens = kNormThreads / LPR;
    __shared__ alignas(16) float sums[kTokens][8 * LPR];
    const int lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    const Part part = block_part(p);
    const Pieces at = pieces(lane, p.rot, 8 * LPR);
    const float inv_d = 1.f / (8 * LPR);
    float w[8], dw[8];
    load_weights(p, part.kind, at, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0.f;
    for (int t0 = blockIdx.x * kTokens; t0 < p.total; t0 += p.blocks_x * kTokens) {
        const int t = min(t0 + slot, p.total - 1);
        uint2 raw[kNormHeads][2];
        QY grad[kNormHeads][2];
        const uint16_t* src = static_cast<const uint16_t*>(p.x.p[part.kind]) + t * p.x.ts[part.kind] + part.h0 * p.x.hs[part.kind];
        const typename Quad<DY32>::E* dy =
            static_cast<const typename Quad<DY32>::E*>(p.y.p[part.kind]) + t * p.y.ts[part.kind] + part.h0 * p.y.hs[part.kind];
#pragma unroll
        for (int h = 0; h < kNormHeads; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                raw[h][k] = make_uint2(0, 0);
                grad[h][k] = QY{};
                if (h < part.heads && RA_CHECKED(t >= 0 && part.h0 + h < p.heads[part.kind], p.err, kSiteNormRow)) {
                    raw[h][k] = *reinterpret_cast<const uint2*>(src + h * p.x.hs[part.kind] + at.at[k]);
                    grad[h][k] = *reinterpret_cast<const QY*>(dy + h * p.y.hs[part.kind] + at.at[k]);
                }
            }
        // (the loads stay before the arithmetic, which the compiler otherwise mixes with them for the second look's sake: bf16 gradients
        // 367 us, 357 so)
        if (FAR) asm volatile("" ::: "memory");
        const int pos = __ldg(p.position + t);
        const bool on = t0 + slot < p.total && pos >= 0 && pos < p.n_pos;
        float c[8], s[8];
        load_turn<INTER>(p, on ? pos : 0, at, c, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] *= p.scale[part.kind];
            s[i] *= -p.scale[part.kind];  // turned back
        }
        typename Quad<DX32>::E* dst =
            static_cast<typename Quad<DX32>::E*>(p.g.p[part.kind]) + t * p.g.ts[part.kind] + part.h0 * p.g.hs[part.kind];
        // u: dout; then dout turned back, g, and u
        auto turn_back = [&](float (&u)[8], float (&g)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = fmaf(u[i], c[i], at.turned ? u[pair_of<INTER>(i)] * s[i] : 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = g[i] * w[i];
        };
        auto store = [&](int h, const float (&x)[8]) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                QX o;
                pack4(x + 4 * k, o);
                *reinterpret_cast<QX*>(dst + h * p.g.hs[part.kind] + at.at[k]) = o;
            }
        };
        uint32_t later = 0;  // heads whose rows are far out
#pragma unroll
        for (int h = 0; h < kNormHeads; ++h) {
            float x[8], g[8], u[8], ss = 0.f, ux = 0.f;
            unpack4(raw[h][0], x);
            unpack4(raw[h][1], x + 4);
            unpack4(grad[h][0], u);
            unpack4(grad[h][1], u + 4);
            turn_back(u, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = fmaf(x[i], x[i], ss);
                ux = fmaf(u[i], x[i], ux);
            }
            const float mean = fmaf(row_sum<LPR>(ss), inv_d, p.eps), r = rsqrtf(mean);
            const float m = row_sum<LPR>(ux) * inv_d * r * r;
            const bool far = FAR && far_out(mean), here = on && h < part.heads && RA_CHECKED(part.h0 + h < p.heads[part.kind], p.err, kSiteNormRow);
            if (here && far) later |= 1u << h;
            if (!here || far) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[i] = fmaf(g[i], x[i] * r, dw[i]);
                u[i] = r * fmaf(-m, x[i], u[i]);
            }
            store(h, u);
        }
        if (FAR && __any_sync(0xffffffffu, later != 0u)) {
#pragma unroll 1
            for (int h = 0; h < part.heads; ++h) {
                const bool mine = later >> h & 1u;
                float x[8] = {}, g[8], u[8] = {}, ux = 0.f, a;
                if (mine) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        unpack4(*reinterpret_cast<const uint2*>(src + h * p.x.hs[part.kind] + at.at[k]), x + 4 * k);
                        unpack4(*reinterpret_cast<const QY*>(dy + h * p.y.hs[part.kind] + at.at[k]), u + 4 * k);
                    }
                }
                turn_back(u, g);
                const float r = bring_in<LPR>(x, p.eps, a);
#pragma unroll
                for (int i = 0; i < 8; ++i) ux = fmaf(u[i], x[i], ux);
                const float m = row_sum<LPR>(ux) * inv_d * r * r;
                if (!mine) continue;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dw[i] = fmaf(g[i], x[i] * r, dw[i]);
                    u[i] = r * fmaf(-m, x[i], u[i]) * a;  // (r of x is a times that of a x, which may be more than fp32 holds)
                }
                store(h, u);
            }
        }
    }
    launch_dependents();
    if (!p.dw[part.kind]) return;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        *reinterpret_cast<float4*>(&sums[slot][at.at[k]]) = make_float4(dw[4 * k], dw[4 * k + 1], dw[4 * k + 2], dw[4 * k + 3]);
    __syncthreads();
    const int e = threadIdx.x;
    if (e < 8 * LPR) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kTokens; ++i) sum += sums[i][e];
        const int row = static_cast<int>(blockIdx.y * gridDim.x + blockIdx.x);
        if (RA_CHECKED(row < (p.groups[0] + p.groups[1]) * p.blocks_x, p.err, kSiteNormPartial))
            p.partial[static_cast<long long>(row) * (8 * LPR) + e] = sum;
    }
}

// The blocks' sums added up, always in the same order: eight columns of q's or k's a block, 32 threads a column.
__global__ void __launch_bounds__(256) norm_dw_kernel(const __grid_constant__ NormParams p) {
    __shared__ float sm[32][8];
    const int kind = blockIdx.y, e = blockIdx.x * 8 + threadIdx.x % 8, part = threadIdx.x / 8;
    const int n = p.groups[kind] * p.blocks_x, first = kind ? p.groups[0] * p.blocks_x : 0;
    if (!p.dw[kind]) return;
    wait_primary();
    float sum = 0.f;
#pragma unroll 4
    for (int i = part; i < n; i += 32) sum += __ldcg(p.partial + static_cast<long long>(first + i) * p.d + e);
    sm[part][threadIdx.x % 8] = sum;
    __syncthreads();
    if (threadIdx.x < 8) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += sm[i][threadIdx.x];
        p.dw[kind][e] = sum;
    }
}

template <int LPR, bool INTER, bool FAR>
void go(const NormParams& p, dim3 grid, cudaStream_t s) {
    norm_kernel<LPR, INTER, FAR><<<grid, kNormThreads, 0, s>>>(p);
}

template <int LPR, bool INTER, bool FAR>
void go_bwd(const NormParams& p, dim3 grid, bool dy_f32, bool dx_f32, cudaStream_t s) {
    if (dy_f32) {
        if (dx_f32) norm_bwd_kernel<LPR, INTER, true, true, FAR><<<grid, kNormThreads, 0, s>>>(p);
        else norm_bwd_kernel<LPR, INTER, true, false, FAR><<<grid, kNormThreads, 0, s>>>(p);
    } else {
        if (dx_f32) norm_bwd_kernel<LPR, INTER, false, true, FAR><<<grid, kNormThreads, 0, s>>>(p);
        else norm_bwd_kernel<LPR, INTER, false, false, FAR><<<grid, kNormThreads, 0, s>>>(p);
    }
}

}  // namespace

int norm_blocks(int total, int groups, int d, int most) {
    const int tokens = kNormThreads / (d / 8);
    const int all = total / tokens + (total % tokens != 0);
    const int cap = most / groups > 1 ? most / groups : 1;
    return all < cap ? all : cap;
}

int launch_qk_norm_rope(NormParams p, int sms, cudaStream_t stream) {
    const int groups = p.groups[0] + p.groups[1];
    p.blocks_x = norm_blocks(p.total, groups, p.d, sms * kNormBlocksPerSm);
    const dim3 grid(p.blocks_x, groups);
    const bool far = p.eps < kFar;
#define RA_GO(LPR, INTER) far ? go<LPR, INTER, true>(p, grid, stream) : go<LPR, INTER, false>(p, grid, stream)
    if (p.d == 128) p.interleaved ? (RA_GO(16, true)) : (RA_GO(16, false));
    else p.interleaved ? (RA_GO(8, true)) : (RA_GO(8, false));
#undef RA_GO
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

int launch_qk_norm_rope_bwd(NormParams p, bool dy_f32, bool dx_f32, int sms, cudaStream_t stream) {
    const int groups = p.groups[0] + p.groups[1];
    p.blocks_x = norm_blocks(p.total, groups, p.d, sms * kNormBwdBlocksPerSm);
    const dim3 grid(p.blocks_x, groups);
    const bool far = p.eps < kFar;
#define RA_GO(LPR, INTER) far ? go_bwd<LPR, INTER, true>(p, grid, dy_f32, dx_f32, stream) : go_bwd<LPR, INTER, false>(p, grid, dy_f32, dx_f32, stream)
    if (p.total == 0) {  // (no rows: the weights' gradients are sums of nothing)
    } else if (p.d == 128) {
        p.interleaved ? (RA_GO(16, true)) : (RA_GO(16, false));
    } else {
        p.interleaved ? (RA_GO(8, true)) : (RA_GO(8, false));
    }
#undef RA_GO
    if (cudaGetLastError() != cudaSuccess) return -4;
    if (!p.dw[0] && !p.dw[1]) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.d / 8, 2);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_dw_kernel, p) == cudaSuccess ? 0 : -4;
}

}  // namespace ra
