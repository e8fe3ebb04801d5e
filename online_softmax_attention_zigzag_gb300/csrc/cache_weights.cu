// cache_weights.cu -- the attention weight that every cached position has had from a call's rows, a KV head:
//
//     w[j] = (j < base ? decay w[j] : 0) + sum over the rows (t, head) that see j of exp(q . k_j - lse)
//
// base = L - T: the T newest positions are the call's own rows, whatever their places held before.  The scores are
// those of attention, once more: K is read again, V is not.  Keys are the rows of the product's tile and query rows its
// columns, so that a key's sum stays with the lanes that hold its scores: no atomics, one order of sums always.
//
// Few-row kernel: a warp takes 16 keys of one page at a time, straight from global memory into mma.sync fragments.  The
// order of the d elements in the product is free as long as K and q agree, so that a lane's fragments of two steps of
// 16 are 16 neighbouring bytes of a row.
#include <cuda_bf16.h>

#include "cache_weights.h"
#include "ptx_paged.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = kWeightsLog2e;

__device__ __forceinline__ uint4 ldg128(const void* p) {
    uint4 x;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
    return x;
}
__device__ __forceinline__ uint4 ldg128_stream(const void* p) {
    uint4 x;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
    return x;
}

// Columns 2 * (lane % 4) and the next one of a block of 8 query rows: what their scores are compared with.
struct Column {
    float bias;    // lse in powers of two; +inf: adds nothing
    int end, from;  // sees j < end, and j >= from or j < sinks
};

__device__ __forceinline__ Column column(const WeightsParams& p, const Seen& r, int h, int c) {
    Column x;
    x.bias = INFINITY;
    x.end = 0;
    x.from = 0;
    if (c >= r.T * p.g) return x;
    const int t = static_cast<int>(fdiv(static_cast<unsigned>(c), p.by_g)), head = h * p.g + c - t * p.g;
    const long long row = r.s.q0 + t;
    if (!RA_CHECKED(paged_row_ok(p.kv, p.hq, row, head), p.err, kSiteWeightsRow)) return x;
    const float lse = __ldg(p.lse + row * p.l_ts + head * p.l_hs);
    x.bias = lse == -INFINITY ? INFINITY : lse * kLog2e;
    x.end = p.causal ? min(r.s.L, r.s.base + t + 1) : r.s.L;
    x.from = p.window > 0 ? r.s.base + t - p.window + 1 : 0;
    return x;
}

// q's fragments of a block of 8 query rows, column lane / 4: words 4 s .. 4 s + 3 are the 8 elements that go with the
// lane's 8 of the keys, in pairs two steps' b0 and b1.  16 bytes of a key are 8 elements in bf16, 16 in e4m3.
template <int D, bool E4M3>
__device__ __forceinline__ void load_q(const WeightsParams& p, const Seen& r, int h, int c, uint32_t (&f)[D / 8]) {
    const bool on = c < r.T * p.g;
    const int t = on ? static_cast<int>(fdiv(static_cast<unsigned>(c), p.by_g)) : 0, head = h * p.g + (on ? c - t * p.g : 0);
    const long long row = r.s.q0 + t;
    const bool ok = on && RA_CHECKED(paged_row_ok(p.kv, p.hq, row, head), p.err, kSiteWeightsRow);
    const char* at = reinterpret_cast<const char*>(static_cast<const uint16_t*>(p.q) + row * p.q_ts + head * p.q_hs);
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (ok) x = ldg128(at + (E4M3 ? 128 * (s / 2) + 16 * (s % 2) + 32 * (threadIdx.x % 4) : 64 * s + 16 * (threadIdx.x % 4)));
        f[4 * s] = x.x;
        f[4 * s + 1] = x.y;
        f[4 * s + 2] = x.z;
        f[4 * s + 3] = x.w;
    }
}

// NB > 0: all query rows of a sequence and KV head fit into NB blocks of 8 columns, which stay in registers.
template <int D, bool E4M3, int NB>
__global__ void __launch_bounds__(kThreads) weights_kernel(const __grid_constant__ WeightsParams p) {
    extern __shared__ long long sums[];
    constexpr int kBlocks = NB > 0 ? NB : 1;
    const PagedKV& kv = p.kv;
    long long* seen = sums;
    long long* other = sums + kv.batch + 1;
    sum_up<kThreads>(kv.batch, seen, other, [&](int b, long long& x, long long& y) {
        const Seen r = look<kWeightsGroup>(p, b);
        x = static_cast<long long>(seen_groups(r)) * kv.hkv;
        y = static_cast<long long>(other_groups(r)) * kv.hkv;
    });
    const int lane = threadIdx.x % 32, quad = lane / 4;
    const long long warp = blockIdx.x * static_cast<long long>(kWarps) + threadIdx.x / 32, warps = gridDim.x * static_cast<long long>(kWarps);

    const long long n = seen[kv.batch];
    long long i = n * warp / warps;
    const long long i_end = n * (warp + 1) / warps;
    while (i < i_end) {
        // one (sequence, KV head) after the other
        const int b = find_sequence(seen, kv.batch, i);
        const Seen r = look<kWeightsGroup>(p, b);
        const int each = seen_groups(r);
        const int h = static_cast<int>((i - seen[b]) / each);
        int u = static_cast<int>((i - seen[b]) - static_cast<long long>(h) * each);
        const int u_end = static_cast<int>(min(static_cast<long long>(each), u + (i_end - i)));
        i += u_end - u;
        const int cols = r.T * p.g;
        uint32_t qf[kBlocks][D / 8];
        Column col[kBlocks][2];
        if (NB > 0) {
#pragma unroll
            for (int c = 0; c < NB; ++c) {
                load_q<D, E4M3>(p, r, h, 8 * c + quad, qf[c]);
                col[c][0] = column(p, r, h, 8 * c + 2 * (lane % 4));
                col[c][1] = column(p, r, h, 8 * c + 2 * (lane % 4) + 1);
            }
        }
        for (; u < u_end; ++u) {
            const int j0 = (u < r.sink_end ? u : u - r.sink_end + r.lo) * kWeightsGroup;
            int row;
            const int pg = paged_page(kv, b, j0, row);
            if (pg < 0 || !RA_CHECKED(paged_place_ok(kv, pg, h, row, kWeightsGroup), p.err, kSiteWeightsPlace)) continue;
            const long long place = static_cast<long long>(h) * kv.page + row;
            uint4 k[2][E4M3 ? D / 64 : D / 32];
            float mul[2] = {kLog2e, kLog2e};
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const char* at = static_cast<const char*>(kv.k) +
                                 (pg * kv.k_ps + (place + quad + 8 * m) * D) * (E4M3 ? 1 : 2) + 16 * (lane % 4);
#pragma unroll
                for (int s = 0; s < (E4M3 ? D / 64 : D / 32); ++s) k[m][s] = ldg128_stream(at + 64 * s);
                if (E4M3) mul[m] = __ldg(kv.k_scale + pg * kv.ks_ps + place + quad + 8 * m) * kLog2e;
            }
            float* wp = p.w + pg * p.w_ps + place + quad;
            float old[2] = {0.f, 0.f};
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int j = j0 + quad + 8 * m;
                old[m] = faded(p, r, j, wp + 8 * m);
            }
            // whether some row does not see some of these keys
            const bool whole = (p.causal ? j0 + kWeightsGroup <= r.s.base + 1 : j0 + kWeightsGroup <= r.s.L) &&
                               (p.window <= 0 || j0 + kWeightsGroup <= p.sinks || j0 > r.s.base + r.T - 1 - p.window);
            float sum[2] = {0.f, 0.f};
            for (int c0 = 0; c0 < cols; c0 += 8 * kBlocks) {
                if (NB == 0) {
                    load_q<D, E4M3>(p, r, h, c0 + quad, qf[0]);
                    col[0][0] = column(p, r, h, c0 + 2 * (lane % 4));
                    col[0][1] = column(p, r, h, c0 + 2 * (lane % 4) + 1);
                }
                float x[kBlocks][4];
#pragma unroll
                for (int c = 0; c < kBlocks; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[c][e] = 0.f;
#pragma unroll
                for (int s = 0; s < D / 32; ++s) {
                    uint4 ka, kb;
                    if (E4M3) {
                        const uint4 ca = k[0][s / 2], cb = k[1][s / 2];
                        expand4(s % 2 ? ca.z : ca.x, ka.x, ka.y);
                        expand4(s % 2 ? ca.w : ca.y, ka.z, ka.w);
                        expand4(s % 2 ? cb.z : cb.x, kb.x, kb.y);
                        expand4(s % 2 ? cb.w : cb.y, kb.z, kb.w);
                    } else {
                        ka = k[0][s];
                        kb = k[1][s];
                    }
                    const uint32_t a0[4] = {ka.x, kb.x, ka.y, kb.y}, a1[4] = {ka.z, kb.z, ka.w, kb.w};
#pragma unroll
                    for (int c = 0; c < kBlocks; ++c) {
                        mma16816<false>(x[c], a0, qf[c][4 * s], qf[c][4 * s + 1]);
                        mma16816<false>(x[c], a1, qf[c][4 * s + 2], qf[c][4 * s + 3]);
                    }
                }
#pragma unroll
                for (int c = 0; c < kBlocks; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const Column& y = col[c][e % 2];
                        bool on = y.bias != INFINITY;
                        if (!whole) {
                            const int j = j0 + quad + 8 * (e / 2);
                            on = on && j < y.end && (j >= y.from || j < p.sinks);
                        }
                        const float pr = ex2(fmaf(x[c][e], mul[e / 2], -y.bias));
                        sum[e / 2] += on ? pr : 0.f;
                    }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], 1);
                sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], 2);
                if (lane % 4 == 0 && j0 + quad + 8 * m < r.s.L) wp[8 * m] = old[m] + sum[m];
            }
        }
    }

    // positions that nobody sees: half a warp 16 of them
    const long long others = other[kv.batch];
    for (long long o = (others * warp / warps) + lane / 16; o < others * (warp + 1) / warps; o += 2) {
        const int b = find_sequence(other, kv.batch, o);
        const Seen r = look<kWeightsGroup>(p, b);
        const int each = other_groups(r);
        const int h = static_cast<int>((o - other[b]) / each), u = static_cast<int>((o - other[b]) - static_cast<long long>(h) * each);
        const int j0 = other_group(r, u) * kWeightsGroup, j = j0 + lane % 16;
        int row;
        const int pg = paged_page(kv, b, j0, row);
        if (pg < 0 || j >= r.s.L || !RA_CHECKED(paged_place_ok(kv, pg, h, row, kWeightsGroup), p.err, kSiteWeightsPlace)) continue;
        float* wp = p.w + pg * p.w_ps + static_cast<long long>(h) * kv.page + row + lane % 16;
        *wp = faded(p, r, j, wp);
    }
}

template <int D, bool E4M3, int NB>
int go(const WeightsParams& p, int sms, cudaStream_t stream) {
    static std::atomic<unsigned long long> done{0};
    const auto kernel = weights_kernel<D, E4M3, NB>;
    // (sums of up to RINGATTN_PAGED_MAX_BATCH sequences)
    if (!once_a_device(done, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 16 * (kPagedMaxBatch + 1)) == cudaSuccess;
        }))
        return -4;
    kernel<<<2 * sms, kThreads, 16 * (p.kv.batch + 1), stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <int D, bool E4M3>
int go_cols(const WeightsParams& p, int sms, cudaStream_t stream) {
    return p.max_q * p.g <= 8 ? go<D, E4M3, 1>(p, sms, stream) : go<D, E4M3, 2>(p, sms, stream);
}

}  // namespace

int launch_cache_weights_few(const WeightsParams& p, int sms, cudaStream_t stream) {
    if (p.kv.d == 128) return p.kv.e4m3 ? go_cols<128, true>(p, sms, stream) : go_cols<128, false>(p, sms, stream);
    return p.kv.e4m3 ? go_cols<64, true>(p, sms, stream) : go_cols<64, false>(p, sms, stream);
}

}  // namespace ra
