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
// 16 are 16 neighbouring bytes of a row.  Bound by HBM: one token each of 64 sequences of up to 16k keys (64 query heads, 8 KV heads,
// d = 128, bf16) 188 us, 6.4 TB/s; of 8 sequences of up to 128k keys in e4m3 190 us, 5.8 TB/s.
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
    float bias;    // lse in powers of two; -inf: adds nothing
    float mul;     // what a product is multiplied by for a score in powers of two, but for the key's scale
    int end, from;  // sees j < end, and j >= from or j < sinks
};

__device__ __forceinline__ Column column(const WeightsParams& p, const Seen& r, int h, int c) {
    Column x;
    x.bias = -INFINITY;
    x.mul = kLog2e;
    x.end = 0;
    x.from = 0;
    if (c >= r.T * p.g) return x;
    const int t = static_cast<int>(fdiv(static_cast<unsigned>(c), p.by_g)), head = h * p.g + c - t * p.g;
    const long long row = r.s.q0 + t;
    if (!RA_CHECKED(paged_row_ok(p.kv, p.hq, row, head), p.err, kSiteWeightsRow)) return x;
    const float lse = __ldg(p.lse + row * p.l_ts + head * p.l_hs);
    x.bias = lse < -0x1p127f && lse > -INFINITY ? -0x1p127f : lse * kLog2e;  // (no other lse becomes -inf)
    x.end = p.causal ? min(r.s.L, r.s.base + t + 1) : r.s.L;
    x.from = p.window > 0 ? r.s.base + t - p.window + 1 : 0;
    return x;
}

// q's fragments of a block of 8 query rows, column lane / 4: words 4 s .. 4 s + 3 are the 8 elements that go with the
// lane's 8 of the keys, in pairs two steps' b0 and b1.  16 bytes of a key are 8 elements in bf16, 16 in e4m3.  For e4m3 they
// become fp16, as the codes do (exactly, in one instruction for two of them): times a power of two that brings the row's largest
// finite element to 2^14 .. 2^15, so that elements below 2^-28 of it lose bits.  Returns what undoes that.
template <int D, bool E4M3>
__device__ __forceinline__ float load_q(const WeightsParams& p, const Seen& r, int h, int c, uint32_t (&f)[D / 8]) {
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
    if (!E4M3) return 1.f;
    int top = 0;  // largest biased exponent of a finite element
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const int lo = (f[i] >> 7) & 0xff, hi = (f[i] >> 23) & 0xff;
        top = max(top, max(lo == 0xff ? 0 : lo, hi == 0xff ? 0 : hi));
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int up = min(141 - top, 126);  // (rows below 2^-112: what fp32 can undo)
    const float a = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) f[i] = pack_f16x2(__uint_as_float(f[i] << 16) * a, __uint_as_float(f[i] & 0xffff0000u) * a);
    return __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
}

// Four e4m3 codes as two pairs of fp16, exact.
__device__ __forceinline__ void codes_f16(uint32_t codes, uint32_t& a, uint32_t& b) {
    a = e4m3x2_f16x2(codes & 0xffffu);
    b = e4m3x2_f16x2(codes >> 16);
}

// Positions that nobody sees: half a warp 16 of them.  other: their groups, summed up over the sequences.
__device__ void fade_others(const WeightsParams& p, const long long* other, long long warp, long long warps) {
    const PagedKV& kv = p.kv;
    const int lane = threadIdx.x % 32;
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

// A group of 16 keys: a lane's pieces of rows lane / 4 and lane / 4 + 8, their scales, weights and where those are.
template <int D, bool E4M3>
struct Keys {
    static constexpr int kPieces = E4M3 ? D / 64 : D / 32;
    uint4 k[2][kPieces];
    float mul[2], old[2];
    float* w;  // null: no page
    int j0;
};

// Blocks of an SM, which share its registers.  bf16 keeps the loads of 16 warps in flight (64 x 16k tokens: 188 us with two, 195
// with three).  In e4m3 a warp has half as many bytes in flight and turns codes into fp16 meanwhile: 8 x 128k take 190 us with
// three, 236 with two, 222 with four, which spill; loading a group ahead, or two at a time, left no registers for the third: 243, 236.
// All that was measured with one block of columns.  Two of them (9 to 16 rows) spill with three as well, 244 bytes a thread at d = 128:
// 8 sequences of 100k to 128k with two tokens of 8 heads take 265 us for a floor of 158, 64 of up to 16k 148 for 84.
template <bool E4M3>
constexpr int blocks_per_sm() { return E4M3 ? 3 : 2; }

// All query rows of a sequence and KV head fit into NB blocks of 8 columns, which stay in registers.
template <int D, bool E4M3, int NB>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<E4M3>()) weights_kernel(const __grid_constant__ WeightsParams p) {
    extern __shared__ long long sums[];
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
        uint32_t qf[NB][D / 8];
        Column col[NB][2];
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            const float undo = load_q<D, E4M3>(p, r, h, 8 * c + quad, qf[c]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                col[c][e] = column(p, r, h, 8 * c + 2 * (lane % 4) + e);
                if (E4M3) col[c][e].mul *= __shfl_sync(0xffffffffu, undo, 4 * (2 * (lane % 4) + e));
            }
        }
        // groups follow one another on a page: its place is looked up once
        int left = 0;  // groups of the page that are still to come
        const char* kp = nullptr;
        const float* sp = nullptr;
        float* wp = nullptr;
        auto fetch = [&](int at, Keys<D, E4M3>& f) {
            f.j0 = (at < r.sink_end ? at : at - r.sink_end + r.lo) * kWeightsGroup;
            if (left == 0 || at == r.sink_end) {
                int row;
                const int pg = paged_page(kv, b, f.j0, row);
                left = (kv.page - row) / kWeightsGroup;
                wp = nullptr;
                if (pg >= 0 && RA_CHECKED(paged_place_ok(kv, pg, h, row, left * kWeightsGroup), p.err, kSiteWeightsPlace)) {
                    const long long place = static_cast<long long>(h) * kv.page + row + quad;
                    wp = p.w + pg * p.w_ps + place;
                    kp = static_cast<const char*>(kv.k) + (pg * kv.k_ps + place * D) * (E4M3 ? 1 : 2) + 16 * (lane % 4);
                    if (E4M3) sp = kv.k_scale + pg * kv.ks_ps + place;
                }
            }
            --left;
            f.w = wp;
            if (!wp) return;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
#pragma unroll
                for (int s = 0; s < Keys<D, E4M3>::kPieces; ++s) f.k[m][s] = ldg128_stream(kp + 8 * m * D * (E4M3 ? 1 : 2) + 64 * s);
                f.mul[m] = E4M3 ? __ldg(sp + 8 * m) : 1.f;
                f.old[m] = faded(p, r, f.j0 + quad + 8 * m, wp + 8 * m);
            }
            kp += kWeightsGroup * D * (E4M3 ? 1 : 2);
            if (E4M3) sp += kWeightsGroup;
            wp += kWeightsGroup;
        };
        auto use = [&](const Keys<D, E4M3>& f) {
            if (!f.w) return;
            const int j0 = f.j0;
            // whether some row does not see some of these keys
            const bool whole = (p.causal ? j0 + kWeightsGroup <= r.s.base + 1 : j0 + kWeightsGroup <= r.s.L) &&
                               (p.window <= 0 || j0 + kWeightsGroup <= p.sinks || j0 > r.s.base + r.T - 1 - p.window);
            float sum[2] = {0.f, 0.f}, x[NB][4];
#pragma unroll
            for (int c = 0; c < NB; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[c][e] = 0.f;
#pragma unroll
            for (int s = 0; s < D / 32; ++s) {
                uint4 ka, kb;
                if (E4M3) {
                    const uint4 ca = f.k[0][s / 2], cb = f.k[1][s / 2];
                    codes_f16(s % 2 ? ca.z : ca.x, ka.x, ka.y);
                    codes_f16(s % 2 ? ca.w : ca.y, ka.z, ka.w);
                    codes_f16(s % 2 ? cb.z : cb.x, kb.x, kb.y);
                    codes_f16(s % 2 ? cb.w : cb.y, kb.z, kb.w);
                } else {
                    ka = f.k[0][s];
                    kb = f.k[1][s];
                }
                const uint32_t a0[4] = {ka.x, kb.x, ka.y, kb.y}, a1[4] = {ka.z, kb.z, ka.w, kb.w};
#pragma unroll
                for (int c = 0; c < NB; ++c) {
                    mma16816<E4M3>(x[c], a0, qf[c][4 * s], qf[c][4 * s + 1]);
                    mma16816<E4M3>(x[c], a1, qf[c][4 * s + 2], qf[c][4 * s + 3]);
                }
            }
#pragma unroll
            for (int c = 0; c < NB; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Column& y = col[c][e % 2];
                    bool on = y.bias != -INFINITY;
                    if (!whole) {
                        const int j = j0 + quad + 8 * (e / 2);
                        on = on && j < y.end && (j >= y.from || j < p.sinks);
                    }
                    const float pr = ex2(fmaf(x[c][e], E4M3 ? f.mul[e / 2] * y.mul : kLog2e, -y.bias));
                    sum[e / 2] += on ? pr : 0.f;
                }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], 1);
                sum[m] += __shfl_xor_sync(0xffffffffu, sum[m], 2);
                if (lane % 4 == 0 && j0 + quad + 8 * m < r.s.L) f.w[8 * m] = f.old[m] + sum[m];
            }
        };
        for (; u < u_end; ++u) {
            Keys<D, E4M3> f;
            fetch(u, f);
            use(f);
        }
    }

    fade_others(p, other, warp, warps);
}

// More rows of a sequence and KV head, up to kWeightsWideRows: too many for registers.  A block takes a stretch of groups, its
// warps every eighth, with q's fragments in shared memory as the lanes take them (16 bytes a lane, no conflicts), and so is what a
// column's scores are compared with.  K is read once whatever the rows are, in e4m3 turned into fp16 once.
// Blocks of an SM.  24 and 64 rows of e4m3 take 107 and 140 us so; with four 122 and 145; with two, and two groups a warp, which halves
// the reads of q from shared memory, 134 and 166.
constexpr int kWideBlocks = 3;

struct WideColumn {
    float bias, mul;
    int end, from;
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, kWideBlocks) weights_wide_kernel(const __grid_constant__ WeightsParams p) {
    constexpr int kSteps = D / 32;  // pairs of steps of 16
    extern __shared__ long long sums[];
    __shared__ uint4 qs[kWeightsWideRows / 8][kSteps][32];
    __shared__ WideColumn cs[kWeightsWideRows];
    const PagedKV& kv = p.kv;
    long long* seen = sums;
    long long* other = sums + kv.batch + 1;
    sum_up<kThreads>(kv.batch, seen, other, [&](int b, long long& x, long long& y) {
        const Seen r = look<kWeightsGroup>(p, b);
        x = static_cast<long long>(seen_groups(r)) * kv.hkv;
        y = static_cast<long long>(other_groups(r)) * kv.hkv;
    });
    const int lane = threadIdx.x % 32, quad = lane / 4, warp = threadIdx.x / 32;
    const long long n = seen[kv.batch];
    long long i = n * blockIdx.x / gridDim.x;
    const long long i_end = n * (blockIdx.x + 1) / gridDim.x;
    while (i < i_end) {
        const int b = find_sequence(seen, kv.batch, i);
        const Seen r = look<kWeightsGroup>(p, b);
        const int each = seen_groups(r);
        const int h = static_cast<int>((i - seen[b]) / each);
        const int u0 = static_cast<int>((i - seen[b]) - static_cast<long long>(h) * each);
        const int u_end = static_cast<int>(min(static_cast<long long>(each), u0 + (i_end - i)));
        i += u_end - u0;
        const int blocks = (r.T * p.g + 7) / 8;  // of 8 columns
        __syncthreads();  // everybody is done with the columns before
        for (int c = warp; c < blocks; c += kWarps) {
            uint32_t f[D / 8];
            const float undo = load_q<D, E4M3>(p, r, h, 8 * c + quad, f);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) qs[c][s][lane] = make_uint4(f[4 * s], f[4 * s + 1], f[4 * s + 2], f[4 * s + 3]);
            if (lane % 4 == 0) {
                const Column x = column(p, r, h, 8 * c + quad);
                cs[8 * c + quad] = WideColumn{x.bias, E4M3 ? x.mul * undo : x.mul, x.end, x.from};
            }
        }
        __syncthreads();
        for (int u = u0 + warp; u < u_end; u += kWarps) {
            const int j0 = (u < r.sink_end ? u : u - r.sink_end + r.lo) * kWeightsGroup;
            int row;
            const int pg = paged_page(kv, b, j0, row);
            if (pg < 0 || !RA_CHECKED(paged_place_ok(kv, pg, h, row, kWeightsGroup), p.err, kSiteWeightsPlace)) continue;
            const long long place = static_cast<long long>(h) * kv.page + row + quad;
            float* wp = p.w + pg * p.w_ps + place;
            uint4 k[2][kSteps];
            float mul[2], old[2], sum[2] = {0.f, 0.f};
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const char* at = static_cast<const char*>(kv.k) + (pg * kv.k_ps + (place + 8 * m) * D) * (E4M3 ? 1 : 2) + 16 * (lane % 4);
                if (E4M3) {
#pragma unroll
                    for (int s = 0; s < kSteps / 2; ++s) {
                        const uint4 x = ldg128_stream(at + 64 * s);
                        codes_f16(x.x, k[m][2 * s].x, k[m][2 * s].y);
                        codes_f16(x.y, k[m][2 * s].z, k[m][2 * s].w);
                        codes_f16(x.z, k[m][2 * s + 1].x, k[m][2 * s + 1].y);
                        codes_f16(x.w, k[m][2 * s + 1].z, k[m][2 * s + 1].w);
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) k[m][s] = ldg128_stream(at + 64 * s);
                }
                mul[m] = E4M3 ? __ldg(kv.k_scale + pg * kv.ks_ps + place + 8 * m) : 1.f;
                old[m] = faded(p, r, j0 + quad + 8 * m, wp + 8 * m);
            }
            const bool whole = (p.causal ? j0 + kWeightsGroup <= r.s.base + 1 : j0 + kWeightsGroup <= r.s.L) &&
                               (p.window <= 0 || j0 + kWeightsGroup <= p.sinks || j0 > r.s.base + r.T - 1 - p.window);
#pragma unroll 2
            for (int c = 0; c < blocks; ++c) {
                float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const uint4 q = qs[c][s][lane];
                    const uint32_t a0[4] = {k[0][s].x, k[1][s].x, k[0][s].y, k[1][s].y}, a1[4] = {k[0][s].z, k[1][s].z, k[0][s].w, k[1][s].w};
                    mma16816<E4M3>(x, a0, q.x, q.y);
                    mma16816<E4M3>(x, a1, q.z, q.w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const WideColumn& y = cs[8 * c + 2 * (lane % 4) + e % 2];
                    bool on = y.bias != -INFINITY;
                    if (!whole) {
                        const int j = j0 + quad + 8 * (e / 2);
                        on = on && j < y.end && (j >= y.from || j < p.sinks);
                    }
                    const float pr = ex2(fmaf(x[e], E4M3 ? mul[e / 2] * y.mul : kLog2e, -y.bias));
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
    fade_others(p, other, blockIdx.x * static_cast<long long>(kWarps) + warp, gridDim.x * static_cast<long long>(kWarps));
}

template <class K>
int go(K kernel, std::atomic<unsigned long long>& done, const WeightsParams& p, int blocks, cudaStream_t stream) {
    // (sums of up to RINGATTN_PAGED_MAX_BATCH sequences)
    if (!once_a_device(done, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 16 * (kPagedMaxBatch + 1)) == cudaSuccess;
        }))
        return -4;
    kernel<<<blocks, kThreads, 16 * (p.kv.batch + 1), stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <int D, bool E4M3>
int go_cols(const WeightsParams& p, int sms, cudaStream_t stream) {
    static std::atomic<unsigned long long> done[3];
    const int cols = p.max_q * p.g, blocks = blocks_per_sm<E4M3>() * sms;
    if (cols <= 8) return go(weights_kernel<D, E4M3, 1>, done[0], p, blocks, stream);
    if (cols <= 16) return go(weights_kernel<D, E4M3, 2>, done[1], p, blocks, stream);
    return go(weights_wide_kernel<D, E4M3>, done[2], p, kWideBlocks * sms, stream);
}

}  // namespace

int launch_cache_weights_few(const WeightsParams& p, int sms, cudaStream_t stream) {
    if (p.kv.d == 128) return p.kv.e4m3 ? go_cols<128, true>(p, sms, stream) : go_cols<128, false>(p, sms, stream);
    return p.kv.e4m3 ? go_cols<64, true>(p, sms, stream) : go_cols<64, false>(p, sms, stream);
}

}  // namespace ra
