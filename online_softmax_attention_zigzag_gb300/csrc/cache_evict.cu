// cache_evict.cu -- of every sequence's cached positions the keep[b] that stay, for each KV head on its own, and the pages
// packed: K, V, scales and weights of the i-th of them move to position i.
//
// A position's rank: the first `sinks` and the last `recent` before all others, then by weight (a NaN above all
// numbers), of equal ones the lower position first.  As a 32-bit number `order` that is unsigned comparison; the n-th
// largest is found digit by digit (a radix selection), and one pass in order of position lists who is above it, and the
// first ones that equal it.
//
// The i-th of the positions that stay is at i or behind it, and they move in order, so packing works in place: a block that
// has read the rows of a tile before it writes them overwrites none that it still needs.
#include <cuda_bf16.h>

#include "cache_weights.h"
#include "ptx_paged.cuh"

namespace ra {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelStep = 4 * kSelThreads;  // positions of a step: four neighbours a thread
constexpr int kDigit = 11;                 // bits; 32 = 11 + 11 + 10
constexpr int kBins = 1 << kDigit;

__device__ __forceinline__ uint32_t order(float w) {
    const uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xfffffffeu;  // NaN
    if ((u & 0x7fffffffu) == 0u) return 0x80000000u;          // either zero
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Sequence {
    int L, n;  // positions, and how many of them stay
};
__device__ __forceinline__ Sequence sequence(const EvictParams& p, int b) {
    Sequence s;
    s.L = min(max(__ldg(p.kv.len + b), 0), p.kv.max_pages * p.kv.page);
    s.n = min(s.L, min(max(__ldg(p.keep + b), 0), p.max_keep));
    return s;
}

// Four neighbouring positions' order (0 behind the last: below all others).
__device__ __forceinline__ void load4(const EvictParams& p, int b, int h, int L, int j0, uint32_t (&key)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) key[e] = 0u;
    if (j0 >= L) return;
    int row;
    const int pg = paged_page(p.kv, b, j0, row);
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, h, row, 4), p.err, kSiteEvictPlace))
        w = *reinterpret_cast<const float4*>(p.w + pg * p.w_ps + static_cast<long long>(h) * p.kv.page + row);
    const float x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int j = j0 + e;
        if (j < L) key[e] = j < p.sinks || j >= L - p.recent ? 0xffffffffu : order(x[e]);
    }
}

// Exclusive sums over the block; `total` gets the sum of all.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* sm, uint32_t& total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t s = x;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    if (lane == 31) sm[warp] = s;
    __syncthreads();
    uint32_t w = sm[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += y;
    }
    const uint32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
    total = __shfl_sync(0xffffffffu, w, 31);
    __syncthreads();
    return s - x + (warp ? before : 0u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t sm[32];
    __shared__ uint32_t found[2];
    const int b = blockIdx.x / p.kv.hkv, h = blockIdx.x - b * p.kv.hkv;
    const Sequence s = sequence(p, b);
    launch_dependents();
    int* kept = p.kept + static_cast<long long>(blockIdx.x) * p.max_keep;
    for (int i = s.n + threadIdx.x; i < p.max_keep; i += kSelThreads) kept[i] = -1;
    if (s.n == s.L) {
        for (int i = threadIdx.x; i < s.n; i += kSelThreads) kept[i] = i;
        return;
    }
    if (s.n == 0) return;
    // the n-th largest: digit by digit, `need` the number still to be taken among those that share the digits so far
    uint32_t prefix = 0, mask = 0, need = static_cast<uint32_t>(s.n);
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass == 2 ? 10 : kDigit, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int j0 = 4 * threadIdx.x; j0 < s.L; j0 += kSelStep) {
            uint32_t key[4];
            load4(p, b, h, s.L, j0, key);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j0 + e < s.L && (key[e] & mask) == prefix) atomicAdd(&hist[(key[e] >> shift) & ((1u << bits) - 1u)], 1u);
        }
        __syncthreads();
        // bins from the largest down: thread t has bins kBins - 1 - 2 t and the one below
        const uint32_t hi = hist[kBins - 1 - 2 * threadIdx.x], lo = hist[kBins - 2 - 2 * threadIdx.x];
        uint32_t total;
        const uint32_t before = block_scan(hi + lo, sm, total);
        if (before < need && need <= before + hi + lo) {
            const bool first = need <= before + hi;
            found[0] = kBins - 1 - 2 * threadIdx.x - (first ? 0 : 1);
            found[1] = need - before - (first ? 0u : hi);
        }
        __syncthreads();
        prefix |= found[0] << shift;
        mask |= ((1u << bits) - 1u) << shift;
        need = found[1];
        __syncthreads();
    }
    // in order of position: everything above `prefix`, and the first `need` that equal it
    uint32_t above = 0, equal = 0;
    for (int base = 0; base < s.L; base += kSelStep) {
        uint32_t key[4];
        const int j0 = base + 4 * threadIdx.x;
        load4(p, b, h, s.L, j0, key);
        uint32_t mine = 0;  // above in the low half, equal in the high one
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j0 + e < s.L) mine += key[e] > prefix ? 1u : key[e] == prefix ? 0x10000u : 0u;
        uint32_t total;
        const uint32_t before = block_scan(mine, sm, total);
        uint32_t a = above + (before & 0xffffu), q = equal + (before >> 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (j0 + e >= s.L) continue;
            const bool is_above = key[e] > prefix, is_equal = key[e] == prefix;
            const uint32_t at = a + min(q, need);
            if ((is_above || (is_equal && q < need)) &&
                RA_CHECKED(at < static_cast<uint32_t>(s.n), p.err, kSiteEvictKept))
                kept[at] = j0 + e;
            a += is_above;
            q += is_equal;
        }
        above += total & 0xffffu;
        equal += total >> 16;
    }
}

constexpr int kMoveThreads = 512;
constexpr int kMoveUnroll = 4;

// One tensor's rows of a sequence and head, PIECES pieces of type T a row.
template <class T, int PIECES>
__device__ __forceinline__ void move_rows(const EvictParams& p, const int* kept, int b, int h, int n, T* x, long long ps) {
    constexpr int kRows = kMoveThreads / PIECES, kTile = kRows * kMoveUnroll;
    const int piece = threadIdx.x % PIECES, r0 = threadIdx.x / PIECES;
    T now[kMoveUnroll], next[kMoveUnroll];
    T* to_now[kMoveUnroll];
    T* to_next[kMoveUnroll];
    auto load = [&](int base, T (&v)[kMoveUnroll], T* (&to)[kMoveUnroll]) {
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int i = base + u * kRows + r0;
            to[u] = nullptr;
            v[u] = T{};
            if (i >= n) continue;
            const int j = kept[i];
            if (j == i) continue;  // stays where it is
            int row;
            int pg = paged_page(p.kv, b, i, row);
            if (pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, h, row), p.err, kSiteEvictPlace))
                to[u] = x + pg * ps + (static_cast<long long>(h) * p.kv.page + row) * PIECES + piece;
            if (!RA_CHECKED(j > i && j < p.kv.max_pages * p.kv.page, p.err, kSiteEvictKept)) continue;
            pg = paged_page(p.kv, b, j, row);
            if (pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, h, row), p.err, kSiteEvictPlace))
                v[u] = x[pg * ps + (static_cast<long long>(h) * p.kv.page + row) * PIECES + piece];
        }
    };
    load(0, now, to_now);
    for (int base = 0; base < n; base += kTile) {
        load(base + kTile, next, to_next);
        __syncthreads();  // everything up to the next tile has been read
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            if (to_now[u]) *to_now[u] = now[u];
            now[u] = next[u];
            to_now[u] = to_next[u];
        }
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kPieces = D * (E4M3 ? 1 : 2) / 16;
    const int b = blockIdx.x / p.kv.hkv, h = blockIdx.x - b * p.kv.hkv;
    wait_primary();
    // (len_out may be kv's own lengths: what this block takes from them is the same before and after)
    const int n = sequence(p, b).n;
    const int* kept = p.kept + static_cast<long long>(blockIdx.x) * p.max_keep;
    constexpr int es = E4M3 ? 1 : 2;
    if (blockIdx.y == 0) {
        move_rows<uint4, kPieces>(p, kept, b, h, n, static_cast<uint4*>(p.kv.k), p.kv.k_ps * es / 16);
    } else if (blockIdx.y == 1) {
        move_rows<uint4, kPieces>(p, kept, b, h, n, static_cast<uint4*>(p.kv.v), p.kv.v_ps * es / 16);
    } else {
        move_rows<float, 1>(p, kept, b, h, n, p.w, p.w_ps);
        if (E4M3) {
            move_rows<float, 1>(p, kept, b, h, n, p.kv.k_scale, p.kv.ks_ps);
            move_rows<float, 1>(p, kept, b, h, n, p.kv.v_scale, p.kv.vs_ps);
        }
        if (h == 0 && threadIdx.x == 0) p.len_out[b] = n;
    }
}

}  // namespace

int launch_cache_evict(const EvictParams& p, int sms, cudaStream_t stream) {
    (void)sms;
    const unsigned heads = static_cast<unsigned>(p.kv.batch) * static_cast<unsigned>(p.kv.hkv);
    evict_select_kernel<<<heads, kSelThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return -4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(heads, 3);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (p.kv.d == 128) e = p.kv.e4m3 ? cudaLaunchKernelEx(&cfg, evict_move_kernel<128, true>, p) : cudaLaunchKernelEx(&cfg, evict_move_kernel<128, false>, p);
    else e = p.kv.e4m3 ? cudaLaunchKernelEx(&cfg, evict_move_kernel<64, true>, p) : cudaLaunchKernelEx(&cfg, evict_move_kernel<64, false>, p);
    return e == cudaSuccess ? 0 : -4;
}

}  // namespace ra
