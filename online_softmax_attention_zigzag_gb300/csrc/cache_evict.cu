// cache_evict.cu -- of every sequence's cached positions the keep[b] that stay, for each KV head on its own, and the pages
// packed: K, V, scales and weights of the i-th of them move to position i.
//
// A position's rank: the first `sinks` and the last `recent` before all others, then by weight (a NaN above all
// numbers), of equal ones the lower position first.  As a 32-bit number `order` that is unsigned comparison; the n-th
// largest is found digit by digit (a radix selection: counts of 11, 11 and 10 bits), and everything above it, and the first ones
// that equal it, is listed in order of position.  A cluster of up to eight blocks shares a (sequence, KV head): each holds
// a stretch of its weights in registers, reads the others' counts from their shared memory, and lists its own stretch.
//
// The i-th of the positions that stay is at i or behind it, and they move in order, so packing works in place: what a cluster
// has read of a round of rows before it writes them, it does not need again, and the rows behind lie behind.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "cache_weights.h"
#include "ptx_paged.cuh"

namespace ra {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;  // most blocks of a (sequence, KV head)
constexpr int kSelThreads = 1024;
constexpr int kKeys = 16;  // neighbouring positions of a thread, all on one page
constexpr int kChunk = kKeys * kSelThreads;
constexpr int kDigit = 11;  // bits; 32 = 11 + 11 + 10
constexpr int kBins = 1 << kDigit;
constexpr int kList = 3840;  // keys with the first digit in question that a block lists

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

// The order of positions [j0, j0 + 16), 0 from `end` on (below all others).
__device__ __forceinline__ void load_keys(const EvictParams& p, int b, int h, int L, int j0, int end, uint32_t (&key)[kKeys]) {
#pragma unroll
    for (int e = 0; e < kKeys; ++e) key[e] = 0u;
    if (j0 >= end) return;
    int row;
    const int pg = paged_page(p.kv, b, j0, row);
    const bool ok = pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, h, row, kKeys), p.err, kSiteEvictPlace);
    const float4* w = reinterpret_cast<const float4*>(p.w + (ok ? pg * p.w_ps + static_cast<long long>(h) * p.kv.page + row : 0));
    float4 x[kKeys / 4];
#pragma unroll
    for (int i = 0; i < kKeys / 4; ++i) x[i] = ok ? w[i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int e = 0; e < kKeys; ++e) {
        const int j = j0 + e;
        const float f = e % 4 == 0 ? x[e / 4].x : e % 4 == 1 ? x[e / 4].y : e % 4 == 2 ? x[e / 4].z : x[e / 4].w;
        if (j < end) key[e] = j < p.sinks || j >= L - p.recent ? 0xffffffffu : order(f);
    }
}

// Inclusive sums over a warp.
__device__ __forceinline__ uint32_t warp_scan(uint32_t x) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (static_cast<int>(threadIdx.x % 32) >= d) x += y;
    }
    return x;
}
// Exclusive sums over the block; `total` gets the sum of all.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* sm, uint32_t& total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t s = warp_scan(x);
    if (lane == 31) sm[warp] = s;
    __syncthreads();
    const uint32_t w = warp_scan(sm[lane]);
    const uint32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
    total = __shfl_sync(0xffffffffu, w, 31);
    __syncthreads();
    return s - x + (warp ? before : 0u);
}
// Of 32 counts, one a lane, from the largest digit (lane 0) down: the lane in which the need-th lies, and what it still needs.
__device__ __forceinline__ int find_lane(uint32_t count, uint32_t& need) {
    const uint32_t to = warp_scan(count);
    const int at = max(__ffs(__ballot_sync(0xffffffffu, to >= need)), 1) - 1;
    need -= __shfl_sync(0xffffffffu, to - count, at);
    return at;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ alignas(16) uint32_t hist[3][kBins];  // of this block
    __shared__ alignas(16) uint32_t all[kBins], coarse[32];  // of the cluster; coarse: 64 bins each, the largest first
    __shared__ uint32_t list[kList], listed;
    __shared__ uint32_t sm[32], counts[2];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
    const int head = blockIdx.x / ranks, b = head / p.kv.hkv, h = head - b * p.kv.hkv;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const Sequence s = sequence(p, b);
    launch_dependents();
    int* kept = p.kept + static_cast<long long>(head) * p.max_keep;
    const int first = rank * kSelThreads + threadIdx.x, step = ranks * kSelThreads;
    for (int i = s.n + first; i < p.max_keep; i += step) kept[i] = -1;
    if (s.n == s.L) {
        for (int i = first; i < s.n; i += step) kept[i] = i;
        return;
    }
    if (s.n == 0) return;
    // this block's stretch
    const int each = ((s.L + ranks - 1) / ranks + kKeys - 1) / kKeys * kKeys;
    const int begin = min(s.L, rank * each), end = min(s.L, begin + each);
    const int chunks = (end - begin + kChunk - 1) / kChunk;
    uint32_t key[kKeys];
    auto load = [&](int c) { load_keys(p, b, h, s.L, begin + c * kChunk + kKeys * static_cast<int>(threadIdx.x), end, key); };
    load(0);
    if (threadIdx.x == 0) listed = 0;
    for (int i = threadIdx.x; i < 3 * kBins / 4; i += kSelThreads) reinterpret_cast<uint4*>(&hist[0][0])[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    auto together = [&]() {
        if (ranks > 1) cluster.sync();
        else __syncthreads();
    };
    // the n-th largest: digit by digit, `need` the number still to be taken among those that share the digits so far
    uint32_t prefix = 0, mask = 0, need = static_cast<uint32_t>(s.n);
    bool use_list = false;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass == 2 ? 10 : kDigit, shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digit = (1u << bits) - 1u;
        if (pass == 1) {
            // the keys that are left, mostly few, listed once: looking through all of them for each digit takes 2 us a time
            for (int c = 0; c < chunks; ++c) {
                if (chunks > 1) load(c);
                uint32_t n = 0;
#pragma unroll
                for (int e = 0; e < kKeys; ++e) n += key[e] != 0u && (key[e] & mask) == prefix;
                const uint32_t to = warp_scan(n);
                uint32_t at = 0;
                if (lane == 31 && to > 0) at = atomicAdd(&listed, to);
                at = __shfl_sync(0xffffffffu, at, 31) + to - n;
                if (n > 0) {
#pragma unroll
                    for (int e = 0; e < kKeys; ++e)
                        if (key[e] != 0u && (key[e] & mask) == prefix) {
                            if (at < kList) list[at] = key[e];
                            ++at;
                        }
                }
            }
            __syncthreads();
            use_list = listed <= kList;
        }
        if (use_list) {
            for (uint32_t i = threadIdx.x; i < listed; i += kSelThreads)
                if ((list[i] & mask) == prefix) atomicAdd(&hist[pass][(list[i] >> shift) & digit], 1u);
        } else {
            for (int c = 0; c < chunks; ++c) {
                if (chunks > 1 && (c > 0 || pass > 0)) load(c);
                // (weights that are all the same, zeros above all: additions to one place wait for each other)
                bool same = true;
#pragma unroll
                for (int e = 1; e < kKeys; ++e) same = same && key[e] == key[0];
                if (same) {
                    if (key[0] != 0u && (key[0] & mask) == prefix) atomicAdd(&hist[pass][(key[0] >> shift) & digit], static_cast<uint32_t>(kKeys));
                } else {
#pragma unroll
                    for (int e = 0; e < kKeys; ++e)
                        if (key[e] != 0u && (key[e] & mask) == prefix) atomicAdd(&hist[pass][(key[e] >> shift) & digit], 1u);
                }
            }
        }
        together();
        // warp w: 64 bins of all blocks, the largest of them first; two a lane
        const int at = kBins - 2 - 2 * static_cast<int>(threadIdx.x);
        uint2 x = *reinterpret_cast<const uint2*>(&hist[pass][at]);
        if (ranks > 1) {
            uint2 y[kCluster];
#pragma unroll
            for (int r = 0; r < kCluster; ++r)
                if (r < ranks) y[r] = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&hist[pass][at], r));
            x = make_uint2(0, 0);
#pragma unroll
            for (int r = 0; r < kCluster; ++r)
                if (r < ranks) {
                    x.x += y[r].x;
                    x.y += y[r].y;
                }
        }
        *reinterpret_cast<uint2*>(&all[at]) = x;
        const uint32_t sum = __reduce_add_sync(0xffffffffu, x.x + x.y);
        if (lane == 0) coarse[warp] = sum;
        __syncthreads();
        // every warp for itself: which of the 32, which pair of bins, which of the two
        const int c = find_lane(coarse[lane], need);
        const uint2 y = *reinterpret_cast<const uint2*>(&all[kBins - 2 - 2 * (32 * c + lane)]);
        const int l = find_lane(y.x + y.y, need);
        const uint32_t upper = __shfl_sync(0xffffffffu, y.y, l), lower = __shfl_sync(0xffffffffu, y.x, l);
        const bool in_upper = need <= upper;
        if (!in_upper) need -= upper;
        const int bin = kBins - 1 - 2 * (32 * c + l) - (in_upper ? 0 : 1);
        prefix |= static_cast<uint32_t>(bin) << shift;
        mask |= digit << shift;
        if (need == (in_upper ? upper : lower)) {  // the whole bin stays: no need to look into it
            prefix -= 1u;
            need = 0;
            break;
        }
    }
    // how many of this stretch are above `prefix`, and how many equal it; and of the stretches before
    uint32_t is_above = 0, is_equal = 0;  // of a thread's keys, a bit each
    auto tally = [&]() {  // above in the low half, equal in the high one (a chunk's counts fit)
        is_above = is_equal = 0;
#pragma unroll
        for (int e = 0; e < kKeys; ++e) {
            is_above |= key[e] > prefix ? 1u << e : 0u;
            is_equal |= key[e] == prefix && key[e] != 0u ? 1u << e : 0u;
        }
        return __popc(is_above) | (__popc(is_equal) << 16);
    };
    uint32_t above = 0, equal = 0, total, before = 0;
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) load(c);
        before = block_scan(tally(), sm, total);
        above += total & 0xffffu;
        equal += total >> 16;
    }
    if (ranks > 1) {
        if (threadIdx.x == 0) {
            counts[0] = above;
            counts[1] = equal;
        }
        cluster.sync();
        above = equal = 0;
        for (int r = 0; r < rank; ++r) {
            const uint32_t* x = cluster.map_shared_rank(counts, r);
            above += x[0];
            equal += x[1];
        }
        cluster.barrier_arrive();  // (a block's shared memory has to be there while others read it)
    } else {
        above = equal = 0;
    }
    // in order of position: everything above `prefix`, and the first `need` that equal it
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) {
            load(c);
            before = block_scan(tally(), sm, total);
        }
        const uint32_t a = above + (before & 0xffffu), q = equal + (before >> 16);
        uint32_t at = a + min(q, need);
        const int j0 = begin + c * kChunk + kKeys * static_cast<int>(threadIdx.x);
        uint32_t left = need - min(q, need);  // how many of the thread's equal ones stay
        while (left < static_cast<uint32_t>(__popc(is_equal))) is_equal &= ~(1u << (31 - __clz(is_equal)));
        // (no more than n: weights that another stream changes meanwhile are counted twice and need not agree)
        for (uint32_t stays = is_above | is_equal; stays && at < static_cast<uint32_t>(s.n); stays &= stays - 1u, ++at) kept[at] = j0 + __ffs(stays) - 1;
        above += total & 0xffffu;
        equal += total >> 16;
    }
    if (ranks > 1) cluster.barrier_wait();
}

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;

// One tensor's rows of a sequence and head, PIECES pieces of type T a row: round by round, the cluster's blocks side by side.
template <class T, int PIECES>
__device__ __forceinline__ void move_rows(const EvictParams& p, const int* kept, int b, int h, int n, T* x, long long ps,
                                          const cg::cluster_group& cluster) {
    constexpr int kRows = kMoveThreads / PIECES, kTile = kRows * kMoveUnroll;
    const int piece = threadIdx.x % PIECES, r0 = threadIdx.x / PIECES;
    const int round = kTile * static_cast<int>(cluster.num_blocks()), mine = kTile * static_cast<int>(cluster.block_rank()) + r0;
    T now[kMoveUnroll], next[kMoveUnroll];
    T* to_now[kMoveUnroll];
    T* to_next[kMoveUnroll];
    auto load = [&](long long base, T (&v)[kMoveUnroll], T* (&to)[kMoveUnroll]) {
        int j[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const long long i = base + mine + u * kRows;
            j[u] = i < n ? __ldcg(kept + i) : -1;
        }
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const int i = static_cast<int>(base) + mine + u * kRows;
            to[u] = nullptr;
            v[u] = T{};
            if (j[u] < 0 || j[u] == i) continue;  // (none, or it stays where it is)
            int row;
            int pg = paged_page(p.kv, b, i, row);
            if (pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, h, row), p.err, kSiteEvictPlace))
                to[u] = x + pg * ps + (static_cast<long long>(h) * p.kv.page + row) * PIECES + piece;
            if (!RA_CHECKED(j[u] > i && j[u] < p.kv.max_pages * p.kv.page, p.err, kSiteEvictKept)) continue;
            pg = paged_page(p.kv, b, j[u], row);
            if (pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, h, row), p.err, kSiteEvictPlace))
                v[u] = x[pg * ps + (static_cast<long long>(h) * p.kv.page + row) * PIECES + piece];
        }
    };
    load(0, now, to_now);
    for (long long base = 0; base < n; base += round) {
        load(base + round, next, to_next);
        if (cluster.num_blocks() > 1) cluster.sync();  // everything up to the next round has been read
        else __syncthreads();
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            if (to_now[u]) *to_now[u] = now[u];
            now[u] = next[u];
            to_now[u] = to_next[u];
        }
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kMoveThreads, 2) evict_move_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kPieces = D * (E4M3 ? 1 : 2) / 16;
    const cg::cluster_group cluster = cg::this_cluster();
    const int head = blockIdx.x / cluster.num_blocks(), b = head / p.kv.hkv, h = head - b * p.kv.hkv;
    wait_primary();
    // (len_out may be kv's own lengths: what this block takes from them is the same before and after)
    const int n = sequence(p, b).n;
    const int* kept = p.kept + static_cast<long long>(head) * p.max_keep;
    constexpr int es = E4M3 ? 1 : 2;
    if (blockIdx.y == 0) {
        move_rows<uint4, kPieces>(p, kept, b, h, n, static_cast<uint4*>(p.kv.k), p.kv.k_ps * es / 16, cluster);
    } else if (blockIdx.y == 1) {
        move_rows<uint4, kPieces>(p, kept, b, h, n, static_cast<uint4*>(p.kv.v), p.kv.v_ps * es / 16, cluster);
    } else {
        move_rows<float, 1>(p, kept, b, h, n, p.w, p.w_ps, cluster);
        if (E4M3) {
            move_rows<float, 1>(p, kept, b, h, n, p.kv.k_scale, p.kv.ks_ps, cluster);
            move_rows<float, 1>(p, kept, b, h, n, p.kv.v_scale, p.kv.vs_ps, cluster);
        }
        if (h == 0 && cluster.block_rank() == 0 && threadIdx.x == 0) p.len_out[b] = n;
    }
}

}  // namespace

namespace {
// Blocks of a cluster: a power of two, so many that `heads` clusters come to about `most` blocks, and each has work.
int cluster_of(long long heads, long long most, long long rows, int least) {
    int n = 1;
    while (n < kCluster && 2 * n * heads <= most && rows > static_cast<long long>(n) * least) n *= 2;
    return n;
}

template <class... Args>
cudaError_t launch_clusters(void (*kern)(Args...), dim3 grid, int threads, int cluster, bool dependent, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    // (one block: no cluster, which costs a launch some time)
    cfg.attrs = cluster > 1 ? at : at + 1;
    cfg.numAttrs = (cluster > 1 ? 1 : 0) + (dependent ? 1 : 0);
    return cudaLaunchKernelEx(&cfg, kern, args...);
}
}  // namespace

int launch_cache_evict(const EvictParams& p, int sms, cudaStream_t stream) {
    const long long heads = static_cast<long long>(p.kv.batch) * p.kv.hkv;
    const long long most_len = static_cast<long long>(p.kv.max_pages) * p.kv.page;
    const int sel = cluster_of(heads, sms, most_len, 4096);
    if (launch_clusters(evict_select_kernel, dim3(static_cast<unsigned>(heads * sel)), kSelThreads, sel, false, stream, p) != cudaSuccess) return -4;
    const int mov = cluster_of(2 * heads, 4LL * sms, p.max_keep, 256);
    const dim3 grid(static_cast<unsigned>(heads * mov), 3);
    cudaError_t e;
    if (p.kv.d == 128) e = p.kv.e4m3 ? launch_clusters(evict_move_kernel<128, true>, grid, kMoveThreads, mov, true, stream, p) : launch_clusters(evict_move_kernel<128, false>, grid, kMoveThreads, mov, true, stream, p);
    else e = p.kv.e4m3 ? launch_clusters(evict_move_kernel<64, true>, grid, kMoveThreads, mov, true, stream, p) : launch_clusters(evict_move_kernel<64, false>, grid, kMoveThreads, mov, true, stream, p);
    return e == cudaSuccess ? 0 : -4;
}

}  // namespace ra
