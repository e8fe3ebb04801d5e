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
//
// 16 sequences of 4k to 16k positions, 8 KV heads, 2k kept, bf16: 68 us out of a flushed L2 (64 without), 4.1 TB/s of what it has to
// read and write.  Selecting is a chain of latencies (three digits and a list, each with two exchanges in the cluster); packing takes
// 46, about what a plain gather of such rows does, 256 bytes one in eight.  One sequence of 128k in e4m3, 16k kept: 46 us,
// selecting 19, then rounds in which blocks of a cluster wait for each other; 64k kept in bf16 144, 3.8 TB/s.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "cache_weights.h"
#include "ptx_paged.cuh"

namespace ra {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;  // most blocks of a (sequence, KV head)
constexpr int kKeys = 16;  // neighbouring positions of a thread, all on one page
constexpr int kDigit = 11;  // bits; 32 = 11 + 11 + 10
constexpr int kBins = 1 << kDigit;
constexpr int kDirect = 512;  // as many keys that are left after the first digit are ranked one against the other
constexpr int kList = 5119;  // as many keys with the first digit in question a block lists

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

// The order of positions [j0, j0 + kKeys), 0 from `end` on (below all others).
__device__ __forceinline__ void load_keys(const EvictParams& p, int b, int h, int L, int j0, int end, uint32_t (&key)[kKeys]) {
#pragma unroll
    for (int e = 0; e < kKeys; ++e) key[e] = 0u;
    if (j0 >= end) return;
    const float4* w[kKeys / 16];
    bool ok[kKeys / 16];
#pragma unroll
    for (int g = 0; g < kKeys / 16; ++g) {
        int row = 0;
        const int pg = j0 + 16 * g < end ? paged_page(p.kv, b, j0 + 16 * g, row) : -1;
        ok[g] = pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, h, row, 16), p.err, kSiteEvictPlace);
        w[g] = reinterpret_cast<const float4*>(p.w + (ok[g] ? pg * p.w_ps + static_cast<long long>(h) * p.kv.page + row : 0));
    }
    float4 x[kKeys / 4];
#pragma unroll
    for (int i = 0; i < kKeys / 4; ++i) x[i] = ok[i / 4] ? w[i / 4][i % 4] : make_float4(0.f, 0.f, 0.f, 0.f);
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
template <int THREADS>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* sm, uint32_t& total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t s = warp_scan(x);
    if (lane == 31) sm[warp] = s;
    __syncthreads();
    const uint32_t w = warp_scan(lane < THREADS / 32 ? sm[lane] : 0u);
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

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_select_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kWarps = THREADS / 32, kChunk = kKeys * THREADS;
    // this block's counts, the cluster's, the keys that are left; at the end the positions that stay
    struct Counts {
        uint32_t hist[3][kBins], list[kList + 1];  // (the last place of the list: for those that are not)
    };
    __shared__ alignas(16) Counts counts;
    // sums of 64 bins each, the largest first: this block's, the cluster's, and the cluster's counts of the 64 in question
    __shared__ alignas(8) uint32_t coarse[3][32], all_coarse[3][32], fine[3][64];
    __shared__ uint32_t sm[kWarps], listed, stretch[2];
    auto& hist = counts.hist;
    auto& list = counts.list;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
    const int head = blockIdx.x / ranks, b = head / p.kv.hkv, h = head - b * p.kv.hkv;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const Sequence s = sequence(p, b);
    launch_dependents();
    int* kept = p.kept + static_cast<long long>(head) * p.max_keep;
    const int first = rank * THREADS + threadIdx.x, step = ranks * THREADS;
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
    if (threadIdx.x < 96) (&all_coarse[0][0])[threadIdx.x] = 0;
    if (threadIdx.x < 192) (&fine[0][0])[threadIdx.x] = 0;
    for (int i = threadIdx.x; i < 3 * kBins / 4; i += THREADS) reinterpret_cast<uint4*>(&hist[0][0])[i] = make_uint4(0, 0, 0, 0);
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
                if (__any_sync(0xffffffffu, n > 0)) {
#pragma unroll
                    for (int e = 0; e < kKeys; ++e) {  // (without branches: sixteen of them took 5000 cycles)
                        const bool on = key[e] != 0u && (key[e] & mask) == prefix;
                        list[on ? min(at, static_cast<uint32_t>(kList)) : kList] = key[e];
                        at += on;
                    }
                }
            }
            __syncthreads();
            use_list = listed <= kList;
            if (ranks == 1 && listed <= kDirect) {
                // so few that each is ranked against all: a warp one after the other (two digits more would take 4 us)
                for (uint32_t i = warp; i < listed; i += kWarps) {
                    const uint32_t mine = list[i];
                    uint32_t both = 0;  // above in the low half, equal in the high one
                    for (uint32_t j = lane; j < listed; j += 32) both += list[j] > mine ? 1u : list[j] == mine ? 0x10000u : 0u;
                    both = __reduce_add_sync(0xffffffffu, both);
                    const uint32_t more = both & 0xffffu, as_much = both >> 16;
                    if (more < need && need <= more + as_much && lane == 0) {  // (equal ones all write the same)
                        stretch[0] = mine;
                        stretch[1] = need - more;
                    }
                }
                __syncthreads();
                prefix = stretch[0];
                need = stretch[1];
                break;
            }
        }
        if (use_list) {
            for (uint32_t i = threadIdx.x; i < listed; i += THREADS)
                if ((list[i] & mask) == prefix) atomicAdd(&hist[pass][(list[i] >> shift) & digit], 1u);
        } else {
            for (int c = 0; c < chunks; ++c) {
                if (chunks > 1 && (c > 0 || pass > 0)) load(c);
                // (weights that are all the same, zeros above all: additions to one place wait for each other)
                bool same = true, whole = pass == 0;
#pragma unroll
                for (int e = 0; e < kKeys; ++e) {
                    same = same && key[e] == key[0];
                    whole = whole && key[e] != 0u;
                }
                if (same) {
                    if (key[0] != 0u && (key[0] & mask) == prefix) atomicAdd(&hist[pass][(key[0] >> shift) & digit], static_cast<uint32_t>(kKeys));
                } else if (whole) {
#pragma unroll
                    for (int e = 0; e < kKeys; ++e) atomicAdd(&hist[0][key[e] >> 21], 1u);
                } else {
#pragma unroll
                    for (int e = 0; e < kKeys; ++e)
                        if (key[e] != 0u && (key[e] & mask) == prefix) atomicAdd(&hist[pass][(key[e] >> shift) & digit], 1u);
                }
            }
        }
        __syncthreads();
        constexpr int kBinsEach = kBins / THREADS, kLanes = 64 / kBinsEach;  // of a thread; threads that have 64 together
        static_assert(kBins == 32 * 64 && kLanes <= 32, "32 sums of 64 bins");
        uint32_t sum = 0;
#pragma unroll
        for (int e = 0; e < kBinsEach; e += 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(&hist[pass][kBins - kBinsEach * (static_cast<int>(threadIdx.x) + 1) + e]);
            sum += x.x + x.y;
        }
#pragma unroll
        for (int d = 1; d < kLanes; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane % kLanes == 0) coarse[pass][threadIdx.x / kLanes] = sum;
        together();
        // of the other blocks' counts only what is needed: first the sums, then the 64 in question (all 2048 of eight blocks took
        // 4500 cycles, three times over)
        if (warp < ranks) atomicAdd(&all_coarse[pass][lane], ranks > 1 ? *cluster.map_shared_rank(&coarse[pass][lane], warp) : coarse[pass][lane]);
        __syncthreads();
        const int c = find_lane(all_coarse[pass][lane], need);
        if (warp < ranks) {
            const uint32_t* y = &hist[pass][kBins - 2 - 2 * (32 * c + lane)];
            const uint2 z = *reinterpret_cast<const uint2*>(ranks > 1 ? cluster.map_shared_rank(const_cast<uint32_t*>(y), warp) : y);
            atomicAdd(&fine[pass][2 * lane], z.y);
            atomicAdd(&fine[pass][2 * lane + 1], z.x);
        }
        __syncthreads();
        const uint2 z = *reinterpret_cast<const uint2*>(&fine[pass][2 * lane]);
        const int l = find_lane(z.x + z.y, need);
        uint32_t count = __shfl_sync(0xffffffffu, z.x, l);
        int bin = kBins - 1 - 2 * (32 * c + l);
        if (need > count) {
            need -= count;
            count = __shfl_sync(0xffffffffu, z.y, l);
            --bin;
        }
        prefix |= static_cast<uint32_t>(bin) << shift;
        mask |= digit << shift;
        if (need == count) {  // the whole bin stays: no need to look into it
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
        before = block_scan<THREADS>(tally(), sm, total);
        above += total & 0xffffu;
        equal += total >> 16;
    }
    if (ranks > 1) {
        if (threadIdx.x == 0) {
            stretch[0] = above;
            stretch[1] = equal;
        }
        cluster.sync();
        above = equal = 0;
        uint32_t x[kCluster][2];
#pragma unroll
        for (int r = 0; r < kCluster; ++r)
            if (r < rank) {
                x[r][0] = *cluster.map_shared_rank(&stretch[0], r);
                x[r][1] = *cluster.map_shared_rank(&stretch[1], r);
            }
#pragma unroll
        for (int r = 0; r < kCluster; ++r)
            if (r < rank) {
                above += x[r][0];
                equal += x[r][1];
            }
        cluster.barrier_arrive();  // (a block's shared memory has to be there while others read it)
    } else {
        above = equal = 0;
    }
    // in order of position: everything above `prefix`, and the first `need` that equal it; through shared memory, as
    // neighbours in the list come from threads far apart (written straight to it they took 5 us)
    uint32_t* stage = &counts.hist[0][0];
    constexpr uint32_t kStage = sizeof(Counts) / 4;
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) {
            load(c);
            before = block_scan<THREADS>(tally(), sm, total);
        }
        const uint32_t a = above + (before & 0xffffu), q = equal + (before >> 16), from = above + min(equal, need);
        above += total & 0xffffu;
        equal += total >> 16;
        const uint32_t stays_here = above + min(equal, need) - from;
        uint32_t at = a + min(q, need) - from;
        const int j0 = begin + c * kChunk + kKeys * static_cast<int>(threadIdx.x);
        const uint32_t left = need - min(q, need);  // how many of the thread's equal ones stay
        while (left < static_cast<uint32_t>(__popc(is_equal))) is_equal &= ~(1u << (31 - __clz(is_equal)));
        uint32_t stays = is_above | is_equal;
        // (no more than n: weights that another stream changes meanwhile are counted twice and need not agree)
        if (stays_here <= kStage) {
            for (; stays && at < kStage; stays &= stays - 1u, ++at) stage[at] = j0 + __ffs(stays) - 1;
            __syncthreads();
            for (uint32_t i = threadIdx.x; i < stays_here && from + i < static_cast<uint32_t>(s.n); i += THREADS) kept[from + i] = stage[i];
            __syncthreads();
        } else {
            for (; stays && from + at < static_cast<uint32_t>(s.n); stays &= stays - 1u, ++at) kept[from + at] = j0 + __ffs(stays) - 1;
        }
    }
    if (ranks > 1) cluster.barrier_wait();
}

constexpr int kMoveThreads = 256;
// Blocks of an SM, and rounds in shared memory.  The first case above and the second, us: 3 of 4 65, 46; 4 of 3 74, 46; 2 of 6 67, 55;
// through registers, a round ahead, 109, 54.
constexpr int kMoveBlocks = 3;
constexpr int kMoveStages = 4;
constexpr int kMoveUnroll = 4;  // pieces of 16 bytes of a thread and round, at most

struct MoveShared {
    uint4 piece[kMoveStages][kMoveUnroll][kMoveThreads];
    long long to[kMoveStages][kMoveThreads];  // where a round's rows go, a warp's 32 together; -1: nowhere
};

// One tensor's rows of a sequence and head, PIECES pieces of 16 bytes a row, of which this block moves those from `slice` of
// SLICES on: round by round, the cluster's blocks side by side, a few rounds on their way to shared memory while one is written.  A
// thread writes the pieces that it has loaded.  Where rows lie and go is found by a lane a row, for 32 of a warp's rows at once.
template <int PIECES, int SLICES>
__device__ __forceinline__ void move_rows(const EvictParams& p, const int* kept, int b, int h, int n, uint4* x, long long ps, int slice,
                                          MoveShared& sh, const cg::cluster_group& cluster) {
    constexpr int kLanes = PIECES / SLICES;    // of a row
    constexpr int kRows = 32 / kLanes;         // of a warp and step
    constexpr int kSteps = kLanes < 4 ? kLanes : kMoveUnroll;  // of a round
    constexpr int kRound = kSteps * kRows, kRounds = 32 / kRound;  // of a warp's rows; of a look-up
    static_assert(kRound * kRounds == 32, "32 rows a look-up");
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, piece = slice * kLanes + lane % kLanes;
    const int block = kRound * kMoveThreads / 32, ranks = static_cast<int>(cluster.num_blocks());
    const int mine = block * static_cast<int>(cluster.block_rank()) + warp * kRound;
    const long long all = (static_cast<long long>(n) + static_cast<long long>(block) * ranks - 1) / (static_cast<long long>(block) * ranks);
    const int rounds = static_cast<int>(all);
    // the lane's row of the look-up that begins with round `r`
    auto row_of = [&](int r) { return static_cast<long long>(r + lane / kRound) * block * ranks + mine + lane % kRound; };
    auto kept_at = [&](int r) {
        const long long i = row_of(r);
        return i < n ? __ldcg(kept + i) : -1;
    };
    long long from = -1, to = -1;  // of this look-up's rows; from -1: zeros, to -1: nowhere
    int j = kept_at(0);
    auto look_up = [&](int r) {
        const int i = static_cast<int>(row_of(r));
        from = to = -1;
        if (j >= 0 && j != i) {  // (it stays where it is)
            int row;
            int pg = paged_page(p.kv, b, i, row);
            if (pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, h, row), p.err, kSiteEvictPlace))
                to = pg * ps + (static_cast<long long>(h) * p.kv.page + row) * PIECES;
            if (RA_CHECKED(j > i && j < p.kv.max_pages * p.kv.page, p.err, kSiteEvictKept)) {
                pg = paged_page(p.kv, b, j, row);
                if (pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, h, row), p.err, kSiteEvictPlace))
                    from = pg * ps + (static_cast<long long>(h) * p.kv.page + row) * PIECES;
            }
        }
        j = kept_at(r + kRounds);
    };
    auto load = [&](int r) {
        if (r < rounds) {
            if (r % kRounds == 0) look_up(r);
            const int s = r % kMoveStages, first = r % kRounds * kRound;
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int of = first + u * kRows + lane / kLanes;
                const long long f = __shfl_sync(0xffffffffu, from, of), t = __shfl_sync(0xffffffffu, to, of);
                if (t >= 0) copy16_async(smem_u32(&sh.piece[s][u][threadIdx.x]), x + max(f, 0ll) + piece, f >= 0);
            }
            if (lane / kRound == r % kRounds) sh.to[s][warp * 32 + lane % kRound] = to;
        }
        copies_commit();
    };
#pragma unroll 1
    for (int r = 0; r < kMoveStages - 1; ++r) load(r);
    if (ranks > 1) {
        copies_wait<kMoveStages - 2>();
        cluster.barrier_arrive();
    }
#pragma unroll 1
    for (int r = 0; r < rounds; ++r) {
        // everything up to this round has been read; that the next one has, a cluster's block says before it writes this one (128k
        // positions to 64k in bf16 187 us with a barrier a round in one piece, 142 so)
        if (ranks > 1) {
            cluster.barrier_wait();
            copies_wait<kMoveStages - 3>();
            cluster.barrier_arrive();
        } else {
            copies_wait<kMoveStages - 2>();
            __syncthreads();
        }
        const int s = r % kMoveStages;
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const long long t = sh.to[s][warp * 32 + u * kRows + lane / kLanes];
            if (t >= 0) x[t + piece] = sh.piece[s][u][threadIdx.x];
        }
        __syncwarp();
        load(r + kMoveStages - 1);
    }
    if (ranks > 1) cluster.barrier_wait();
}

// The same for N tensors of one number a row, whose places are looked up once.
struct Numbers {
    float* x;
    long long ps;
};
template <int N>
__device__ __forceinline__ void move_numbers(const EvictParams& p, const int* kept, int b, int h, int n, const Numbers (&x)[N],
                                             const cg::cluster_group& cluster) {
    constexpr int kUnroll = N > 1 ? 4 : 8, kTile = kMoveThreads * kUnroll;
    const int round = kTile * static_cast<int>(cluster.num_blocks()), mine = kTile * static_cast<int>(cluster.block_rank()) + static_cast<int>(threadIdx.x);
    for (long long base = 0; base < n; base += round) {
        float v[N][kUnroll];
        float* to[N][kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long i = base + mine + u * kMoveThreads;
            const int j = i < n ? __ldcg(kept + i) : -1;
            int row, from_row;
            int dst = -1, src = -1;
            if (j >= 0 && j != static_cast<int>(i) && RA_CHECKED(j > i && j < p.kv.max_pages * p.kv.page, p.err, kSiteEvictKept)) {
                dst = paged_page(p.kv, b, static_cast<int>(i), row);
                src = paged_page(p.kv, b, j, from_row);
                if (dst >= 0 && !RA_CHECKED(paged_place_ok(p.kv, dst, h, row), p.err, kSiteEvictPlace)) dst = -1;
                if (src >= 0 && !RA_CHECKED(paged_place_ok(p.kv, src, h, from_row), p.err, kSiteEvictPlace)) src = -1;
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                v[k][u] = src >= 0 ? x[k].x[src * x[k].ps + static_cast<long long>(h) * p.kv.page + from_row] : 0.f;
                to[k][u] = dst >= 0 ? x[k].x + dst * x[k].ps + static_cast<long long>(h) * p.kv.page + row : nullptr;
            }
        }
        if (cluster.num_blocks() > 1) cluster.sync();
        else __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (to[k][u]) *to[k][u] = v[k][u];
        // (what is written now lies before what the next round reads)
    }
}

// blockIdx.y: slices of K, then of V, then the weights and scales.
template <int D, bool E4M3, int SLICES>
__global__ void __launch_bounds__(kMoveThreads, kMoveBlocks) evict_move_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ uint4 raw[];
    MoveShared& sh = *reinterpret_cast<MoveShared*>(raw);
    constexpr int es = E4M3 ? 1 : 2, kPieces = D * es / 16;
    const cg::cluster_group cluster = cg::this_cluster();
    const int head = blockIdx.x / cluster.num_blocks(), b = head / p.kv.hkv, h = head - b * p.kv.hkv;
    wait_primary();
    // (len_out may be kv's own lengths: what this block takes from them is the same before and after)
    const int n = sequence(p, b).n, y = blockIdx.y;
    const int* kept = p.kept + static_cast<long long>(head) * p.max_keep;
    if (y < SLICES) {
        move_rows<kPieces, SLICES>(p, kept, b, h, n, static_cast<uint4*>(p.kv.k), p.kv.k_ps * es / 16, y, sh, cluster);
    } else if (y < 2 * SLICES) {
        move_rows<kPieces, SLICES>(p, kept, b, h, n, static_cast<uint4*>(p.kv.v), p.kv.v_ps * es / 16, y - SLICES, sh, cluster);
    } else {
        if constexpr (E4M3) {
            const Numbers x[3] = {{p.w, p.w_ps}, {p.kv.k_scale, p.kv.ks_ps}, {p.kv.v_scale, p.kv.vs_ps}};
            move_numbers<3>(p, kept, b, h, n, x, cluster);
        } else {
            const Numbers x[1] = {{p.w, p.w_ps}};
            move_numbers<1>(p, kept, b, h, n, x, cluster);
        }
        if (h == 0 && cluster.block_rank() == 0 && threadIdx.x == 0) p.len_out[b] = n;
    }
}

}  // namespace

namespace {
// Blocks of a cluster: a power of two, so many that `heads` clusters come to about `most` blocks, and each has work: by the most
// that there may be, since the lengths are on the device.  A table much longer than its sequences costs them some exchanges: one
// of 700 positions, or five of up to 700, 21 us with a table for 128k, 17 with one of their size.
int cluster_of(long long heads, long long most, long long rows, int least) {
    int n = 1;
    while (n < kCluster && 2 * n * heads <= most && rows > static_cast<long long>(n) * least) n *= 2;
    return n;
}

template <class... Args>
cudaError_t launch_clusters(void (*kern)(Args...), dim3 grid, int threads, int smem, int cluster, bool dependent, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
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

template <int D, bool E4M3, int SLICES>
cudaError_t launch_move(const EvictParams& p, dim3 grid, int cluster, cudaStream_t stream) {
    const auto kernel = evict_move_kernel<D, E4M3, SLICES>;
    constexpr int kSmem = sizeof(MoveShared);
    static std::atomic<unsigned long long> done{0};
    if (!once_a_device(done, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess; }))
        return cudaErrorUnknown;
    return launch_clusters(kernel, grid, kMoveThreads, kSmem, cluster, true, stream, p);
}
}  // namespace

int launch_cache_evict(const EvictParams& p, int sms, cudaStream_t stream) {
    const long long heads = static_cast<long long>(p.kv.batch) * p.kv.hkv;
    const long long most_len = static_cast<long long>(p.kv.max_pages) * p.kv.page;
    const int sel = cluster_of(heads, sms, most_len, 4096);
    const dim3 sel_grid(static_cast<unsigned>(heads * sel));
    // Blocks of half the threads, two an SM, where there are many, or where a stretch is no longer than their 8192 keys (512 heads of 8k
    // 236 us, 220 so; 8 heads of 32k 54, 50; but 128 heads of 16k, with one block each, 68, 82).
    const bool half = heads > sms || most_len <= 8192LL * sel;
    if ((half ? launch_clusters(evict_select_kernel<512>, sel_grid, 512, 0, sel, false, stream, p)
             : launch_clusters(evict_select_kernel<1024>, sel_grid, 1024, 0, sel, false, stream, p)) != cudaSuccess)
        return -4;
    // (a cluster's blocks wait for one another every round: 128 heads, two blocks each, 87 us, one 65)
    const int mov = cluster_of(2 * heads, 2LL * sms, p.max_keep, 256);
    // few blocks: rows in two halves, each of which is packed by itself (8 heads of 128k in e4m3, 16k of them kept: 46 us, 55 whole;
    // 128 heads 75, 65)
    const int slices = 2 * heads * mov <= sms ? 2 : 1;
    const dim3 grid(static_cast<unsigned>(heads * mov), 2 * slices + 1);
    cudaError_t e;
#define RA_MOVE(D, E4M3) e = slices == 2 ? launch_move<D, E4M3, 2>(p, grid, mov, stream) : launch_move<D, E4M3, 1>(p, grid, mov, stream)
    if (p.kv.d == 128) {
        if (p.kv.e4m3) RA_MOVE(128, true);
        else RA_MOVE(128, false);
    } else {
        if (p.kv.e4m3) RA_MOVE(64, true);
        else RA_MOVE(64, false);
    }
#undef RA_MOVE
    return e == cudaSuccess ? 0 : -4;
}

}  // namespace ra
