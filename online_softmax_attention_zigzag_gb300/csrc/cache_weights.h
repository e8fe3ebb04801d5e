// cache_weights.h -- parameter blocks and launchers of the attention weights that cached positions have had
// (ringattn_cache_weights) and of eviction by them (ringattn_cache_evict).
#pragma once
#include "paged.h"

namespace ra {

// Sites of the check build (internal.h).
enum WeightsCheckSite : int {
    kSiteWeightsRow = 71,    // a row of q and lse
    kSiteWeightsPlace = 72,  // a position's place in the pool and its weight
    kSiteEvictPlace = 73,    // a place that eviction reads or writes
    kSiteEvictKept = 74      // an entry of the list of kept positions
};

constexpr int kWeightsGroup = 16;  // keys that a warp of the few-row kernel takes at a time, all on one page
constexpr int kWeightsPair = 256;  // keys of an item of the chunk kernel: two tiles
constexpr int kWeightsSumsShared = 224;  // batches up to this keep the chunk kernel's sums in shared memory (what its tiles leave)

// What a block of the chunk kernel leaves of an item whose query rows others have too.
struct WeightsPartial {
    int b, h, pair;  // b < 0: none
    int ends;        // the item's last unit is in it
    float sum[kWeightsPair];
};
// The chunk kernel's part of the workspace: two partial results a block (of the item that it goes on with, and of the
// one that it begins and does not end), the number of pairs that nobody sees, sums of large batches a block.
struct WeightsSpace {
    WeightsPartial part[kPagedMaxShares][2];
    long long others;
    long long sums[kPagedMaxShares][kPagedMaxBatch + 1];
};

struct WeightsParams {
    PagedKV kv;
    const void* q;
    const float* lse;
    float* w;
    long long q_ts, q_hs, l_ts, l_hs, w_ps;
    float decay;
    int hq, g, max_q, causal, window, sinks;
    FastDiv by_g;
    // chunk kernel: tokens of a unit of at most 128 query rows (a power of two, and its exponent), rows of a TMA box of
    // the pool, scratch
    int unit_tokens, unit_log, box_rows;
    int item_units;  // what an item costs beside its units, in units
    WeightsSpace* space;
    unsigned long long timeout_ns;
    int* err;
};

struct EvictParams {
    PagedKV kv;
    float* w;
    long long w_ps;
    const int* keep;  // [batch]
    int* len_out;     // [batch]
    int* kept;        // [batch, Hkv, max_keep]
    int max_keep, sinks, recent;
    int* err;
};

// weights_few
int launch_cache_weights_few(const WeightsParams& p, int sms, cudaStream_t stream);
// any number, g <= 128; maps of K's pool and of q in boxes of a unit's tokens
int launch_cache_weights_chunk(const WeightsParams& p, const CUtensorMap& tk, const CUtensorMap& tq, int shares, cudaStream_t stream);
int launch_cache_evict(const EvictParams& p, int sms, cudaStream_t stream);

// Most rows of a sequence and KV head that the kernels on mma.sync take.  What they do grows with the rows, while the chunk
// kernel does a tile of 128 keys at the cost of 128 rows; in bf16 both wait for K's bytes for long, in e4m3 the chunk kernel waits
// for the warps that expand codes.  16 sequences of 1k to 32k keys, 8 KV heads, us with these and with the chunk kernel:
//   bf16, d = 128: 24 rows 105, 109; 32 rows 134, 112.  d = 64: 24 rows 72, 90; 32 rows 74, 68
//   e4m3, d = 128: 64 rows 141, 191; 80 rows 199, 293; 96 rows 198, 200; 128 rows 300, 255.  d = 64: 80 rows 144, 179; 96 rows 164, 146
// max_q decides for the whole batch, as the rows are on the device: one sequence of 100 rows on 8000 keys takes 63 single tokens
// (200 to 16k keys) along to the chunk kernel, bf16 263 us where two calls take 221, e4m3 526 where they take 155.
constexpr int kWeightsWideRows = 80;
inline bool weights_few(long long rows, bool e4m3) { return rows <= (e4m3 ? kWeightsWideRows : 24); }

#ifdef __CUDACC__
constexpr float kWeightsLog2e = 1.4426950408889634f;

// What the rows of one sequence see, its positions taken `G` at a time ("groups"): groups [0, sink_end) and [lo, hi) hold
// keys that some row sees; those between them only fade, those from hi on start from zero.
struct Seen {
    PagedSeq s;
    int T;  // rows that count
    int keys;  // positions that the last of them may see
    int lo, sink_end, hi, end;
    int fades;  // groups [sink_end, lo) have to be scaled
};

template <int G>
__device__ __forceinline__ Seen look(const WeightsParams& p, int b) {
    Seen r;
    r.s = paged_seq(p.kv, b);
    r.T = min(r.s.T, p.max_q);
    r.keys = r.lo = r.sink_end = r.hi = r.end = r.fades = 0;
    if (r.T <= 0 || r.s.L <= 0) return r;
    r.keys = p.causal ? max(0, min(r.s.L, r.s.base + r.T)) : r.s.L;
    r.hi = (r.keys + G - 1) / G;
    r.end = (r.s.L + G - 1) / G;
    if (p.window > 0) {
        r.lo = min(max(0, r.s.base - p.window + 1) / G, r.hi);
        r.sink_end = min((min(p.sinks, r.keys) + G - 1) / G, r.lo);
        r.fades = p.decay != 1.f;
    }
    return r;
}
__device__ __forceinline__ int seen_groups(const Seen& r) { return r.sink_end + r.hi - r.lo; }
__device__ __forceinline__ int other_groups(const Seen& r) { return (r.fades ? r.lo - r.sink_end : 0) + r.end - r.hi; }
// The u-th of a sequence's groups that nobody sees.
__device__ __forceinline__ int other_group(const Seen& r, int u) {
    const int gap = r.fades ? r.lo - r.sink_end : 0;
    return u < gap ? r.sink_end + u : r.hi + u - gap;
}

// Sums up to every sequence of two counts, sums[0 .. batch], by a block of THREADS threads: f(b, x, y) gives them.
template <int THREADS, class F>
__device__ void sum_up(int batch, long long* xs, long long* ys, F&& f) {
    constexpr int kWarps = THREADS / 32;
    __shared__ long long part[2][kWarps];
    const int each = (batch + THREADS - 1) / THREADS;
    const int b0 = min(batch, static_cast<int>(threadIdx.x) * each), b1 = min(batch, b0 + each);
    long long a = 0, o = 0;
    for (int b = b0; b < b1; ++b) {
        long long x, y;
        f(b, x, y);
        xs[b] = a;
        ys[b] = o;
        a += x;
        o += y;
    }
    // inclusive sums over the warp's lanes, then over the warps
    const long long a0 = a, o0 = o;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, o, d);
        if (static_cast<int>(threadIdx.x) % 32 >= d) {
            a += x;
            o += y;
        }
    }
    if (threadIdx.x % 32 == 31) {
        part[0][threadIdx.x / 32] = a;
        part[1][threadIdx.x / 32] = o;
    }
    __syncthreads();
    for (int w = 0; w < static_cast<int>(threadIdx.x) / 32; ++w) {
        a += part[0][w];
        o += part[1][w];
    }
    if (threadIdx.x == THREADS - 1) {
        xs[batch] = a;
        ys[batch] = o;
    }
    a -= a0;
    o -= o0;
    for (int b = b0; b < b1; ++b) {
        xs[b] += a;
        ys[b] += o;
    }
    __syncthreads();
}

// The sequence that holds number i of a list (sums[b] <= i < sums[b + 1]).
__device__ __forceinline__ int find_sequence(const long long* sums, int batch, long long i) {
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Position j's weight: what is left of the old one.
__device__ __forceinline__ float faded(const WeightsParams& p, const Seen& r, int j, const float* w) {
    return j < r.s.base && p.decay != 0.f ? p.decay * *w : 0.f;
}

// Four e4m3 codes as two pairs of bf16, exact: an e4m3 number's bits, moved to where bf16 has its own, are the number
// times 2^-120 (a subnormal code becomes a subnormal bf16 number).  prmt puts a code into a low byte with its sign all
// over the byte above; 4 bits further up everything is in its place.
__device__ __forceinline__ uint32_t e4m3_bf16(uint32_t codes, uint32_t select) {
    uint32_t x, r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(x) : "r"(codes), "r"(select));
    x = (x << 4) & 0x87f087f0u;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x7b807b80u));  // 2^120
    return r;
}
__device__ __forceinline__ void expand4(uint32_t codes, uint32_t& a, uint32_t& b) {
    a = e4m3_bf16(codes, 0x9180u);
    b = e4m3_bf16(codes, 0xb3a2u);
}
#endif

}  // namespace ra
