// cache_weights_chunk.cu -- ringattn_cache_weights for more than a few query rows of a sequence and KV head: the scores on
// the tcgen05 tensor cores, keys as the rows of the product (M) and query rows as its columns (N).
//
// S = K Q^T puts a key into a TMEM lane: a thread owns one key, reads its scores column by column, and adds up
// exp(s - lse) in a register.  No maximum, no exchange between threads, no second product.  lse differs from column to column:
// read by the threads it is 4 bytes of shared memory for every lane and score, and shared memory, which feeds the products at
// all of its 128 bytes a cycle, was what everything waited for.  So -lse / scale comes out of the product as well, from one more
// step of 16 of its long axis: 1 / scale in three bf16 parts on K's side, -lse in three on q's, all nine products of them.  A unit of
// 256 x 128 scores costs 9 / 8 of 1024 cycles of MMA, and 1024 of the exponential unit at 32 a cycle.
//
// An item is 256 keys of a (sequence, KV head), two tiles, and the units (128 query rows: a power of two of tokens, all heads
// of the group) that see some of them.  All units of all items form one list, sequence by sequence, head by head, pair of
// tiles by pair; a block takes an equal stretch of it.  How many units see a pair is a clamped linear function of the pair,
// so that sums over pairs have closed forms and every role finds its way through the list by itself.  An item that the
// stretches cut leaves partial sums, which a second kernel adds up in the blocks' order.
//
// Roles: sixteen warps add up, four for each tile and half of a unit's columns: both halves' scores leave tensor memory
// at once, so that the next product begins while the exponentials run.  Two warps issue, one a tile; one loads q and makes q's
// share of the last step; one loads K, in e4m3 the codes, which four more warps expand to bf16.  Tensor memory: two accumulators
// of 128 columns a tile.
//
// 4096 rows on 32k keys, 64 query heads, 8 KV heads, d = 128, bf16: 1350 us in ten calls (1456 in long runs, at the power limit),
// 1.53 PFLOP/s of its 2.06 TFLOP; copies of it at 1364: the products alone 1222, without the exponentials 1252.  lse from shared
// memory 1860.  12
// sequences of up to 1023 rows behind up to 9000 keys in e4m3, a window of 2500: 127 us.  Items are short there, and what an item
// costs beside its units (finding it, its pages, two tiles of codes) is what bounds it: 16 sequences of 32 rows 123 us in bf16, 253
// in e4m3, where expanding an item's codes takes longer than its two units.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_weights.h"
#include "ptx_paged.cuh"

namespace ra {
namespace {

constexpr int kTile = kPagedTile;
constexpr int kSumWarps = 16, kMmaWarp = 16, kQWarp = 18, kKWarp = 19, kExpandWarp = 20;
constexpr int kHalf = kTile / 2;  // columns of a warp's share of a unit
// Tiles of q, and in e4m3 of codes, in shared memory.  Of K four in bf16, an item ahead; in e4m3 three and two of codes (two and
// four: the same).  A third tile of q in place of one of K gains little where items are long, and loses more where they are not:
// 4096 rows of 32k 1337 us for 1346, 16 x 32 rows of 1k to 32k keys 147 for 123, in e4m3 276 for 253.
constexpr uint32_t kQSlots = 2, kRawSlots = 2;
constexpr int kAccs = 2, kItems = 4;  // (accumulators of each tile)
constexpr int kBiasBytes = kTile * 32;  // a step of 16 of a product's operand
constexpr uint32_t kTmemCols = 512;

template <int D, bool E4M3>
struct Cfg {
    static constexpr int kThreads = (E4M3 ? 24 : 20) * 32;
    static constexpr uint32_t kKSlots = E4M3 ? 3 : 4, kSlots = kKSlots + kQSlots;
    static constexpr int kTilesOff = kSlots * kBiasBytes;
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kBoxBytes = kTile * 128;  // 64 columns of a tile
    static constexpr int kBoxes = D / 64;
    static constexpr int kRawOff = kTilesOff + kSlots * kTileBytes;
    static constexpr int kRawBytes = kTile * (D + 4);  // codes of a tile, then its scales
    static constexpr int kSumsOff = kRawOff + (E4M3 ? kRawSlots * kRawBytes : 0);
};

// One item of a block's stretch, as its loader hands it to the others.
struct Item {
    int b, h, pair;
    int u0, u1;        // units; none: no more items
    int begins, ends;  // whether the first and the last unit that see the pair are among them
    int T, base, L, keys;
    int page[2][8], row[2][8];  // of the tiles' boxes; page < 0: none
    float scale[kWeightsPair];  // e4m3: of the keys, as held_scale gives them
    int q0;                     // the sequence's first row
};
__device__ __forceinline__ int tiles_of(int pair, int keys) { return pair * kWeightsPair + kTile < keys ? 2 : 1; }

struct Shared {
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t item_raw[kItems], raw_full[kRawSlots], raw_empty[kRawSlots];  // e4m3
    uint64_t k_full[4], k_empty[4], q_full[kQSlots], q_empty[kQSlots], q_landed,
        acc_full[2][kAccs], acc_empty[2][kAccs], half_full[2], half_empty[2], drain[2];
    Item item[kItems];
    float half[2][kTile];  // what the second half of the columns gives a tile's keys
    uint32_t tmem;
    int abort_flag;
};

// ------------------------------------------------------------------ the list of units
__device__ __forceinline__ long long tri(long long n) { return n * (n - 1) / 2; }  // 0 + ... + n - 1

// Units that see some key of a pair p: first(p) .. last(p), for the pairs of a sequence that are seen.
struct Units {
    int n;         // of the sequence
    int step_log;  // units' worth of tokens of a pair: 256 / unit_tokens
    int first0, last0;  // first(p) = max(0, first0 + p step), last(p) = min(n - 1, last0 + p step)
    int whole;     // pairs below this are seen by the last unit (sinks; all without a window)
    int extra;
};
__device__ __forceinline__ Units units_of(const WeightsParams& p, const Seen& r) {
    Units u;
    u.n = (r.T + p.unit_tokens - 1) >> p.unit_log;
    u.step_log = 8 - p.unit_log;
    u.extra = p.item_units;
    // (floor of a token's number by a unit's tokens; a pair's 256 keys are a multiple of those)
    u.first0 = p.causal ? (-r.s.base) >> p.unit_log : INT_MIN / 2;
    u.last0 = static_cast<int>(min((kWeightsPair - 2ll - r.s.base + p.window) >> p.unit_log, 1ll << 30));
    u.whole = p.window > 0 ? (min(p.sinks, r.keys) + kWeightsPair - 1) / kWeightsPair : INT_MAX;
    return u;
}
__device__ __forceinline__ int first_unit(const Units& u, int p) {
    return static_cast<int>(max(0ll, u.first0 + (static_cast<long long>(p) << u.step_log)));
}
__device__ __forceinline__ int last_unit(const Units& u, int p) {
    return p < u.whole ? u.n - 1 : static_cast<int>(min(static_cast<long long>(u.n - 1), u.last0 + (static_cast<long long>(p) << u.step_log)));
}
// Units of the pairs [a, b), all of them seen, with what each pair costs beside.
__device__ long long count_units(const Units& u, int a, int b) {
    if (b <= a) return 0;
    const long long step = 1ll << u.step_log;
    auto from = [&](long long x) {  // the first pair with x + p step >= 0
        const long long q = x >= 0 ? 0 : (-x + step - 1) >> u.step_log;
        return min(max(q, static_cast<long long>(a)), static_cast<long long>(b));
    };
    const long long f = from(u.first0);
    const long long firsts = step * (tri(b) - tri(f)) + u.first0 * (b - f);
    const long long w = min(max(u.whole, a), b);  // [a, w): the last unit
    const long long l = max(w, from(u.last0 - static_cast<long long>(u.n - 1)));
    const long long lasts = (w - a + b - l) * static_cast<long long>(u.n - 1) + step * (tri(l) - tri(w)) + u.last0 * (l - w);
    return lasts - firsts + (1ll + u.extra) * (b - a);
}
__device__ __forceinline__ long long seen_units(const Seen& r, const Units& u) {
    return count_units(u, 0, r.sink_end) + count_units(u, r.lo, r.hi);
}

// A block's stretch, item by item: units [u0, u1) of pair `pair`, of [first, last].  An item takes `extra` places of the list
// before its units: who gets those alone does nothing for it.
struct Walk {
    const long long* sums;
    long long at, end;
    int b, h, pair, v0, u0, u1, first, last;
    long long each;  // places of the sequence and head
    Seen r;
    Units u;
};

__device__ void walk_sequence(const WeightsParams& p, Walk& w) {
    w.b = find_sequence(w.sums, p.kv.batch, w.at);
    w.r = look<kWeightsPair>(p, w.b);
    w.u = units_of(p, w.r);
    w.each = seen_units(w.r, w.u);
}
// The pair's units from place `skip` of it on; false if the stretch ends before the first.
__device__ __forceinline__ bool walk_item(Walk& w, long long skip) {
    w.first = first_unit(w.u, w.pair);
    w.last = last_unit(w.u, w.pair);
    w.v0 = w.first - w.u.extra + static_cast<int>(skip);
    w.u0 = max(w.first, w.v0);
    w.u1 = static_cast<int>(min(static_cast<long long>(w.last + 1), w.v0 + (w.end - w.at)));
    return w.u1 > w.first;
}
// The first item; false if there is none.
__device__ bool walk_begin(const WeightsParams& p, const long long* sums, Walk& w) {
    const long long n = sums[p.kv.batch], each = (n + gridDim.x - 1) / gridDim.x;
    w.sums = sums;
    w.at = min(n, each * blockIdx.x);
    w.end = min(n, w.at + each);
    if (w.at >= w.end) return false;
    walk_sequence(p, w);
    const long long in_seq = w.at - sums[w.b];
    w.h = static_cast<int>(in_seq / w.each);
    long long rest = in_seq - w.h * w.each;
    // the pair: the last one with at most `rest` units before it
    const long long sink = count_units(w.u, 0, w.r.sink_end);
    int lo = 0, hi = w.r.sink_end, from = 0;
    if (rest >= sink) {
        rest -= sink;
        lo = from = w.r.lo;
        hi = w.r.hi;
    }
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (count_units(w.u, from, mid) <= rest) lo = mid;
        else hi = mid;
    }
    w.pair = lo;
    return walk_item(w, rest - count_units(w.u, from, lo));
}
// The next one.
__device__ bool walk_next(const WeightsParams& p, Walk& w) {
    w.at += w.u1 - w.v0;
    if (w.at >= w.end) return false;
    if (++w.pair == w.r.sink_end) w.pair = w.r.lo;
    if (w.pair >= w.r.hi) {
        if (++w.h == p.kv.hkv) {
            walk_sequence(p, w);
            w.h = 0;
        }
        w.pair = w.r.sink_end > 0 ? 0 : w.r.lo;
    }
    return walk_item(w, 0);
}

// ------------------------------------------------------------------ loading
// A slot of a ring: waits until it is free.
__device__ __forceinline__ bool take(uint64_t* empty, uint32_t i, uint32_t n, const WaitCtl& wc) {
    return __all_sync(0xffffffffu, mbar_wait(&empty[i % n], ((i / n) & 1u) ^ 1u, wc, 32));
}
__device__ __forceinline__ void drain_ring(uint64_t* full, uint32_t issued, uint32_t n, const WaitCtl& wc) {
    for (uint32_t s = 0; s < n && s < issued; ++s) {
        const uint32_t last = issued - 1 - ((issued - 1 - s) % n);
        drain_wait(&full[s], (last / n) & 1u, wc.timeout_ns);
    }
}

// A number as three bf16 parts of 8 bits each, in the upper halves of words: all of its 24 bits, unless the last are subnormal.
__device__ __forceinline__ void split3(float x, uint32_t (&part)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        part[i] = __float_as_uint(x) & 0xffff0000u;
        x -= __uint_as_float(part[i]);
    }
}
// (upper halves of two words)
__device__ __forceinline__ uint32_t both_parts(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }
// Row r of an operand's last step, 16 elements without swizzle: 8 rows x 16 bytes lie together, then the next 8 rows; the other
// 8 elements 2048 bytes on.
constexpr uint32_t kBiasStep = 2048;
__device__ __forceinline__ uint32_t bias_row(uint32_t at, int r) { return at + (r / 8) * 128 + (r % 8) * 16; }
// K's: 1 / scale, in parts each three times over.  With q's (-lse in parts, over and over) the step adds -lse / scale to a score.
__device__ __forceinline__ void store_k_bias(uint32_t at, int r, float inv_scale) {
    uint32_t a[3];
    split3(inv_scale, a);
    sts128(bias_row(at, r), both_parts(a[0], a[0]), both_parts(a[0], a[1]), both_parts(a[1], a[1]), both_parts(a[2], a[2]));
    sts128(bias_row(at + kBiasStep, r), a[2] >> 16, 0, 0, 0);
}
// (bf16: 1 / scale is 1, one part, and all but the first three elements stay zero)
template <bool E4M3>
__device__ __forceinline__ void store_q_bias(uint32_t at, int r, float x) {
    uint32_t b[3];
    split3(x, b);
    if constexpr (E4M3) {
        sts128(bias_row(at, r), both_parts(b[0], b[1]), both_parts(b[2], b[0]), both_parts(b[1], b[2]), both_parts(b[0], b[1]));
        sts32(bias_row(at + kBiasStep, r), b[2] >> 16);
    } else {
        sts64(bias_row(at, r), both_parts(b[0], b[1]), b[2] >> 16);
    }
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Inverse scales and lse stay within 2^60, so that no product of their parts leaves fp32: a score of a row with a smaller scale is
// nothing anyhow, and where lse is beyond, fp32 scores are whole trillions apart.
__device__ __forceinline__ float held_scale(float scale) { return scale < 0x1p-60f ? 0x1p-60f : scale; }

// One warp.  The next unit's lse is on its way while a unit is handed on (8 rows of 16 sequences 123 us without, 108 so), and a slot that
// holds the unit already, where only a few see each pair, is handed on as it is (32 rows 140 us without, 123).
// A row whose lse is -inf adds nothing: with zeros in place of its q, and -2^60 for -lse, its weights are 0 whatever it holds (but for
// keys that hold no numbers: `again`).  The loop that sees to such rows (OUT) goes on from unit `first`, where the one that does not
// has come to one and returns false: in one loop 16 sequences of 32 rows in e4m3, none of them such a row, took 270 us, 254 so.
template <int D, bool E4M3, bool OUT>
__device__ __forceinline__ bool q_units(const WeightsParams& p, const CUtensorMap* tq, uint32_t smem, Shared& sh, const long long* sums, const WaitCtl& wc, uint32_t& first) {
    using C = Cfg<D, E4M3>;
    const int lane = threadIdx.x % 32;
    const uint32_t bytes = static_cast<uint32_t>(p.unit_tokens * p.g) * 128u * C::kBoxes;
    const uint64_t keep = make_policy_evict_last();
    const uint32_t q_base = smem + C::kTilesOff + C::kKSlots * C::kTileBytes, b_base = smem + C::kKSlots * kBiasBytes;
    // where a lane's columns lie in a unit
    int token[4];
    long long place[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = lane + 32 * i;
        token[i] = c < p.unit_tokens * p.g ? static_cast<int>(fdiv(static_cast<unsigned>(c), p.by_g)) : INT_MAX / 2;
        place[i] = c < p.unit_tokens * p.g ? token[i] * p.l_ts + (c - token[i] * p.g) * p.l_hs : 0;
    }
    struct Unit {
        int b, h, q0, T, u;
    };
    auto unit = [&](const Walk& w, int u) { return Unit{w.b, w.h, w.r.s.q0, w.r.T, u}; };
    auto load = [&](const Unit& a, float (&x)[4]) {
        const int t0 = a.u << p.unit_log, tokens = a.T - t0;
        const float* from = p.lse + (a.q0 + t0) * p.l_ts + a.h * p.g * p.l_hs;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int head = a.h * p.g + lane + 32 * i - token[i] * p.g;
            x[i] = 0.f;
            if (token[i] < tokens && RA_CHECKED(paged_row_ok(p.kv, p.hq, a.q0 + t0 + token[i], head), p.err, kSiteWeightsRow)) x[i] = __ldg(from + place[i]);
        }
    };
    Walk w = {};
    bool more = walk_begin(p, sums, w), ok = true;
    uint32_t n = 0, landed = 0;
    Unit now = {}, held[2] = {{-1, 0, 0, 0, 0}, {-1, 0, 0, 0, 0}};  // held: what the slots hold, the next one's first
    auto after = [&](const Unit& a) {
        if (a.u + 1 < w.u1) return unit(w, a.u + 1);
        more = walk_next(p, w);
        return more ? unit(w, w.u0) : a;
    };
    float x[4];
    if (more) now = unit(w, w.u0);
    if (OUT)
        for (; n < first && more; ++n) now = after(now);
    if (more) load(now, x);
    while (more) {
        float y[4];
        const Unit next = after(now);
        if (more) load(next, y);
        ok = take(sh.q_empty, n, kQSlots, wc);
        if (!ok) break;
        const uint32_t s = n % kQSlots;
        if (held[0].b != now.b || held[0].h != now.h || held[0].u != now.u) {
            const bool out = __any_sync(0xffffffffu, x[0] == -INFINITY || x[1] == -INFINITY || x[2] == -INFINITY || x[3] == -INFINITY);
            if (!OUT && out) {
                first = n;
                return false;
            }
            uint64_t* bar = OUT && out ? &sh.q_landed : &sh.q_full[s];
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, bytes);
                int tok = now.q0 + (now.u << p.unit_log);
                if (!RA_CHECKED(paged_row_ok(p.kv, p.hq, tok, now.h * p.g + p.g - 1), p.err, kSiteWeightsRow)) tok = 0;
                for (int i = 0; i < C::kBoxes; ++i)
                    tma_load_3d(q_base + s * C::kTileBytes + i * C::kBoxBytes, tq, bar, i * 64, now.h * p.g, tok, keep);
            }
            __syncwarp();
            if (OUT && out) {
                ok = __all_sync(0xffffffffu, mbar_wait(&sh.q_landed, landed & 1u, wc, 32));
                if (!ok) {
                    drain_wait(&sh.q_landed, landed & 1u, wc.timeout_ns);
                    break;
                }
                ++landed;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    for (int k = 0; k < C::kBoxes * 8 && x[i] == -INFINITY; ++k)
                        sts128(q_base + s * C::kTileBytes + k / 8 * C::kBoxBytes + (lane + 32 * i) * 128 + k % 8 * 16, 0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = x[i] == -INFINITY ? -0x1p60f : -x[i];
                store_q_bias<E4M3>(b_base + s * kBiasBytes, lane + 32 * i, v < -0x1p60f ? -0x1p60f : v > 0x1p60f ? 0x1p60f : v);
            }
            fence_async_shared();
            __syncwarp();
            if (OUT && out && lane == 0) mbar_arrive(&sh.q_full[s]);
        } else if (lane == 0) {
            mbar_arrive(&sh.q_full[s]);
        }
        if (lane == 0) mbar_arrive(&sh.q_full[s]);
        held[0] = held[1];
        held[1] = now;
        ++n;
        now = next;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = y[i];
    }
    if (!ok && lane == 0) drain_ring(sh.q_full, n, kQSlots, wc);  // copies in flight land before the block ends
    return true;
}
template <int D, bool E4M3>
__device__ __noinline__ void q_units_out(const WeightsParams& p, const CUtensorMap* tq, uint32_t smem, Shared& sh, const long long* sums, uint32_t first) {
    q_units<D, E4M3, true>(p, tq, smem, sh, sums, WaitCtl{&sh.abort_flag, p.err, p.timeout_ns}, first);
}
template <int D, bool E4M3>
__device__ void q_role(const WeightsParams& p, const CUtensorMap* tq, uint32_t smem, Shared& sh, const long long* sums, const WaitCtl& wc) {
    uint32_t first = 0;
    if (!q_units<D, E4M3, false>(p, tq, smem, sh, sums, wc, first)) q_units_out<D, E4M3>(p, tq, smem, sh, sums, first);
}

// Hands an item on to the warps that issue and add up (null: no more); one warp of the loaders.
__device__ __forceinline__ void describe(Item& it, const Walk* w) {
    if (!w) {
        it.u0 = it.u1 = 0;
        return;
    }
    it.b = w->b;
    it.h = w->h;
    it.pair = w->pair;
    it.u0 = w->u0;
    it.u1 = w->u1;
    it.begins = w->u0 == w->first;
    it.ends = w->u1 == w->last + 1;
    it.q0 = w->r.s.q0;
    it.T = w->r.T;
    it.base = w->r.s.base;
    it.L = w->r.s.L;
    it.keys = w->r.keys;
}

// One warp, a lane a box of rows of one page.  In e4m3 the codes and scales of a tile, as they lie in the pool.
template <int D, bool E4M3>
__device__ void k_role(const WeightsParams& p, const CUtensorMap* tk, uint32_t smem, Shared& sh, const long long* sums, const WaitCtl& wc) {
    using C = Cfg<D, E4M3>;
    constexpr uint32_t kRing = E4M3 ? kRawSlots : C::kKSlots;
    uint64_t* full = E4M3 ? sh.raw_full : sh.k_full;
    uint64_t* empty = E4M3 ? sh.raw_empty : sh.k_empty;
    uint64_t* item_full = E4M3 ? sh.item_raw : sh.item_full;
    const PagedKV& kv = p.kv;
    const int lane = threadIdx.x % 32, rows = p.box_rows, boxes = kTile / rows;
    const uint64_t policy = make_policy_evict_first();
    uint32_t n = 0, ni = 0;
    Walk w;
    // an item's table entries are asked for while the slots for the item before are waited for
    int entry[2], row[2];
    auto look_up = [&]() {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int pos = w.pair * kWeightsPair + k * kTile + lane * rows;
            entry[k] = -1;
            row[k] = 0;
            if (lane < boxes && pos < w.r.s.L) entry[k] = paged_entry(kv, w.b, pos, row[k]);
        }
    };
    bool more = walk_begin(p, sums, w), ok = true;
    if (more) look_up();
    for (; ok; ++ni) {
        ok = take(sh.item_empty, ni, kItems, wc);
        if (!ok) break;
        Item& it = sh.item[ni % kItems];
        int pg[2], y[2];
#pragma unroll
        for (int k = 0; k < 2 && more; ++k) {
            pg[k] = paged_checked(kv, entry[k]);
            if (pg[k] >= 0 && !RA_CHECKED(paged_place_ok(kv, pg[k], w.h, row[k], rows), p.err, kSiteWeightsPlace)) pg[k] = -1;
            y[k] = w.h * kv.page + row[k];
            if (lane < 8) {
                it.page[k][lane] = pg[k];
                it.row[k][lane] = y[k];
            }
        }
        if (lane == 0) describe(it, more ? &w : nullptr);
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_full[ni % kItems]);
        if (!more) break;
        const int tiles = tiles_of(w.pair, w.r.keys);
        more = walk_next(p, w);
        if (more) look_up();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k >= tiles || !ok) continue;
            ok = take(empty, n, kRing, wc);
            if (!ok) continue;
            const uint32_t s = n % kRing;
            ++n;
            if constexpr (E4M3) {
                // (no page: what lies in the slot, since nothing comes of a key that has none, and no other key sees it)
                const uint32_t there = __popc(__ballot_sync(0xffffffffu, pg[k] >= 0));
                if (lane == 0) mbar_arrive_expect_tx(&full[s], there * rows * (D + 4));
                __syncwarp();
                if (pg[k] >= 0) {
                    const uint32_t at = smem + C::kRawOff + s * C::kRawBytes;
                    bulk_load(at + lane * rows * D, static_cast<const uint8_t*>(kv.k) + pg[k] * kv.k_ps + static_cast<long long>(y[k]) * D, rows * D, &full[s], policy);
                    bulk_load(at + kTile * D + lane * rows * 4, kv.k_scale + pg[k] * kv.ks_ps + y[k], rows * 4, &full[s], policy);
                }
            } else {
                if (lane == 0) mbar_arrive_expect_tx(&full[s], C::kTileBytes);
                __syncwarp();
                if (lane < boxes)
                    for (int i = 0; i < C::kBoxes; ++i)  // (no page: zeros)
                        tma_load_3d(smem + C::kTilesOff + s * C::kTileBytes + i * C::kBoxBytes + lane * rows * 128, tk, &full[s], i * 64, y[k], pg[k], policy);
            }
        }
    }
    if (!ok && lane == 0) drain_ring(full, n, kRing, wc);
}

// e4m3: four warps expand a tile's codes, a thread one 16-byte piece of D / 16 rows, and put the scales into the item.
template <int D>
__device__ void expand_role(const WeightsParams& p, uint32_t smem, Shared& sh, const WaitCtl& wc) {
    using C = Cfg<D, true>;
    constexpr int kPieces = D / 16, kRows = 128 / kPieces, kLoads = kTile / kRows;
    const int i0 = threadIdx.x, lane = i0 % 32, piece = i0 % kPieces, r0 = i0 / kPieces;
    uint32_t n = 0;
    for (uint32_t ni = 0;; ++ni) {
        if (!mbar_wait_w(&sh.item_raw[ni % kItems], (ni / kItems) & 1u, wc)) return;
        Item& it = sh.item[ni % kItems];
        const bool none = it.u0 == it.u1;
        const int tiles = none ? 0 : tiles_of(it.pair, it.keys);
        for (int k = 0; k < tiles; ++k, ++n) {
            const uint32_t s = n % kRawSlots, raw = smem + C::kRawOff + s * C::kRawBytes, slot = n % C::kKSlots;
            if (!mbar_wait_w(&sh.raw_full[s], (n / kRawSlots) & 1u, wc)) return;
            const float scale = held_scale(lds32f(raw + kTile * D + i0 * 4));
            uint4 x[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) x[i] = lds128(raw + (i * kRows + r0) * D + piece * 16);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.raw_empty[s]);
            it.scale[k * kTile + i0] = scale;
            if (k == tiles - 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.item_full[ni % kItems]);
            }
            if (!take(sh.k_empty, n, C::kKSlots, wc)) return;
            store_k_bias(smem + slot * kBiasBytes, i0, 1.f / scale);
            const uint32_t stage = smem + C::kTilesOff + slot * C::kTileBytes + (piece / 4) * C::kBoxBytes;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int r = i * kRows + r0;
                uint32_t y[8];
                expand4(x[i].x, y[0], y[1]);
                expand4(x[i].y, y[2], y[3]);
                expand4(x[i].z, y[4], y[5]);
                expand4(x[i].w, y[6], y[7]);
                const uint32_t at = stage + r * 128, c = 2 * (piece % 4);
                sts128(at + ((c ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
                sts128(at + (((c + 1) ^ (r & 7)) << 4), y[4], y[5], y[6], y[7]);
            }
            fence_async_shared();
            mbar_arrive(&sh.k_full[slot]);
        }
        if (none) {
            if (lane == 0) mbar_arrive(&sh.item_full[ni % kItems]);
            return;
        }
    }
}

// Item after item, until there are none (true) or a wait has run out: f(item) returns whether all went well.  Every warp of the
// takers takes every item.
template <class F>
__device__ __forceinline__ bool take_items(Shared& sh, const WaitCtl& wc, F&& f) {
    for (uint32_t n = 0;; ++n) {
        const uint32_t s = n % kItems;
        if (!mbar_wait_w(&sh.item_full[s], (n / kItems) & 1u, wc)) return false;
        const volatile Item& it = sh.item[s];
        if (it.u0 == it.u1) return true;
        if (!f(it)) return false;
        __syncwarp();
        if (threadIdx.x % 32 == 0) mbar_arrive(&sh.item_empty[s]);
    }
}

// ------------------------------------------------------------------ MMA
// Shared-memory matrix descriptor of a K-major operand without swizzle: `lbo` bytes to the next 16 bytes of a row, `sbo` to the
// next 8 rows.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | static_cast<uint64_t>((lbo >> 4) & 0x3fffu) << 16 |
           static_cast<uint64_t>((sbo >> 4) & 0x3fffu) << 32 | 1ull << 46;
}

// S = K Q^T - lse / scale of a tile: 128 keys x n query rows.
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t d_tmem, uint32_t k_base, uint32_t q_base, uint32_t k_bias, uint32_t q_bias, uint32_t idesc) {
    const uint64_t kd = sdesc_sw128(k_base, 16, 1024), qd = sdesc_sw128(q_base, 16, 1024);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * (kTile * 128 >> 4) + (kk % 4) * (32 >> 4);
        mma_ss_e(d_tmem, desc_add(kd, off), desc_add(qd, off), idesc, kk > 0 ? 1u : 0u);
    }
    // last, so that the sums before are rounded at their own size
    mma_ss_e(d_tmem, sdesc_plain(k_bias, kBiasStep, 128), sdesc_plain(q_bias, kBiasStep, 128), idesc, 1u);
}

// One warp a tile: each of an issuer's waits takes 100 to 300 cycles even where its barrier has long completed.
template <int D, bool E4M3>
__device__ void mma_role(const WeightsParams& p, int tile, uint32_t smem, Shared& sh, uint32_t tmem, const WaitCtl& wc) {
    using C = Cfg<D, E4M3>;
    const uint32_t q_base = smem + C::kTilesOff + C::kKSlots * C::kTileBytes, b_base = smem + C::kKSlots * kBiasBytes;
    uint32_t nk = 0, nq = 0, na = 0;
    const bool ok = take_items(sh, wc, [&](const volatile Item& it) -> bool {
        const int tiles = tiles_of(it.pair, it.keys), u1 = it.u1, T = it.T;
        const bool on = tile < tiles;
        const uint32_t slot = (nk + tile) % C::kKSlots;
        // Both tiles: an issuer that does not look at a slot's every round could take one for the next but one.  In e4m3, where
        // tiles come in order, the last one that it looked at shows that the slot's round before is over: its own tile will do.
        for (int k = E4M3 ? min(tile, tiles - 1) : 0; k < (E4M3 ? min(tile + 1, tiles) : tiles); ++k)
            if (!mbar_wait_w(&sh.k_full[(nk + k) % C::kKSlots], ((nk + k) / C::kKSlots) & 1u, wc)) return false;
        nk += tiles;
        for (int u = it.u0; u < u1; ++u, ++nq) {
            const int cols = min(p.unit_tokens, T - (u << p.unit_log)) * p.g;
            const uint32_t idesc = idesc_bf16(kTile, 16, 0) + (static_cast<uint32_t>((cols - 1) / 16 * 2) << 17);  // N: cols, in sixteens
            const uint32_t qs = nq % kQSlots;
            if (on) {
                const uint32_t acc = na % kAccs;
                if (!mbar_wait2_w(&sh.q_full[qs], (nq / kQSlots) & 1u, &sh.acc_empty[tile][acc], ((na / kAccs) & 1u) ^ 1u, wc)) return false;
                ++na;
                tc_fence_after();
                issue_scores<D>(tmem + (tile * kAccs + acc) * kTile, smem + C::kTilesOff + slot * C::kTileBytes, q_base + qs * C::kTileBytes,
                                smem + (E4M3 ? slot * kBiasBytes : 0), b_base + qs * kBiasBytes, idesc);
                mma_commit_e(&sh.acc_full[tile][acc]);
            } else if (!mbar_wait_w(&sh.q_full[qs], (nq / kQSlots) & 1u, wc)) {
                return false;
            }
            mma_commit_e(&sh.q_empty[qs]);
        }
        // (two arrivals a slot; e4m3: its own tile's, but the only one's with the other issuer)
        for (int k = 0; k < tiles; ++k) mma_commit_e(&sh.k_empty[(nk - tiles + (E4M3 && on ? tile : k)) % C::kKSlots]);
        return true;
    });
    if (!ok) {  // every MMA that was issued must finish before TMEM is released
        mma_commit_e(&sh.drain[tile]);
        drain_wait(&sh.drain[tile], 0, wc.timeout_ns);
    }
}

// ------------------------------------------------------------------ the keys' sums
// Adds up 32 columns; all of them are seen.  (s: scores less lse; mul: their scale, to powers of two)
__device__ __forceinline__ void add_block(const uint32_t (&s)[32], float mul, float (&sum)[4]) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        float x[4];
        fmul2(x[0], x[1], __uint_as_float(s[i]), __uint_as_float(s[i + 1]), mul, mul);
        fmul2(x[2], x[3], __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]), mul, mul);
        fadd2(sum[0], sum[1], sum[0], sum[1], ex2(x[0]), ex2(x[1]));
        fadd2(sum[2], sum[3], sum[2], sum[3], ex2(x[2]), ex2(x[3]));
    }
}
// Those among [from, to).
__device__ __forceinline__ void add_some(const uint32_t (&s)[32], float mul, int from, int to, float (&sum)[4]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float x = ex2(__uint_as_float(s[i]) * mul);
        sum[i & 3] += i >= from && i < to ? x : 0.f;
    }
}

// A key that holds an infinity or a NaN makes NaN of a row of zeros as well, so that its sum may be NaN because of rows that add nothing.
// The sums of such keys, one after the other, once more from where q and K lie, a row of the item's units a lane; the others stay.
// (Out of line, and looked for once an item: the times of calls without any stay within 1 %, but for items of few units in e4m3, 16
// sequences of 32 rows 248 us, 254.  Told by a flag from q's loader, unit by unit, 4 % everywhere and 16 % in mixed batches.)
template <int D, bool E4M3>
__device__ __noinline__ float again(const WeightsParams& p, const volatile Item& it, int tile, float total) {
    const int r = threadIdx.x % kTile, lane = threadIdx.x % 32, box_log = 31 - __clz(p.box_rows), T = it.T, q0 = it.q0, h = it.h;
    const int j = it.pair * kWeightsPair + tile * kTile + r, t_from = p.causal ? max(0, j - it.base) : 0;
    const int t_to = p.window > 0 && j >= p.sinks ? static_cast<int>(min(static_cast<long long>(T), static_cast<long long>(j) - it.base + p.window)) : T;
    const float mul = E4M3 ? kWeightsLog2e * it.scale[tile * kTile + r] : kWeightsLog2e;
    const char* key = static_cast<const char*>(p.kv.k);
    bool numbers = true;
    const int pg = it.page[tile][r >> box_log], row = it.row[tile][r >> box_log] + (r & (p.box_rows - 1));
    if (total != total && j < it.L && pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, h, row - h * p.kv.page), p.err, kSiteWeightsPlace)) {
        key += (pg * p.kv.k_ps + static_cast<long long>(row) * D) * (E4M3 ? 1 : 2);
        if (E4M3) numbers = fabsf(mul) < INFINITY;
        else
            for (int e = 0; e < D; ++e) numbers = numbers && (reinterpret_cast<const uint16_t*>(key)[e] & 0x7f80u) != 0x7f80u;
    }
    for (uint32_t bad = __ballot_sync(0xffffffffu, !numbers); bad; bad &= bad - 1u) {
        const int of = __ffs(bad) - 1, from = __shfl_sync(0xffffffffu, t_from, of), to = __shfl_sync(0xffffffffu, t_to, of);
        const char* k = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(key), of));
        const float scale = __shfl_sync(0xffffffffu, mul, of);
        float sum = 0.f;
        for (int u = it.u0; u < it.u1; ++u) {
            for (int c = lane; c < kTile; c += 32) {
                const int in_unit = static_cast<int>(fdiv(static_cast<unsigned>(c), p.by_g)), t = (u << p.unit_log) + in_unit, head = h * p.g + c - in_unit * p.g;
                if (in_unit >= p.unit_tokens || t < from || t >= to || !RA_CHECKED(paged_row_ok(p.kv, p.hq, q0 + t, head), p.err, kSiteWeightsRow)) continue;
                const float lse = __ldg(p.lse + (q0 + t) * p.l_ts + head * p.l_hs);
                if (lse == -INFINITY) continue;
                const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.q) + (q0 + t) * p.q_ts + head * p.q_hs);
                float s = 0.f;
                for (int e = 0; e < D / 2; ++e) {
                    const uint32_t a = __ldg(q + e);
                    float2 b;
                    if (E4M3) {
                        const uint32_t w = e4m3x2_f16x2(reinterpret_cast<const uint16_t*>(k)[e]);
                        b = __half22float2(*reinterpret_cast<const __half2*>(&w));
                    } else {
                        const uint32_t w = reinterpret_cast<const uint32_t*>(k)[e];
                        b = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
                    }
                    s = fmaf(__uint_as_float(a << 16), b.x, s);
                    s = fmaf(__uint_as_float(a & 0xffff0000u), b.y, s);
                }
                sum += ex2(fmaf(s, scale, -lse * kWeightsLog2e));
            }
            if (__any_sync(0xffffffffu, sum != sum)) break;
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == of) total = sum;
    }
    return total;
}

// Four warps: columns [64 half, 64 half + 64) of tile `tile`, a key a thread.
template <int D, bool E4M3>
__device__ void sum_role(const WeightsParams& p, int tile, int half, Shared& sh, uint32_t tmem, const WaitCtl& wc) {
    const int r = threadIdx.x % kTile, lane = threadIdx.x % 32, c0 = half * kHalf, box_log = 31 - __clz(p.box_rows);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(threadIdx.x / 32 % 4 * 32) << 16) + tile * kAccs * kTile + c0;
    uint32_t na = 0, item = 0;
    take_items(sh, wc, [&](const volatile Item& it) -> bool {
        const int T = it.T, u1 = it.u1, base = it.base, j = it.pair * kWeightsPair + tile * kTile + r;
        const bool on = tile < tiles_of(it.pair, it.keys), whole_item = it.begins && it.ends;
        // where the key's weight is, and what it was: asked for now, used after the last unit
        float* wp = nullptr;
        float old = 0.f, total = 0.f;
        const float mul = E4M3 ? kWeightsLog2e * it.scale[tile * kTile + r] : kWeightsLog2e;
        if (half == 0 && j < it.L) {
            const int pg = it.page[tile][r >> box_log], row = it.row[tile][r >> box_log] + (r & (p.box_rows - 1));
            if (pg >= 0 && RA_CHECKED(paged_place_ok(p.kv, pg, it.h, row - it.h * p.kv.page), p.err, kSiteWeightsPlace)) {
                wp = p.w + pg * p.w_ps + row;
                if (whole_item && j < base && p.decay != 0.f) old = *wp;
            }
        }
        // tokens that see the key
        const int t_from = p.causal ? max(0, j - base) : 0;
        const int t_to = p.window > 0 && j >= p.sinks ? static_cast<int>(min(static_cast<long long>(T), static_cast<long long>(j) - base + p.window)) : T;
        for (int u = it.u0; u < u1 && on; ++u, ++na) {
            const int t0 = u << p.unit_log, t1 = min(t0 + p.unit_tokens, T);
            // the share's rows that see the key, and whether all rows see all the warp's keys
            const int from = min(max(t_from - t0, 0), p.unit_tokens) * p.g - c0, to = max(min(t_to, t1) - t0, 0) * p.g - c0;
            const bool all = __all_sync(0xffffffffu, from <= 0 && to >= kHalf);
            const uint32_t acc = na % kAccs;
            if (!mbar_wait_w(&sh.acc_full[tile][acc], (na / kAccs) & 1u, wc)) return false;
            tc_fence_after();
            const uint32_t at = lanes + acc * kTile;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            if (all) {
                // The scores leave tensor memory at once, so that the next product can begin.  (In two halves, the next unit's first
                // one on its way under this one's second, they held it longer: 4096 rows of 32k 1559 us for 1350.)
                uint32_t x[2][32];
                tmem_ld32(at, x[0]);
                tmem_ld32(at + 32, x[1]);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.acc_empty[tile][acc]);
                add_block(x[0], mul, sum);
                add_block(x[1], mul, sum);
            } else {
#pragma unroll 1
                for (int c = 0; c < kHalf; c += 32) {
                    // (a block of columns that sees none of the warp's keys, or all)
                    if (__all_sync(0xffffffffu, from >= c + 32 || to <= c || from >= to)) continue;
                    uint32_t x[32];
                    tmem_ld32(at + c, x);
                    tmem_wait_ld();
                    if (__all_sync(0xffffffffu, from <= c && to >= c + 32)) add_block(x, mul, sum);
                    else add_some(x, mul, from - c, to - c, sum);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.acc_empty[tile][acc]);
            }
            total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        // the halves together
        const uint32_t round = item++ & 1u;
        if (half == 1) {
            if (!mbar_wait_w(&sh.half_empty[tile], round ^ 1u, wc)) return false;
            sh.half[tile][r] = total;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.half_full[tile]);
            return true;
        }
        if (!mbar_wait_w(&sh.half_full[tile], round, wc)) return false;
        total += sh.half[tile][r];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.half_empty[tile]);
        if (__any_sync(0xffffffffu, total != total)) total = again<D, E4M3>(p, it, tile, total);
        if (whole_item) {
            if (wp) *wp = (old != 0.f ? p.decay * old : 0.f) + total;
        } else {
            WeightsPartial& rest = p.space->part[blockIdx.x][it.begins];
            rest.sum[tile * kTile + r] = total;
            if (tile == 0 && r == 0) {
                rest.h = it.h;
                rest.pair = it.pair;
                rest.ends = it.ends;
                rest.b = it.b;
            }
        }
        return true;
    });
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, E4M3>::kThreads, 1) weights_chunk_kernel(const __grid_constant__ WeightsParams p, const __grid_constant__ CUtensorMap tk,
                                                                    const __grid_constant__ CUtensorMap tq) {
    using C = Cfg<D, E4M3>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared sh;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    // (e4m3: the warps that expand come first, who are given way before the others: 8 sequences of 500 to 900 rows 62 us, 61 so;
    // 8192 rows 434, 412)
    const int warp = E4M3 ? (threadIdx.x / 32 + kExpandWarp) % (C::kThreads / 32) : threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < C::kKSlots; ++i) {
            mbar_init(&sh.k_full[i], E4M3 ? 128 : 1);
            mbar_init(&sh.k_empty[i], 2);
        }
        for (uint32_t i = 0; i < kQSlots; ++i) {
            mbar_init(&sh.q_full[i], 2);  // q, and -lse
            mbar_init(&sh.q_empty[i], 2);
        }
        mbar_init(&sh.q_landed, 1);
        for (uint32_t i = 0; i < kRawSlots; ++i) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 4);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_raw[i], 1);
            mbar_init(&sh.item_full[i], E4M3 ? 4 : 1);
            mbar_init(&sh.item_empty[i], kSumWarps + 2);
        }
        for (int i = 0; i < 2; ++i) {
            for (int k = 0; k < kAccs; ++k) {
                mbar_init(&sh.acc_full[i][k], 1);
                mbar_init(&sh.acc_empty[i][k], 8);
            }
            mbar_init(&sh.half_full[i], 4);
            mbar_init(&sh.half_empty[i], 4);
            mbar_init(&sh.drain[i], 1);
        }
        sh.abort_flag = 0;
        p.space->part[blockIdx.x][0].b = p.space->part[blockIdx.x][1].b = -1;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem, kTmemCols);
        tmem_relinquish();
    }
    long long* sums = p.kv.batch <= kWeightsSumsShared ? reinterpret_cast<long long*>(smem + C::kSumsOff) : p.space->sums[blockIdx.x];
    // (the counts of pairs that nobody sees lie where tiles will: only their sum is kept)
    long long* others = p.kv.batch <= kWeightsSumsShared ? sums + kWeightsSumsShared + 1 : reinterpret_cast<long long*>(smem);
    sum_up<C::kThreads>(p.kv.batch, sums, others, [&](int b, long long& x, long long& y) {
        const Seen r = look<kWeightsPair>(p, b);
        x = seen_units(r, units_of(p, r)) * p.kv.hkv;
        y = static_cast<long long>(other_groups(r)) * p.kv.hkv;
    });
    if (blockIdx.x == 0 && threadIdx.x == 0) p.space->others = others[p.kv.batch];
    __syncthreads();  // (others may lie where the tiles will)
    if (!E4M3 && threadIdx.x < kTile) store_k_bias(smem_u32(smem), threadIdx.x, 1.f);
    for (int i = threadIdx.x; i < static_cast<int>(kQSlots) * kBiasBytes / 16; i += C::kThreads)
        sts128(smem_u32(smem) + C::kKSlots * kBiasBytes + 16 * i, 0, 0, 0, 0);
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    launch_dependents();
    const uint32_t tmem = sh.tmem, base = smem_u32(smem);
    const WaitCtl wc{&sh.abort_flag, p.err, p.timeout_ns};
    if (warp < kSumWarps) sum_role<D, E4M3>(p, warp / 8, warp / 4 % 2, sh, tmem, wc);
    else if (warp < kQWarp) mma_role<D, E4M3>(p, warp - kMmaWarp, base, sh, tmem, wc);
    else if (warp == kQWarp) q_role<D, E4M3>(p, &tq, base, sh, sums, wc);
    else if (warp == kKWarp) k_role<D, E4M3>(p, &tk, base, sh, sums, wc);
    else if constexpr (E4M3) expand_role<D>(p, base, sh, wc);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// The items that the stretches cut, each by the block that begins it: the parts in the blocks' order.  And the pairs that
// nobody sees.
__global__ void __launch_bounds__(kWeightsPair) weights_join_kernel(const __grid_constant__ WeightsParams p) {
    extern __shared__ long long both[];
    const PagedKV& kv = p.kv;
    wait_primary();
    const int shares = gridDim.x, x = blockIdx.x, i = threadIdx.x;
    const WeightsPartial& mine = p.space->part[x][1];
    if (mine.b >= 0 && RA_CHECKED(mine.b < kv.batch && mine.h >= 0 && mine.h < kv.hkv && mine.pair >= 0, p.err, kSiteWeightsPlace)) {
        const Seen r = look<kWeightsPair>(p, mine.b);
        float sum = mine.sum[i];
        for (int y = x + 1; y < shares; ++y) {
            const WeightsPartial& part = p.space->part[y][0];
            if (part.b < 0) break;
            sum += part.sum[i];
            if (part.ends) break;
        }
        const int j = mine.pair * kWeightsPair + i;
        if (j < r.s.L) {
            int row;
            const int pg = paged_page(kv, mine.b, j, row);
            if (pg >= 0 && RA_CHECKED(paged_place_ok(kv, pg, mine.h, row), p.err, kSiteWeightsPlace)) {
                float* wp = p.w + pg * p.w_ps + static_cast<long long>(mine.h) * kv.page + row;
                *wp = faded(p, r, j, wp) + sum;
            }
        }
    }
    const long long n = p.space->others;
    if (n == 0) return;
    long long* others = both;
    sum_up<kWeightsPair>(kv.batch, others, both + kv.batch + 1, [&](int b, long long& a, long long& o) {
        a = static_cast<long long>(other_groups(look<kWeightsPair>(p, b))) * kv.hkv;
        o = 0;
    });
    for (long long o = x; o < n; o += shares) {
        const int b = find_sequence(others, kv.batch, o);
        const Seen r = look<kWeightsPair>(p, b);
        const int each = other_groups(r), h = static_cast<int>((o - others[b]) / each);
        const int j = other_group(r, static_cast<int>((o - others[b]) - static_cast<long long>(h) * each)) * kWeightsPair + i;
        if (j >= r.s.L) continue;
        int row;
        const int pg = paged_page(kv, b, j, row);
        if (pg < 0 || !RA_CHECKED(paged_place_ok(kv, pg, h, row), p.err, kSiteWeightsPlace)) continue;
        float* wp = p.w + pg * p.w_ps + static_cast<long long>(h) * kv.page + row;
        *wp = faded(p, r, j, wp);
    }
}

template <int D, bool E4M3>
int launch_t(const WeightsParams& p, const CUtensorMap& tk, const CUtensorMap& tq, int shares, cudaStream_t stream) {
    using C = Cfg<D, E4M3>;
    constexpr int kSmem = C::kSumsOff + 16 * (kWeightsSumsShared + 1) + 1024;
    const auto kernel = weights_chunk_kernel<D, E4M3>;
    static std::atomic<unsigned long long> done{0};
    if (!once_a_device(done, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess &&
                   cudaFuncSetAttribute(weights_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 16 * (kPagedMaxBatch + 1)) == cudaSuccess;
        }))
        return -4;
    kernel<<<shares, C::kThreads, kSmem, stream>>>(p, tk, tq);
    if (cudaGetLastError() != cudaSuccess) return -4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(shares);
    cfg.blockDim = dim3(kWeightsPair);
    cfg.dynamicSmemBytes = 16 * (p.kv.batch + 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weights_join_kernel, p) == cudaSuccess ? 0 : -4;
}

}  // namespace

int launch_cache_weights_chunk(const WeightsParams& p, const CUtensorMap& tk, const CUtensorMap& tq, int shares, cudaStream_t stream) {
    if (p.kv.d == 128) return p.kv.e4m3 ? launch_t<128, true>(p, tk, tq, shares, stream) : launch_t<128, false>(p, tk, tq, shares, stream);
    return p.kv.e4m3 ? launch_t<64, true>(p, tk, tq, shares, stream) : launch_t<64, false>(p, tk, tq, shares, stream);
}

}  // namespace ra
