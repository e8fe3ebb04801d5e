// cache_weights_chunk.cu -- ringattn_cache_weights for more than a few query rows of a sequence and KV head: the scores on
// the tcgen05 tensor cores, keys as the rows of the product (M) and query rows as its columns (N).
//
// S = K Q^T puts a key into a TMEM lane: a thread owns one key, reads its scores column by column, and adds up
// exp(s - lse) in a register.  No maximum, no exchange between threads, no second product: a unit of 128 x 128
// scores costs 512 cycles of MMA, and as much of the exponential unit at 32 a cycle.
//
// An item is 256 keys of a (sequence, KV head), two tiles that stay in shared memory, and the units (128 query rows: a power of
// two of tokens, all heads of the group) that see some of them; with one tile an SM would have to take in 64 bytes of q a
// cycle, with two it is 32.  All units of all items form one list, sequence by sequence, head by head, pair of
// tiles by pair; a block takes an equal stretch of it.  How many units see a pair is a clamped linear function of the pair,
// so that sums over pairs have closed forms and every role finds its way through the list by itself.  An item that the
// stretches cut leaves partial sums, which a second kernel adds up in the blocks' order.
//
// Warps: 0-3 the sums of the first tile, 4-7 of the second, 8 issues the MMAs, 9 loads q and lse, 10-13 K (bf16: one of them
// page boxes by TMA; e4m3: all four expand codes).  TMEM: four accumulators of 128 columns, in turn.
#include <cuda_bf16.h>

#include <cstddef>

#include "cache_weights.h"
#include "ptx_paged.cuh"

namespace ra {
namespace {

constexpr int kTile = kPagedTile;
constexpr int kMmaWarp = 8, kQWarp = 9, kKWarp = 10;
constexpr int kThreads = 14 * 32;
constexpr int kKSlots = 3, kQSlots = 3, kBiasSlots = 8, kAccs = 4;
constexpr uint32_t kTmemCols = 512;

template <int D>
struct Cfg {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kBoxBytes = kTile * 128;  // 64 columns of a tile
    static constexpr int kBoxes = D / 64;
    static constexpr int kQOff = kKSlots * kTileBytes;
    static constexpr int kSumsOff = kQOff + kQSlots * kTileBytes;
};

struct Shared {
    uint64_t k_full[kKSlots], k_empty[kKSlots], q_full[kQSlots], q_empty[kQSlots], bias_full[kBiasSlots], bias_empty[kBiasSlots],
        acc_full[kAccs], acc_empty[kAccs], drain;
    alignas(16) float bias[kBiasSlots][kTile];  // -lse in powers of two of a unit's rows; -inf: adds nothing
    int care[kBiasSlots];           // some row of the unit adds nothing
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
};
__device__ __forceinline__ Units units_of(const WeightsParams& p, const Seen& r) {
    Units u;
    u.n = (r.T + p.unit_tokens - 1) >> p.unit_log;
    u.step_log = 8 - p.unit_log;
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
// Units of the pairs [a, b), all of them seen.
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
    return lasts - firsts + (b - a);
}
__device__ __forceinline__ long long seen_units(const Seen& r, const Units& u) {
    return count_units(u, 0, r.sink_end) + count_units(u, r.lo, r.hi);
}

// A block's stretch, item by item: units [u0, u1) of pair `pair`, of [first, last].
struct Walk {
    const long long* sums;
    long long at, end;
    int b, h, pair, u0, u1, first, last;
    long long each;  // units of the sequence and head
    Seen r;
    Units u;
};

__device__ void walk_sequence(const WeightsParams& p, Walk& w) {
    w.b = find_sequence(w.sums, p.kv.batch, w.at);
    w.r = look<kWeightsPair>(p, w.b);
    w.u = units_of(p, w.r);
    w.each = seen_units(w.r, w.u);
}
__device__ __forceinline__ void walk_item(Walk& w, int u0) {
    w.first = first_unit(w.u, w.pair);
    w.last = last_unit(w.u, w.pair);
    w.u0 = u0 < 0 ? w.first : u0;
    w.u1 = static_cast<int>(min(static_cast<long long>(w.last + 1), w.u0 + (w.end - w.at)));
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
    walk_item(w, first_unit(w.u, lo) + static_cast<int>(rest - count_units(w.u, from, lo)));
    return true;
}
// The next one.
__device__ bool walk_next(const WeightsParams& p, Walk& w) {
    w.at += w.u1 - w.u0;
    if (w.at >= w.end) return false;
    if (++w.pair == w.r.sink_end) w.pair = w.r.lo;
    if (w.pair >= w.r.hi) {
        if (++w.h == p.kv.hkv) {
            walk_sequence(p, w);
            w.h = 0;
        }
        w.pair = w.r.sink_end > 0 ? 0 : w.r.lo;
    }
    walk_item(w, -1);
    return true;
}
__device__ __forceinline__ int tiles_of(const Walk& w) { return w.pair * kWeightsPair + kTile < w.r.keys ? 2 : 1; }

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

template <int D>
__device__ void q_role(const WeightsParams& p, const CUtensorMap* tq, uint32_t smem, Shared& sh, const long long* sums, const WaitCtl& wc) {
    using C = Cfg<D>;
    const int lane = threadIdx.x % 32;
    const uint32_t bytes = static_cast<uint32_t>(p.unit_tokens * p.g) * 128u * C::kBoxes;
    const uint64_t keep = make_policy_evict_last();
    uint32_t n = 0;
    Walk w;
    bool ok = true;
    for (bool more = walk_begin(p, sums, w); more && ok; more = walk_next(p, w)) {
        for (int u = w.u0; u < w.u1; ++u, ++n) {
            const int t0 = u << p.unit_log, cols = min(p.unit_tokens, w.r.T - t0) * p.g;
            // the unit's lse, asked for before the wait for its place
            float x[4];
            bool care = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = lane + 32 * i;
                x[i] = -INFINITY;
                if (c >= cols) continue;
                const int t = static_cast<int>(fdiv(static_cast<unsigned>(c), p.by_g)), head = w.h * p.g + c - t * p.g;
                const long long row = w.r.s.q0 + t0 + t;
                if (!RA_CHECKED(paged_row_ok(p.kv, p.hq, row, head), p.err, kSiteWeightsRow)) continue;
                const float lse = __ldg(p.lse + row * p.l_ts + head * p.l_hs);
                x[i] = lse == -INFINITY ? -INFINITY : -lse * kWeightsLog2e;
                care |= x[i] == -INFINITY;
            }
            care = __any_sync(0xffffffffu, care);
            ok = take(sh.q_empty, n, kQSlots, wc);
            if (!ok) break;
            if (lane == 0) {
                const uint32_t s = n % kQSlots;
                mbar_arrive_expect_tx(&sh.q_full[s], bytes);
                int tok = w.r.s.q0 + t0;
                if (!RA_CHECKED(paged_row_ok(p.kv, p.hq, tok, w.h * p.g + p.g - 1), p.err, kSiteWeightsRow)) tok = 0;
                for (int i = 0; i < C::kBoxes; ++i)
                    tma_load_3d(smem + C::kQOff + s * C::kTileBytes + i * C::kBoxBytes, tq, &sh.q_full[s], i * 64, w.h * p.g, tok, keep);
            }
            __syncwarp();
            ok = take(sh.bias_empty, n, kBiasSlots, wc);
            if (!ok) {
                ++n;
                break;
            }
            const uint32_t s = n % kBiasSlots;
#pragma unroll
            for (int i = 0; i < 4; ++i) sh.bias[s][lane + 32 * i] = x[i];
            if (lane == 0) sh.care[s] = care;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.bias_full[s]);
        }
    }
    if (!ok && lane == 0) drain_ring(sh.q_full, n, kQSlots, wc);  // copies in flight land before the block ends
}

// bf16: one warp, a lane a box of rows of one page.
template <int D>
__device__ void k_role(const WeightsParams& p, const CUtensorMap* tk, uint32_t smem, Shared& sh, const long long* sums, const WaitCtl& wc) {
    using C = Cfg<D>;
    const PagedKV& kv = p.kv;
    const int lane = threadIdx.x % 32, rows = p.box_rows, boxes = kTile / rows;
    const uint64_t policy = make_policy_evict_first();
    uint32_t n = 0;
    Walk w;
    bool ok = true;
    for (bool more = walk_begin(p, sums, w); more && ok; more = walk_next(p, w)) {
        const int tiles = tiles_of(w);
        int pg[2], y[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int pos = w.pair * kWeightsPair + k * kTile + lane * rows;
            int row = 0;
            pg[k] = lane < boxes && pos < w.r.keys ? paged_page(kv, w.b, pos, row) : -1;
            if (pg[k] >= 0 && !RA_CHECKED(paged_place_ok(kv, pg[k], w.h, row, rows), p.err, kSiteWeightsPlace)) pg[k] = -1;
            y[k] = w.h * kv.page + row;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k >= tiles) continue;
            ok = take(sh.k_empty, n, kKSlots, wc);
            if (!ok) break;
            const uint32_t s = n % kKSlots;
            ++n;
            if (lane == 0) mbar_arrive_expect_tx(&sh.k_full[s], C::kTileBytes);
            __syncwarp();
            if (lane < boxes)
                for (int i = 0; i < C::kBoxes; ++i)  // (no page: zeros)
                    tma_load_3d(smem + s * C::kTileBytes + i * C::kBoxBytes + lane * rows * 128, tk, &sh.k_full[s], i * 64, y[k], pg[k], policy);
        }
    }
    if (!ok && lane == 0) drain_ring(sh.k_full, n, kKSlots, wc);
}

// e4m3: four warps expand codes, a thread one 16-byte piece of D / 16 rows at a time.  The scales stay with the keys' sums.
template <int D>
__device__ void expand_role(const WeightsParams& p, uint32_t smem, Shared& sh, const long long* sums, const WaitCtl& wc) {
    using C = Cfg<D>;
    constexpr int kPieces = D / 16, kRows = 128 / kPieces, kLoads = kTile / kRows;
    const PagedKV& kv = p.kv;
    const int i0 = threadIdx.x - kKWarp * 32, piece = i0 % kPieces, r0 = i0 / kPieces;
    uint32_t n = 0;
    Walk w;
    for (bool more = walk_begin(p, sums, w); more; more = walk_next(p, w)) {
        const int tiles = tiles_of(w);
        for (int k = 0; k < tiles; ++k, ++n) {
            uint4 x[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int pos = w.pair * kWeightsPair + k * kTile + i * kRows + r0;
                x[i] = make_uint4(0, 0, 0, 0);
                if (pos >= w.r.keys) continue;
                int row;
                const int pg = paged_page(kv, w.b, pos, row);
                if (pg < 0 || !RA_CHECKED(paged_place_ok(kv, pg, w.h, row), p.err, kSiteWeightsPlace)) continue;
                x[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv.k) + pg * kv.k_ps +
                                                            (static_cast<long long>(w.h) * kv.page + row) * D) + piece);
            }
            if (!take(sh.k_empty, n, kKSlots, wc)) return;
            const uint32_t stage = smem + (n % kKSlots) * C::kTileBytes + (piece / 4) * C::kBoxBytes;
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
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(&sh.k_full[n % kKSlots]);
        }
    }
}

// ------------------------------------------------------------------ MMA
// S = K Q^T of a tile: 128 keys x n query rows.
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t d_tmem, uint32_t k_base, uint32_t q_base, uint32_t idesc) {
    const uint64_t kd = sdesc_sw128(k_base, 16, 1024), qd = sdesc_sw128(q_base, 16, 1024);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * (kTile * 128 >> 4) + (kk % 4) * (32 >> 4);
        mma_ss_e(d_tmem, desc_add(kd, off), desc_add(qd, off), idesc, kk > 0 ? 1u : 0u);
    }
}

template <int D>
__device__ void mma_role(const WeightsParams& p, uint32_t smem, Shared& sh, const long long* sums, uint32_t tmem, const WaitCtl& wc) {
    using C = Cfg<D>;
    uint32_t nk = 0, nq = 0, na = 0;
    Walk w;
    bool ok = true;
    for (bool more = walk_begin(p, sums, w); more && ok; more = walk_next(p, w)) {
        const int tiles = tiles_of(w);
        for (int k = 0; k < tiles && ok; ++k) ok = mbar_wait_w(&sh.k_full[(nk + k) % kKSlots], ((nk + k) / kKSlots) & 1u, wc);
        for (int u = w.u0; u < w.u1 && ok; ++u, ++nq) {
            const int cols = min(p.unit_tokens, w.r.T - (u << p.unit_log)) * p.g;
            const uint32_t idesc = idesc_bf16(kTile, 16, 0) + (static_cast<uint32_t>((cols - 1) / 16 * 2) << 17);  // N: cols, in sixteens
            ok = mbar_wait_w(&sh.q_full[nq % kQSlots], (nq / kQSlots) & 1u, wc);
            for (int k = 0; k < tiles && ok; ++k, ++na) {
                ok = mbar_wait_w(&sh.acc_empty[na % kAccs], ((na / kAccs) & 1u) ^ 1u, wc);
                if (!ok) break;
                tc_fence_after();
                issue_scores<D>(tmem + (na % kAccs) * kTile, smem + ((nk + k) % kKSlots) * C::kTileBytes,
                                smem + C::kQOff + (nq % kQSlots) * C::kTileBytes, idesc);
                mma_commit_e(&sh.acc_full[na % kAccs]);
            }
            if (ok) mma_commit_e(&sh.q_empty[nq % kQSlots]);
        }
        if (ok)
            for (int k = 0; k < tiles; ++k) mma_commit_e(&sh.k_empty[(nk + k) % kKSlots]);
        nk += tiles;
    }
    if (!ok) {  // every MMA that was issued must finish before TMEM is released
        mma_commit_e(&sh.drain);
        drain_wait(&sh.drain, 0, wc.timeout_ns);
    }
}

// ------------------------------------------------------------------ the keys' sums
// Adds up 32 columns from c on; all of them are seen.
__device__ __forceinline__ void add_block(const uint32_t (&s)[32], const float* bias, float mul, float (&sum)[4]) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const float4 m = *reinterpret_cast<const float4*>(bias + i);
        float x[4];
        ffma2(x[0], x[1], __uint_as_float(s[i]), __uint_as_float(s[i + 1]), mul, mul, m.x, m.y);
        ffma2(x[2], x[3], __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]), mul, mul, m.z, m.w);
        fadd2(sum[0], sum[1], sum[0], sum[1], ex2(x[0]), ex2(x[1]));
        fadd2(sum[2], sum[3], sum[2], sum[3], ex2(x[2]), ex2(x[3]));
    }
}
// Those among [from, to) whose row adds something.
__device__ __forceinline__ void add_some(const uint32_t (&s)[32], const float* bias, float mul, int from, int to, float (&sum)[4]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float m = bias[i], x = ex2(fmaf(__uint_as_float(s[i]), mul, m));
        sum[i & 3] += i >= from && i < to && m != -INFINITY ? x : 0.f;
    }
}

template <bool E4M3>
__device__ void sum_role(const WeightsParams& p, int tile, Shared& sh, const long long* sums, uint32_t tmem, const WaitCtl& wc) {
    const PagedKV& kv = p.kv;
    const int r = threadIdx.x % kTile, lane = threadIdx.x % 32;
    const uint32_t lanes = static_cast<uint32_t>(threadIdx.x / 32 % 4 * 32) << 16;
    uint32_t nq = 0, na = 0;
    Walk w;
    for (bool more = walk_begin(p, sums, w); more; more = walk_next(p, w)) {
        const int tiles = tiles_of(w);
        const int j0 = w.pair * kWeightsPair + tile * kTile, j = j0 + r;
        // where the key's weight is, what it was, and its scale: used after the last unit, and from the first one on
        float* wp = nullptr;
        float old = 0.f, mul = kWeightsLog2e;
        if (j < w.r.s.L) {
            int row;
            const int pg = paged_page(kv, w.b, j, row);
            if (pg >= 0 && RA_CHECKED(paged_place_ok(kv, pg, w.h, row), p.err, kSiteWeightsPlace)) {
                const long long at = static_cast<long long>(w.h) * kv.page + row;
                wp = p.w + pg * p.w_ps + at;
                if (E4M3 && j < w.r.keys) mul *= __ldg(kv.k_scale + pg * kv.ks_ps + at);
            }
        }
        const bool whole_item = w.u0 == w.first && w.u1 == w.last + 1;
        if (wp && whole_item) old = faded(p, w.r, j, wp);
        // tokens that see the key
        const int t_from = p.causal ? max(0, j - w.r.s.base) : 0;
        auto before = [&](int key) { return static_cast<int>(min(static_cast<long long>(w.r.T), static_cast<long long>(key) - w.r.s.base + p.window)); };
        const int t_to = p.window > 0 && j >= p.sinks ? before(j) : w.r.T;
        // and those that see the whole tile (positions behind the last included: they are not written)
        const int all_from = p.causal ? max(0, j0 + kTile - 1 - w.r.s.base) : 0;
        const int all_to = p.window > 0 && j0 + kTile > p.sinks ? before(max(j0, p.sinks)) : w.r.T;
        float total = 0.f;
        for (int u = w.u0; u < w.u1; ++u, ++nq, na += tiles) {
            const uint32_t slot = nq % kBiasSlots;
            if (!mbar_wait_w(&sh.bias_full[slot], (nq / kBiasSlots) & 1u, wc)) return;
            if (tile < tiles) {
                const int t0 = u << p.unit_log, t1 = min(t0 + p.unit_tokens, w.r.T), cols = (t1 - t0) * p.g;
                const bool whole = t0 >= all_from && t1 <= all_to && !sh.care[slot];
                const int from = min(max(t_from - t0, 0), p.unit_tokens) * p.g, to = max(min(t_to, t1) - t0, 0) * p.g;
                const uint32_t acc = (na + tile) % kAccs;
                if (!mbar_wait_w(&sh.acc_full[acc], ((na + tile) / kAccs) & 1u, wc)) return;
                tc_fence_after();
                const uint32_t at = tmem + lanes + acc * kTile;
                const float* bias = sh.bias[slot];
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                if (whole && cols == kTile) {
                    uint32_t a[32], b[32];
                    tmem_ld32(at, a);
                    tmem_wait_ld();
                    tmem_ld32(at + 32, b);
                    add_block(a, bias, mul, sum);
                    tmem_wait_ld();
                    tmem_ld32(at + 64, a);
                    add_block(b, bias + 32, mul, sum);
                    tmem_wait_ld();
                    tmem_ld32(at + 96, b);
                    add_block(a, bias + 64, mul, sum);
                    tmem_wait_ld();
                    add_block(b, bias + 96, mul, sum);
                } else {
                    for (int c = 0; c < cols; c += 32) {
                        uint32_t a[32];
                        tmem_ld32(at + c, a);
                        tmem_wait_ld();
                        if (whole && c + 32 <= cols) add_block(a, bias + c, mul, sum);
                        else add_some(a, bias + c, mul, from - c, to - c, sum);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.acc_empty[acc]);
                total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            } else {
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&sh.bias_empty[slot]);
        }
        if (whole_item) {
            if (wp) *wp = old + total;
        } else {
            WeightsPartial& part = p.space->part[blockIdx.x][w.u0 == w.first];
            part.sum[tile * kTile + r] = total;
            if (threadIdx.x == 0) {
                part.h = w.h;
                part.pair = w.pair;
                part.ends = w.u1 == w.last + 1;
                part.b = w.b;
            }
        }
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) weights_chunk_kernel(const __grid_constant__ WeightsParams p, const __grid_constant__ CUtensorMap tk,
                                                                    const __grid_constant__ CUtensorMap tq) {
    using C = Cfg<D>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared sh;
    static_assert(offsetof(Shared, bias) % 16 == 0 && alignof(Shared) >= 16, "bias is read four at a time");
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kKSlots; ++i) {
            mbar_init(&sh.k_full[i], E4M3 ? 128 : 1);
            mbar_init(&sh.k_empty[i], 1);
        }
        for (int i = 0; i < kQSlots; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
        }
        for (int i = 0; i < kBiasSlots; ++i) {
            mbar_init(&sh.bias_full[i], 1);
            mbar_init(&sh.bias_empty[i], 8);
        }
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 4);
        }
        mbar_init(&sh.drain, 1);
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
    sum_up<kThreads>(p.kv.batch, sums, others, [&](int b, long long& x, long long& y) {
        const Seen r = look<kWeightsPair>(p, b);
        x = seen_units(r, units_of(p, r)) * p.kv.hkv;
        y = static_cast<long long>(other_groups(r)) * p.kv.hkv;
    });
    if (blockIdx.x == 0 && threadIdx.x == 0) p.space->others = others[p.kv.batch];
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    launch_dependents();
    const uint32_t tmem = sh.tmem, base = smem_u32(smem);
    const WaitCtl wc{&sh.abort_flag, p.err, p.timeout_ns};
    if (warp < 8) {
        sum_role<E4M3>(p, warp / 4, sh, sums, tmem, wc);
    } else if (warp == kMmaWarp) {
        mma_role<D>(p, base, sh, sums, tmem, wc);
    } else if (warp == kQWarp) {
        q_role<D>(p, &tq, base, sh, sums, wc);
    } else if (E4M3) {
        expand_role<D>(p, base, sh, sums, wc);
    } else if (warp == kKWarp) {
        k_role<D>(p, &tk, base, sh, sums, wc);
    }
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
    using C = Cfg<D>;
    constexpr int kSmem = C::kSumsOff + 16 * (kWeightsSumsShared + 1) + 1024;
    const auto kernel = weights_chunk_kernel<D, E4M3>;
    static std::atomic<unsigned long long> done{0};
    if (!once_a_device(done, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess &&
                   cudaFuncSetAttribute(weights_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 16 * (kPagedMaxBatch + 1)) == cudaSuccess;
        }))
        return -4;
    kernel<<<shares, kThreads, kSmem, stream>>>(p, tk, tq);
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
