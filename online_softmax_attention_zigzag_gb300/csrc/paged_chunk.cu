// paged_chunk.cu -- attention of a chunk of new tokens over a paged K/V cache on the tcgen05 tensor
// cores: more rows of a sequence and KV head than the few-row kernel takes.
//
// The mathematics is the ring kernel's (one online softmax over tiles of 128 keys, the running
// max moved only when it is exceeded by 2^8, out = sum of bf16(p) v / sum of bf16(p), lse from the
// unrounded p).  What differs:
//   * rows: a unit is 128 / g tokens times the g query heads of a KV head, so that grouped heads
//     share every K/V tile inside one matrix tile; an item is two units.
//   * keys: tiles come page by page, a TMA box is gcd(page, 128) rows of one page; a tile is read
//     when some row of the item sees a key of it (sinks first, then the window up to the last
//     row's position).
//   * work: items (sequence, KV head, pair of units) are dealt out whole, one round of blocks after
//     the other, so that the blocks work on one or two heads at a time and their K and V stay in L2, as
//     long as no block gets more than an equal share of all tiles; the tiles of the items
//     that are left, in one line, then fill every block up to its share.  An item that lies in several
//     blocks' fillings leaves partial results that a join kernel combines.  Every SM ends
//     within one tile of the others, whatever the lengths are, at the price of at most 2 * 132 KB of
//     partial results a block, about two tiles' time.  The list is made on the device by a
//     one-block kernel, because the lengths are there.
//   * values: a row of P is 0 where a key is hidden, but 0 * NaN is NaN, so tiles that not every
//     row sees whole have their V looked over before the product: rows that nobody sees
//     become zeros, and infinities and NaN become zeros that the rows that do see them add at
//     the end.
//   * e4m3: eight warps expand codes into the bf16 tiles: exponent and mantissa bits moved into
//     place are the value times 2^-120, exact for subnormal codes too, and one packed
//     multiplication by 2^120 * scale finishes it, exact for scales that are powers of two.
//   * long contexts: the tensor cores' sums are moved to memory every 512 tiles (fold_o).
//
//   * calls whose items all have one unit (at most 128 rows a sequence and KV head) have no partner
//     whose softmax would overlap its products: the scores then alternate between the two units' S
//     columns, S(j + 2) is issued behind P V(j), and the softmax goes from tile to tile without
//     waiting for either; half the warps have nothing to do, and the other unit's Q makes room for
//     e4m3 tiles on their way.
//
// What it takes, 64 query and 8 KV heads, d = 128 (the products' floor is the measured 1912 TFLOP/s):
//     4096 tokens behind 28672, bf16: 2.56 ms, 1610 TFLOP/s, as the ring kernel's in a long loop: bound by
//     each unit's chain of S, softmax, P V
//     1024 tokens behind 15360: bf16 342 - 353 us (1560 - 1510), e4m3 394 us (1350), d = 64 265 and 330: in
//     e4m3 the expanding warps, 0.5 us each for V and K and 0.4 us for their scales' addresses, take as
//     long as the two softmaxes
//     16 x 8 tokens of 1k - 33k keys (one unit): bf16 170 us (5.8 TB/s), e4m3 174 us (2.9 TB/s: the expansion again)
// Short items pay about 9 us each for their first and last tiles and their epilogue.
//
// Warps: 0-7 softmax (four a unit), 8 and 9 issue the units' MMAs, 10 loads, 11 lists the block's
// parts; bf16: 12-15 look values over; e4m3: 12-19 expand and look over.  TMEM as in the ring kernel: S_x at
// [128 x, 128 x + 128), P_x over the upper half of S_x, O_x at 256 + D x.
#include <cuda_bf16.h>

#include "paged.h"
#include "ptx_paged.cuh"

namespace ra {
namespace {

constexpr int kTile = kPagedTile;
constexpr int kMmaWarp = 8, kLoadWarp = 10, kExpandWarp = 12;  // (11 lists)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kPBar = 1;                   // named barriers kPBar + x: unit x's P is written
constexpr int kPBarThreads = 4 * 32 + 32;  // its softmax warps and its issuer
constexpr int kPoison = 8;  // marks of the last parts, in turn: part k's holds k + 1 if it needs care

// ALONE: every item has one unit
template <int D, bool E4M3, bool ALONE>
struct Cfg {
    static constexpr int kThreads = E4M3 ? 640 : 512;
    // registers: what the softmax warps take, what the next four keep and what those behind them (that
    // expand or look over) do, of what all start with
    static constexpr int kStartRegs = E4M3 ? 96 : 128, kSoftmaxRegs = 168, kOtherRegs = E4M3 ? 64 : 88,
                         kExpandRegs = E4M3 ? 40 : 88;
    static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs + (kThreads - 384) * kExpandRegs <= kThreads * kStartRegs, "register split");
    static constexpr int kTileBytes = kTile * D * 2;  // a bf16 tile
    static constexpr int kBoxBytes = kTile * 128;     // 64 columns of it
    static constexpr int kBoxes = D / 64;
    static constexpr int kRawBytes = kTile * D;       // an e4m3 tile as it comes
    static constexpr int kStageBytes = 2 * kTileBytes;  // V of one tile and K of the next
    static constexpr int kStages = D == 128 ? 2 : 4;
    // e4m3 tiles on their way: what memory is left (one unit alone leaves the other's Q)
    static constexpr int kRaw = E4M3 ? (D == 128 ? (ALONE ? 4 : 2) : 8) : 0;
    static constexpr int kKVOff = (ALONE ? 1 : 2) * kTileBytes;
    static constexpr int kRawOff = kKVOff + kStages * kStageBytes;
    static constexpr int kSmemBytes = kRawOff + kRaw * kRawBytes + 1024;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kOCol = 256;
};

constexpr int kFixes = 8;  // more than the stages there are
constexpr int kParts = 4;  // parts listed ahead

// A V tile that not every row sees whole: where it lies and which of its keys are used.
struct Fix {
    int slot, parity;  // stage and parity of its load; slot < 0: no more requests
    int k, j0, hi, first;
};

struct Bars {
    uint64_t q_full[2], q_empty[2], s_full[2], o_done[2], o_free[2], drain[2];
    uint64_t pv_done;  // one unit alone: P V of a tile is in O
    uint64_t kv_full[4], kv_empty[4];
    // bf16: the loader asks for a V tile to be looked over (fix_req, its particulars in Shared::fix), the
    // issuers wait for it (fixed).  Requests are numbered; at most kStages are open at a time, one a stage.
    uint64_t fix_req[kFixes], fixed[kFixes];
    uint64_t raw_full[8], raw_empty[8];  // e4m3
    uint64_t part_full[kParts], part_empty[kParts];
};
// ------------------------------------------------------------------ items
// Pair `pair` of units of sequence b: tokens [ta, tb) of it, key tiles [0, ns) and from lo on.
struct Chunk {
    int b, pair;
    PagedSeq s;
    int ta, tb;   // tokens of the item
    int hi;       // keys at and behind hi are seen by no row
    int first;    // nor are keys below first that are no sinks
    int ns, lo, n;
    __device__ __forceinline__ int key(int t) const { return (t < ns ? t : lo + t - ns) * kTile; }
};

__device__ __forceinline__ Chunk make_chunk(const PagedAttnParams& p, int b, int pair, const PagedSeq& s) {
    Chunk c;
    c.b = b;
    c.pair = pair;
    c.s = s;
    const int tt = p.item_tokens;
    c.ta = pair * tt;
    c.tb = min(min(c.s.T, p.max_q), c.ta + tt);
    c.hi = p.causal ? min(c.s.L, max(0, c.s.base + c.tb)) : c.s.L;
    c.first = p.window > 0 ? max(0, c.s.base + c.ta - p.window + 1) : 0;
    const int hi = (c.hi + kTile - 1) / kTile;
    c.lo = min(c.first / kTile, hi);
    c.ns = p.window > 0 ? min((min(p.sinks, c.hi) + kTile - 1) / kTile, c.lo) : 0;
    c.n = max(1, c.ns + hi - c.lo);
    return c;
}

// Does every row of the item see every key of the tile at j0?
__device__ __forceinline__ bool whole_tile(const PagedAttnParams& p, const Chunk& c, int j0) {
    return j0 + kTile <= (p.causal ? c.s.base + c.ta + 1 : c.s.L) &&
           (p.window == 0 || j0 >= c.s.base + c.tb - p.window || j0 + kTile <= p.sinks);
}

__device__ __forceinline__ int pairs_of(const PagedAttnParams& p, int b) {
    const int tt = p.item_tokens;
    return (min(paged_seq(p.kv, b).T, p.max_q) + tt - 1) / tt;
}

// The list of items: base[b] = pairs of the sequences before b; pre[e] = tiles of the pairs before
// pair e (of one head).  Items are numbered by sequence, then head, then pair; the first rounds *
// grid are whole, one a block and round; block x takes tiles [fill[x], fill[x + 1]) of the rest.
struct Plan {
    long long* pre;
    long long* fill;
    int* base;
    int* rounds;
};
__device__ __forceinline__ Plan plan_at(const PagedAttnParams& p) {
    Plan x;
    x.pre = reinterpret_cast<long long*>(static_cast<uint8_t*>(p.workspace) + p.plan_off);
    x.fill = x.pre + p.max_pairs + 1;
    x.rounds = reinterpret_cast<int*>(x.fill + kPagedMaxShares + 1);
    x.base = x.rounds + 1;
    return x;
}

// Sequence, head and pair of item i.
struct Item {
    int b, h, e;
};
__device__ __forceinline__ Item find_item(const Plan& plan, int B, int H, long long i) {
    int lo = 0, hi = B;  // base[lo] * H <= i < base[hi] * H
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<long long>(plan.base[mid]) * H <= i) lo = mid;
        else hi = mid;
    }
    const int first = plan.base[lo], pairs = plan.base[lo + 1] - first;
    const long long in = i - static_cast<long long>(first) * H;
    Item it;
    it.b = lo;
    it.h = static_cast<int>(in / pairs);
    it.e = first + static_cast<int>(in - static_cast<long long>(it.h) * pairs);
    return it;
}
// Tiles before item `it`, all heads counted.
__device__ __forceinline__ long long tiles_before(const Plan& plan, int H, const Item& it) {
    const int e0 = plan.base[it.b], e1 = plan.base[it.b + 1];
    return plan.pre[e0] * H + (plan.pre[e1] - plan.pre[e0]) * it.h + plan.pre[it.e] - plan.pre[e0];
}

constexpr int kPlanThreads = 1024;

// Exclusive sum over the block; `all` receives the total.
__device__ __forceinline__ long long block_scan(long long x, long long* scratch, long long& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    long long y = x;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    if (lane == 31) scratch[warp] = y;
    __syncthreads();
    long long w = scratch[lane], v = w;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long z = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += z;
    }
    all = __shfl_sync(0xffffffffu, v, 31);
    const long long before = __shfl_sync(0xffffffffu, v - w, warp);
    __syncthreads();
    return before + y - x;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PagedAttnParams p, int grid) {
    __shared__ long long scratch[32];
    launch_dependents();
    const Plan plan = plan_at(p);
    const int B = p.kv.batch;
    long long sum = 0, all;
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        const long long at = block_scan(b < B ? pairs_of(p, b) : 0, scratch, all);
        // (a cu that decreases could list more than there is room for)
        if (b < B) plan.base[b] = static_cast<int>(min(sum + at, static_cast<long long>(p.max_pairs)));
        sum += all;
    }
    const int E = static_cast<int>(min(sum, static_cast<long long>(p.max_pairs)));
    if (threadIdx.x == 0) plan.base[B] = E;
    __syncthreads();
    sum = 0;
    for (int e0 = 0; e0 < E; e0 += kPlanThreads) {
        const int e = e0 + threadIdx.x;
        int n = 0;
        if (e < E) {
            int lo = 0, hi = B;  // base[lo] <= e < base[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (plan.base[mid] <= e) lo = mid;
                else hi = mid;
            }
            n = make_chunk(p, lo, e - plan.base[lo], paged_seq(p.kv, lo)).n;
        }
        const long long at = block_scan(n, scratch, all);
        if (e < E) plan.pre[e] = sum + at;
        sum += all;
    }
    if (threadIdx.x == 0) plan.pre[E] = sum;
    __syncthreads();
    // whole rounds, while every block's stay within an equal share
    const int H = p.kv.hkv, x = threadIdx.x;
    const long long W = sum * H, N = static_cast<long long>(E) * H, each = W / grid;
    long long load = 0;
    int rounds = 0;
    for (long long i = x; (rounds + 1LL) * grid <= N; i += grid, ++rounds) {
        long long more = 0;
        if (x < grid) {
            const Item it = find_item(plan, B, H, i);
            more = plan.pre[it.e + 1] - plan.pre[it.e];
        }
        if (__syncthreads_or(load + more > each)) break;
        load += more;
    }
    // A few items in all blocks: a tile less for each block is a part more for the join, which reads an item's
    // parts one after the other, a quarter of a tile's time each.  Shares of s tiles of T cost
    // s + T / (4 s), least where s = sqrt(T / 4).  (2 items of 118 tiles: 57 us in equal shares, 38 so;
    // one of 470: 77 us and 65.)
    const long long least = N > 0 ? static_cast<long long>(sqrtf(static_cast<float>(W / N) * 0.25f)) : 0;
    long long cap = 0;
    if (x < grid) cap = each >= least ? each + (x < W % grid ? 1 : 0) - load : max(0ll, min(least, W - least * x));
    const long long at = block_scan(cap, scratch, all);
    if (x < grid) plan.fill[x] = at;
    if (x == 0) {
        plan.fill[grid] = all;
        plan.rounds[0] = rounds;
    }
}

// Tiles [ta, tb) of an item, for KV head h.
struct Part {
    Chunk c;
    int h, ta, tb;
    int k;     // its number among this block's parts
    int slot;  // where its partial results go if it is cut: 0, or 1 behind the first of the filling
};

struct Shared {
    Bars b;
    uint32_t tmem;
    int abort_flag;
    uint32_t turn;
    int poison[kPoison];
    Fix fix[kFixes];
    Part part[kParts];
};

// Walks this block's parts: f(part) until it returns false.
template <class F>
__device__ __forceinline__ void for_each_part(const PagedAttnParams& p, F&& f) {
    const Plan plan = plan_at(p);
    const int B = p.kv.batch, H = p.kv.hkv;
    const int E = plan.base[B], rounds = plan.rounds[0];
    long long w = plan.fill[blockIdx.x];
    const long long w1 = plan.fill[blockIdx.x + 1];
    Part q;
    q.k = 0;
    q.slot = 0;
    int b = -1;
    PagedSeq s;
    for (int round = 0;; ++round) {
        // a whole item, or the first of the filling, which is found by its tile
        Item it;
        long long skip = 0;
        if (round < rounds) {
            it = find_item(plan, B, H, static_cast<long long>(round) * gridDim.x + blockIdx.x);
        } else {
            if (w >= w1) return;
            const long long N = static_cast<long long>(E) * H, i0 = static_cast<long long>(rounds) * gridDim.x;
            const long long t = w + (i0 < N ? tiles_before(plan, H, find_item(plan, B, H, i0)) : 0);
            int lo = 0, hi = B;  // the sequence: pre[base[lo]] * H <= t < pre[base[hi]] * H
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (plan.pre[plan.base[mid]] * H <= t) lo = mid;
                else hi = mid;
            }
            it.b = lo;
            const int e0 = plan.base[lo], e1 = plan.base[lo + 1];
            const long long off = plan.pre[e0], per = plan.pre[e1] - off;  // tiles of one head
            it.h = static_cast<int>((t - off * H) / per);
            const long long in = t - off * H - it.h * per + off;
            lo = e0;
            hi = e1;  // the pair: pre[lo] <= in < pre[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (plan.pre[mid] <= in) lo = mid;
                else hi = mid;
            }
            it.e = lo;
            skip = in - plan.pre[lo];
        }
        while (true) {
            if (it.b != b) {
                b = it.b;
                s = paged_seq(p.kv, b);
            }
            q.c = make_chunk(p, b, it.e - plan.base[b], s);
            q.h = it.h;
            q.ta = static_cast<int>(skip);
            q.tb = round < rounds ? q.c.n : static_cast<int>(min(static_cast<long long>(q.c.n), q.ta + (w1 - w)));
            if (!RA_CHECKED(it.b >= 0 && it.b < B && it.h >= 0 && it.h < H && it.e >= plan.base[it.b] && it.e < plan.base[it.b + 1] &&
                                q.c.ta < q.c.tb && q.ta >= 0 && q.ta < q.tb && q.tb <= q.c.n,
                            p.err, kSitePagedShare))
                return;
            if (!f(q)) return;
            ++q.k;
            if (round < rounds) break;
            w += q.tb - q.ta;
            if (w >= w1) return;
            q.slot = 1;
            skip = 0;
            if (++it.e == plan.base[it.b + 1]) {
                it.e = plan.base[it.b];
                if (++it.h == H) {
                    it.h = 0;
                    do ++it.b; while (plan.base[it.b + 1] == plan.base[it.b]);
                    it.e = plan.base[it.b];
                }
            }
        }
    }
}

// One warp walks the block's parts and lists them for the others, a few ahead: the walk's searches and
// loads are then in nobody's way, and the registers that it takes in nobody's count.
__device__ void list_role(const PagedAttnParams& p, Bars& b, Part* ring, const volatile uint32_t* turn, const WaitCtl& wc) {
    uint32_t k = 0;
    bool ok = true;
    auto put = [&](const Part& q) {
        ok = __all_sync(0xffffffffu, mbar_wait_idle(&b.part_empty[k % kParts], ((k / kParts) & 1u) ^ 1u, wc, 20000, turn));
        if (!ok) return false;
        if ((threadIdx.x & 31) == 0) {
            ring[k % kParts] = q;
            mbar_arrive(&b.part_full[k % kParts]);
        }
        ++k;
        return true;
    };
    for_each_part(p, put);
    Part end = {};
    if (ok) put(end);  // tb = 0: no more
}

// Takes the listed parts in order: f(part) until it returns false; false when it or a wait did.  Run by
// whole warps; `wait` is the role's way of waiting.
template <class Wait, class F>
__device__ __forceinline__ bool take_parts(Bars& b, const Part* ring, Wait&& wait, F&& f) {
    for (uint32_t k = 0;; ++k) {
        if (!wait(&b.part_full[k % kParts], (k / kParts) & 1u)) return false;
        const Part q = ring[k % kParts];
        if (q.tb == 0) return true;
        if (!f(q)) return false;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&b.part_empty[k % kParts]);
    }
}

// Units of an item: the second is there when its first token is.
template <bool ALONE>
__device__ __forceinline__ int units_of(const PagedAttnParams& p, const Chunk& c) {
    if (ALONE) return 1;
    return c.ta + p.unit_tokens < c.tb ? 2 : 1;
}

// How many tiles K runs ahead of V: a part's stages hold V(i - ahead) and K(i), what there is of them.
template <bool ALONE>
__device__ __forceinline__ int ahead_of(const Part& q) {
    return ALONE && q.tb - q.ta >= 2 ? 2 : 1;
}

// ------------------------------------------------------------------ the loading warp
// V at a stage's base, K a tile above it.  e4m3: the tiles go one by one into the raw ring, in
// the same order.
template <int D, bool E4M3, bool ALONE>
__device__ void load_role(const PagedAttnParams& p, const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv,
                          uint32_t smem, Bars& b, volatile Fix* fix, const Part* parts, const WaitCtl& wc) {
    using C = Cfg<D, E4M3, ALONE>;
    const PagedKV& kv = p.kv;
    const int lane = threadIdx.x & 31;
    const int rows = p.box_rows, boxes = kTile / rows;
    const uint32_t q_bytes = static_cast<uint32_t>(p.unit_tokens * p.g) * 128u * C::kBoxes;
    const uint64_t keep = make_policy_evict_last(), stream = make_policy_evict_first();
    uint32_t st = 0, qit[2] = {0, 0}, nf = 0;
    bool ok = true;
    auto ask = [&](int slot, int parity, int k, int j0, int hi, int first) {  // (one lane)
        volatile Fix& f = fix[nf % kFixes];
        f.slot = slot;
        f.parity = parity;
        f.k = k;
        f.j0 = j0;
        f.hi = hi;
        f.first = first;
        mbar_arrive(&b.fix_req[nf % kFixes]);
    };
    auto wait_part = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, 32)); };
    ok = take_parts(b, parts, wait_part, [&](const Part& q) -> bool {
        const int nx = units_of<ALONE>(p, q.c);
        for (int x = 0; x < nx; ++x) {
            ok = __all_sync(0xffffffffu, mbar_wait(&b.q_empty[x], (qit[x] & 1u) ^ 1u, wc, 32));
            if (!ok) return false;
            ++qit[x];
            if (lane == 0) {
                mbar_arrive_expect_tx(&b.q_full[x], q_bytes);
                int tok = q.c.s.q0 + q.c.ta + x * p.unit_tokens;
                if (!RA_CHECKED(paged_row_ok(kv, p.hq, tok, q.h * p.g + p.g - 1), p.err, kSitePagedToken)) tok = 0;
                for (int i = 0; i < C::kBoxes; ++i)
                    tma_load_3d(smem + x * C::kTileBytes + i * C::kBoxBytes, tq, &b.q_full[x], i * 64, q.h * p.g, tok, stream);
            }
            __syncwarp();
        }
        // K and V are read again by the sequence's other pairs, if it has any
        const uint64_t policy = q.c.s.T > p.item_tokens ? keep : stream;
        // the page of this lane's box, asked for a tile ahead and looked at only when it is needed: a load
        // waited for here would hold up the copies
        const int ahead = ahead_of<ALONE>(q);
        int entry = -1, row = 0, v_page = -1, v_y = 0, prev_page = -1, prev_y = 0;
        auto look = [&](int t) {  // no page behind the last key
            const int pos = q.c.key(t) + lane * rows;
            entry = -1;
            row = 0;
            if (lane < boxes && pos < q.c.hi) entry = paged_entry(kv, q.c.b, pos, row);
        };
        look(q.ta);
        for (int t = q.ta; t < q.tb + ahead; ++t) {
            int pg = paged_checked(kv, entry);
            if (pg >= 0 && !RA_CHECKED(paged_place_ok(kv, pg, q.h, row, rows), p.err, kSitePagedBox)) pg = -1;
            const int y = q.h * kv.page + row;
            if (t + 1 < q.tb) look(t + 1);
            const bool has_v = t >= q.ta + ahead, has_k = t < q.tb;
            if (ahead == 1) {
                v_page = prev_page;
                v_y = prev_y;
            }
            if constexpr (E4M3) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // V, then K
                    if (half ? !has_k : !has_v) continue;
                    const uint32_t slot = st % C::kRaw;
                    ok = __all_sync(0xffffffffu, mbar_wait(&b.raw_empty[slot], ((st / C::kRaw) & 1u) ^ 1u, wc, 32));
                    if (!ok) return false;
                    ++st;
                    if (lane == 0) mbar_arrive_expect_tx(&b.raw_full[slot], C::kRawBytes);
                    __syncwarp();
                    if (lane < boxes)
                        tma_load_3d(smem + C::kRawOff + slot * C::kRawBytes + lane * rows * D, half ? tk : tv, &b.raw_full[slot], 0,
                                    half ? y : v_y, half ? pg : v_page, policy);
                }
            } else {
                const uint32_t slot = st % C::kStages;
                ok = __all_sync(0xffffffffu, mbar_wait(&b.kv_empty[slot], ((st / C::kStages) & 1u) ^ 1u, wc, 32));
                if (!ok) return false;
                ++st;
                if (lane == 0) mbar_arrive_expect_tx(&b.kv_full[slot], (has_v && has_k) ? C::kStageBytes : C::kTileBytes);
                __syncwarp();
                if (lane < boxes) {
                    const uint32_t dst = smem + C::kKVOff + slot * C::kStageBytes + lane * rows * 128;
#pragma unroll
                    for (int i = 0; i < C::kBoxes; ++i) {
                        if (has_v) tma_load_3d(dst + i * C::kBoxBytes, tv, &b.kv_full[slot], i * 64, v_y, v_page, policy);
                        if (has_k)
                            tma_load_3d(dst + C::kTileBytes + i * C::kBoxBytes, tk, &b.kv_full[slot], i * 64, y, pg, policy);
                    }
                }
                if (has_v && !whole_tile(p, q.c, q.c.key(t - ahead))) {
                    if (lane == 0) ask(slot, ((st - 1) / C::kStages) & 1u, q.k, q.c.key(t - ahead), q.c.hi, q.c.first);
                    ++nf;
                }
            }
            v_page = prev_page;
            v_y = prev_y;
            prev_page = pg;
            prev_y = y;
        }
        return true;
    });
    if (!E4M3 && ok && lane == 0) ask(-1, 0, 0, 0, 0, 0);
    if (!ok && lane == 0) {  // let the copies in flight land before the block ends
        constexpr uint32_t kN = E4M3 ? C::kRaw : C::kStages;
        uint64_t* full = E4M3 ? b.raw_full : b.kv_full;
        for (uint32_t s = 0; s < kN && s < st; ++s) {
            const uint32_t last = st - 1 - ((st - 1 - s) % kN);
            drain_wait(&full[s], (last / kN) & 1u, wc.timeout_ns);
        }
        for (int x = 0; x < 2; ++x)
            if (qit[x] > 0) drain_wait(&b.q_full[x], (qit[x] - 1) & 1u, wc.timeout_ns);
    }
}

// ------------------------------------------------------------------ values that must not spread
__device__ __forceinline__ bool key_used(int j, int hi, int first, int sinks) {
    return j < hi && (j >= first || j < sinks);
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A pair of bf16 with infinities and NaN as zeros.
__device__ __forceinline__ uint32_t finite2(uint32_t y) {
    return y & ~(((y & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((y & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u));
}

// bf16: four warps, 32 keys each, clean the V tiles that they are asked to, in place.  (One warp took
// longer than a tile's other work, and the product waited.)
template <int D, bool ALONE>
__device__ void fix_role(const PagedAttnParams& p, uint32_t smem, Bars& b, const volatile Fix* fix, volatile int* poison,
                         const volatile uint32_t* turn, const WaitCtl& wc) {
    using C = Cfg<D, false, ALONE>;
    const int lane = threadIdx.x & 31, quarter = threadIdx.x / 32 - kExpandWarp;
    for (uint32_t nf = 0;; ++nf) {
        if (!__all_sync(0xffffffffu, mbar_wait_idle(&b.fix_req[nf % kFixes], (nf / kFixes) & 1u, wc, 20000, turn))) return;
        const volatile Fix& f = fix[nf % kFixes];
        const int slot = f.slot, j0 = f.j0, hi = f.hi, first = f.first, k = f.k;
        if (slot < 0) return;
        // (the stage stays as it is until the issuers have had this tile, so its parity says enough)
        if (!mbar_wait_w(&b.kv_full[slot], f.parity, wc)) return;
        const uint32_t v = smem + C::kKVOff + slot * C::kStageBytes + lane * 16;
        bool bad = false;
        // eight lanes a row of 128 bytes, so four rows a load; eight loads in flight.  (The
        // swizzle permutes chunks inside a row only.)
#pragma unroll 1
        for (int i = 0; i < C::kBoxes; ++i) {
            const uint32_t at = v + i * C::kBoxBytes + quarter * (32 * 128);
            const int r = quarter * 32 + lane / 8;  // and r + 4, ... r + 28
            uint4 x[8];
            uint32_t top = 0, drop = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = lds128(at + e * 512);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t m = __vmaxu2(__vmaxu2(x[e].x & 0x7fff7fffu, x[e].y & 0x7fff7fffu),
                                            __vmaxu2(x[e].z & 0x7fff7fffu, x[e].w & 0x7fff7fffu));
                if (key_used(j0 + r + 4 * e, hi, first, p.sinks)) top = __vmaxu2(top, m);
                else drop |= 1u << e;
            }
            const bool sick = max(top & 0xffffu, top >> 16) >= 0x7f80u;
            if (drop || sick) {
                bad |= sick;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t keep = (drop >> e) & 1u ? 0u : 0xffffffffu;
                    sts128(at + e * 512, finite2(x[e].x) & keep, finite2(x[e].y) & keep, finite2(x[e].z) & keep,
                           finite2(x[e].w) & keep);
                }
            }
        }
        if (bad) poison[k % kPoison] = k + 1;
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.fixed[nf % kFixes]);
    }
}

// Two of a word's four bytes (the upper two if `upper`) as the low bytes of halves, each sign-extended.
__device__ __forceinline__ uint32_t spread_signed(uint32_t w, bool upper) {
    uint32_t a;
    if (upper) asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(a) : "r"(w));
    else asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(w));
    return a;
}

__device__ __forceinline__ uint32_t times(uint32_t x, __nv_bfloat162 m) {
    const __nv_bfloat162 z = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), m);
    return *reinterpret_cast<const uint32_t*>(&z);
}

// e4m3: 256 threads, half a row each, expand every tile into its bf16 stage.
template <int D, bool ALONE>
__device__ void expand_role(const PagedAttnParams& p, uint32_t smem, Bars& b, const Part* parts, volatile int* poison,
                            const WaitCtl& wc) {
    using C = Cfg<D, true, ALONE>;
    const PagedKV& kv = p.kv;
    const int r = threadIdx.x & (kTile - 1);
    const int c0 = threadIdx.x >= kExpandWarp * 32 + kTile ? D / 32 : 0;  // first chunk of this half
    uint32_t st = 0, raw = 0;
    const uint32_t row_at = r * 128, sw = r & 7;
    auto expand = [&](uint32_t dst, float scale, bool zero) -> bool {
        const uint32_t slot = raw % C::kRaw;
        if (!mbar_wait_w(&b.raw_full[slot], (raw / C::kRaw) & 1u, wc)) return false;
        ++raw;
        const uint32_t src = smem + C::kRawOff + slot * C::kRawBytes + r * D;
        const uint32_t src_sw = D == 128 ? sw : ((r >> 1) & 3);
        // 2^120 * scale, in two factors where it is no bf16 number; 0 where the row counts as zeros
        // (a scale that is no number is kept out of the product there)
        const bool big = scale > 128.f;
        const __nv_bfloat162 m1 = __float2bfloat162_rn(zero ? 0.f : big ? 0x1p120f : scale * 0x1p120f);
        uint4 next = lds128(src + ((c0 ^ src_sw) << 4));
#pragma unroll
        for (int i2 = 0; i2 < D / 32; ++i2) {
            const int c = c0 + i2;
            const uint4 x = next;
            if (i2 + 1 < D / 32) next = lds128(src + (((c + 1) ^ src_sw) << 4));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // a code in each low byte with its sign all over the byte above: 4 bits up, the sign and the
                // rest are where bf16 has them (one operation less than moving them apart, of five: the
                // chunk of 1024 tokens of 16k took 464 us, 416 now)
                const uint32_t v = (spread_signed(w[i >> 1], i & 1) << 4) & 0x87f087f0u;
                const __nv_bfloat162 z = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), m1);
                y[i] = *reinterpret_cast<const uint32_t*>(&z);
            }
            const uint32_t d = dst + (c >> 2) * C::kBoxBytes + row_at;
            sts128(d + ((((2 * c) & 7) ^ sw) << 4), y[0], y[1], y[2], y[3]);
            sts128(d + ((((2 * c + 1) & 7) ^ sw) << 4), y[4], y[5], y[6], y[7]);
        }
        if (big && !zero) {  // (a pass of its own: a second factor for every pair cost 8 % of the whole kernel's time)
            const __nv_bfloat162 m2 = __float2bfloat162_rn(scale);
#pragma unroll 1
            for (int c = 2 * c0; c < 2 * c0 + D / 16; ++c) {
                const uint32_t d = dst + (c >> 3) * C::kBoxBytes + row_at + (((c & 7) ^ sw) << 4);
                const uint4 x = lds128(d);
                sts128(d, times(x.x, m2), times(x.y, m2), times(x.z, m2), times(x.w, m2));
            }
        }
        // Only now, when every loaded code has been used: an arrival right behind the loads let the
        // next tile's copy overtake them (seen as wrong values in the chunks loaded last).
        mbar_arrive(&b.raw_empty[slot]);
        return true;
    };
    take_parts(b, parts, [&](uint64_t* bar, uint32_t parity) { return mbar_wait_w(bar, parity, wc); }, [&](const Part& q) -> bool {
        // this row's page two tiles ahead, and its scales one: neither load is waited for at once
        float ks = 0.f, vs = 0.f;
        int entry = -1, row = 0;
        auto look = [&](int t) {
            const int pos = q.c.key(t) + r;
            entry = -1;
            if (t < q.tb && pos < q.c.hi) entry = paged_entry(kv, q.c.b, pos, row);
        };
        auto fetch = [&]() {
            int pg = paged_checked(kv, entry);
            if (pg >= 0 && !RA_CHECKED(paged_place_ok(kv, pg, q.h, row), p.err, kSitePagedPlace)) pg = -1;
            const long long at = static_cast<long long>(q.h) * kv.page + row;
            ks = pg >= 0 ? __ldg(kv.k_scale + pg * kv.ks_ps + at) : 0.f;
            vs = pg >= 0 ? __ldg(kv.v_scale + pg * kv.vs_ps + at) : 0.f;
        };
        look(q.ta);
        fetch();
        look(q.ta + 1);
        const int ahead = ahead_of<ALONE>(q);
        float vs1 = 0.f, vs2 = 0.f;  // V scales of one and two tiles ago
        for (int t = q.ta; t < q.tb + ahead; ++t, ++st) {
            const float k1 = ks, v1 = ahead == 1 ? vs1 : vs2;
            vs2 = vs1;
            vs1 = vs;
            const uint32_t slot = st % C::kStages;
            if (!mbar_wait_w(&b.kv_empty[slot], ((st / C::kStages) & 1u) ^ 1u, wc)) return false;
            const uint32_t stage = smem + C::kKVOff + slot * C::kStageBytes;
            if (t >= q.ta + ahead) {
                bool zero = false;
                const int j0 = q.c.key(t - ahead);
                if (!whole_tile(p, q.c, j0)) {
                    zero = !key_used(j0 + r, q.c.hi, q.c.first, p.sinks);
                    if (!zero && !(fabsf(v1) < INFINITY)) {
                        zero = true;
                        poison[q.k % kPoison] = q.k + 1;
                    }
                }
                if (!expand(stage, v1, zero)) return false;
            }
            fetch();
            look(t + 2);
            if (t < q.tb && !expand(stage + C::kTileBytes, k1, false)) return false;
            fence_async_shared();
            mbar_arrive(&b.kv_full[slot]);
        }
        return true;
    });
}

// ------------------------------------------------------------------ MMA issuers
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t smem_addr, uint32_t lbo) {
    return ((smem_addr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}
constexpr uint32_t kSdescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // sbo 1024 B, version 1, 128 B swizzle

// S = Q K^T: K slice kk lies (kk / 4) boxes and (kk % 4) * 32 bytes in.
template <int D>
__device__ __forceinline__ void issue_s(uint32_t d_tmem, uint32_t q_base, uint32_t k_base) {
    constexpr uint32_t idesc = idesc_bf16(kTile, kTile, 0);
    const uint32_t qlo = sdesc_lo(q_base, 16), klo = sdesc_lo(k_base, 16);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk / 4) * (kTile * 128 >> 4) + (kk % 4) * (32 >> 4);
        asm volatile(
            "{\n\t.reg .b64 da, db;\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(qlo + off), "r"(klo + off), "r"(idesc), "r"(kk > 0 ? 1u : 0u), "r"(kSdescHi)
            : "memory");
    }
}
// O += P V, P from tensor memory.
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_base, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16(kTile, D, 1);
    const uint32_t vlo = sdesc_lo(v_base, kTile * 128);
    const uint32_t acc = accumulate ? 1u : 0u;
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk) {
        asm volatile(
            "{\n\t.reg .b64 db;\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "mov.b64 db, {%2, %5};\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(p_tmem + kk * 8), "r"(vlo + ((kk * 16 * 128) >> 4)), "r"(idesc), "r"(kk > 0 ? 1u : acc),
            "r"(kSdescHi)
            : "memory");
    }
}

__device__ __forceinline__ bool wait_turn(volatile uint32_t* turn, uint32_t mine, const WaitCtl& wc) {
    if (*turn == mine) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (*turn == mine) return true;
        if ((i & 255u) == 0u) {
            if (*wc.abort_flag) return false;
            if (globaltimer_ns() - t0 > wc.timeout_ns) {
                raise_abort(wc, reinterpret_cast<uint64_t*>(const_cast<uint32_t*>(turn)));
                return false;
            }
        }
    }
}

// The issuer of unit x.  The two take turns batch by batch (`turn` counts the batches issued), so
// that the tensor pipe sees each unit's batch whole while one issuer's waits overlap the
// other's batch.  Every stage is released once by each of them.  (One unit alone: one issuer.)
template <int D, bool E4M3, bool ALONE>
__device__ void mma_role(const PagedAttnParams& p, int x, uint32_t smem, Bars& b, const Part* parts, uint32_t tmem,
                         volatile uint32_t* turn, const WaitCtl& wc) {
    using C = Cfg<D, E4M3, ALONE>;
    const uint32_t q_base = smem + x * C::kTileBytes, kv_base = smem + C::kKVOff;
    const uint32_t o_tmem = tmem + C::kOCol + x * D;
    uint32_t st = 0, qit = 0, seq = 0, nf = 0;
    auto wait_part = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_w(bar, parity, wc); };
    const bool ok = take_parts(b, parts, wait_part, [&](const Part& q) -> bool {
        const int n = q.tb - q.ta, nx = units_of<ALONE>(p, q.c);
        auto wait_stage = [&](uint32_t& slot, uint32_t& base) -> bool {
            slot = st % C::kStages;
            base = kv_base + slot * C::kStageBytes;
            const bool r = mbar_wait_w(&b.kv_full[slot], (st / C::kStages) & 1u, wc);
            ++st;
            return r;
        };
        uint32_t slot, base;
        const int ahead = ahead_of<ALONE>(q);
        if (x >= nx) {  // no second unit: pass every stage
            for (int i = 0; i < n + ahead; ++i) {
                if (!wait_stage(slot, base)) return false;
                if ((threadIdx.x & 31) == 0) mbar_arrive(&b.kv_empty[slot]);
                if (!E4M3 && i >= ahead && !whole_tile(p, q.c, q.c.key(q.ta + i - ahead))) ++nf;
            }
            seq += n + ahead;
            return true;
        }
        // batches: the first scores' of unit x are seq + x (and, one unit ahead by two, seq + 1), tile j's
        // seq + nx j + x behind them
        if (!mbar_wait_w(&b.q_full[x], qit & 1u, wc)) return false;
        for (int i = 0; i < ahead; ++i) {
            if (!wait_stage(slot, base)) return false;
            if (!__all_sync(0xffffffffu, wait_turn(turn, seq + x, wc))) return false;
            tc_fence_after();
            issue_s<D>(tmem + (x + i) * kTile, q_base, base + C::kTileBytes);
            mma_commit_e(&b.s_full[x + i]);
            if (i + 1 < ahead) ++seq;
            *turn = seq + x + (i + 1 < ahead ? 0 : 1);
            mma_commit_e(&b.kv_empty[slot]);
            if (i + 1 == n) mma_commit_e(&b.q_empty[x]);
        }
        for (int j = 0; j < n; ++j) {
            if (!wait_stage(slot, base)) return false;  // V(j) and, unless there is none, K(j + ahead)
            if (!E4M3 && !whole_tile(p, q.c, q.c.key(q.ta + j))) {
                if (!mbar_wait_w(&b.fixed[nf % kFixes], (nf / kFixes) & 1u, wc)) return false;
                ++nf;
            }
            const int y = ahead == 2 ? (j & 1) : x;  // whose S columns tile j's scores are in
            const uint32_t mine = seq + nx * (j + 1) + x;
            if (!__all_sync(0xffffffffu, wait_turn(turn, mine, wc))) return false;
            if (j == 0 && !mbar_wait_w(&b.o_free[x], (qit & 1u) ^ 1u, wc)) return false;
            // P on a hardware named barrier, which releases the issuer as the last softmax warp arrives,
            // sooner than an mbarrier's wake.  It cannot time out: it is entered only while no role has
            // given up, after S(j) was queued, and the softmax warps arrive for every tile whose S they see.
            if (__any_sync(0xffffffffu, *wc.abort_flag != 0)) return false;
            named_bar_sync(kPBar + y, kPBarThreads);
            tc_fence_after();
            issue_pv<D>(o_tmem, tmem + y * kTile + 64, base, j > 0);
            if (ALONE) mma_commit_e(&b.pv_done);
            if (j + ahead < n) {
                issue_s<D>(tmem + y * kTile, q_base, base + C::kTileBytes);
                mma_commit_e(&b.s_full[y]);
            }
            if (j + 1 == n) mma_commit_e(&b.o_done[x]);
            *turn = mine + 1;
            mma_commit_e(&b.kv_empty[slot]);
            if (j + ahead + 1 == n) mma_commit_e(&b.q_empty[x]);
        }
        seq += nx * (n + 1);
        ++qit;
        return true;
    });
    if (!ok) {  // every MMA this warp issued must finish before TMEM is released
        mma_commit_e(&b.drain[x]);
        drain_wait(&b.drain[x], 0, wc.timeout_ns);
    }
}

// ------------------------------------------------------------------ softmax
// Bits [0, n) set, n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}
// Which of 32 keys a row sees: below hi, and from lo on or below the sinks (all relative to them).
__device__ __forceinline__ uint32_t seen_bits(int hi, int lo, int sinks) {
    return low_bits(hi) & (~low_bits(lo) | low_bits(sinks));
}

// Hides what this row does not see of a tile: its scores from hi on, and those below lo that are not
// below sinks.  In place, 32 columns at a time in a rolled loop and not inlined: it is rare, and as
// straight code over 128 registers it ran at the speed of instruction fetches (9 us a tile).
__device__ __noinline__ void mask_scores(uint32_t s_tmem, int hi, int lo, int sinks) {
#pragma unroll 1
    for (int cc = 0; cc < kTile; cc += 32) {
        const uint32_t see = seen_bits(hi - cc, lo - cc, sinks - cc);
        if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
        uint32_t r[32];
        tmem_ld32(s_tmem + cc, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = (see & (1u << i)) ? r[i] : 0xff800000u;
        tmem_st32(s_tmem + cc, r);
    }
    tmem_wait_st();
}

// 64 bytes of a row (16-byte aligned; `wide`: 32-byte).  A lane has a row to itself: stores of 32 bytes fill
// whole sectors of their lines without an exchange between lanes, which took longer than it saved.
__device__ __forceinline__ void store_row(void* dst, const uint32_t (&w)[16], bool wide) {
    if (wide) {
#pragma unroll
        for (int i = 0; i < 16; i += 8)
            stg256(static_cast<uint32_t*>(dst) + i, w[i], w[i + 1], w[i + 2], w[i + 3], w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<uint4*>(static_cast<uint32_t*>(dst) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
}

// Values that are no numbers, of the keys a row sees in the part's tiles that were looked over:
// columns [cc, cc + 32) of the row's sum.  (Those of other tiles went into the product.)
template <bool E4M3, int D>
__device__ __noinline__ void add_sick(const PagedAttnParams& p, const Chunk& c, int h, int ta, int tb, int hi, int lo,
                                      int cc, float (&o)[32]) {
    for (int t = ta; t < tb; ++t) {
        const int j0 = c.key(t);
        if (whole_tile(p, c, j0)) continue;
        for (int j = j0; j < min(j0 + kTile, hi); ++j) {
            if (j < lo && j >= p.sinks) continue;
            int r;
            const int pg = paged_page(p.kv, c.b, j, r);
            if (pg < 0 || !RA_CHECKED(paged_place_ok(p.kv, pg, h, r), p.err, kSitePagedPlace)) continue;
            const long long at = static_cast<long long>(h) * p.kv.page + r;
            if constexpr (E4M3) {
                if (fabsf(__ldg(p.kv.v_scale + pg * p.kv.vs_ps + at)) < INFINITY) continue;
                for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(0x7fc00000u);
            } else {
                const uint32_t* v = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.kv.v) + pg * p.kv.v_ps + at * D + cc);
                for (int i = 0; i < 16; ++i) {
                    const uint32_t y = __ldg(v + i);
                    if ((y & 0x7f80u) == 0x7f80u) o[2 * i] += __uint_as_float(y << 16);
                    if ((y & 0x7f800000u) == 0x7f800000u) o[2 * i + 1] += __uint_as_float(y & 0xffff0000u);
                }
            }
        }
    }
}

// This row's O times f.  (Rolled and not inlined, as mask_scores: rare, and the less code the warps of all
// roles run through, the fewer wait for instructions.)
template <int D>
__device__ __noinline__ void scale_o(uint32_t o_tmem, float f) {
#pragma unroll 1
    for (int cc = 0; cc < D; cc += 32) {
        uint32_t o[32];
        tmem_ld32(o_tmem + cc, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st32(o_tmem + cc, o);
    }
    tmem_wait_st();
}

// The tensor cores add to O with truncation, a step of up to 2^-23 of it for every 16 keys and always
// towards zero, so a million keys in one sum lost 0.4 % (of equal weights and positive values).  So O is
// moved to memory every kFold tiles of a part and added up there, rounded to nearest; 64k keys
// lose 5e-5 with equal weights, 4e-4 with others, of which every addend is cut off.  The place is the block's second partial result, which nothing else needs before the
// part that ends there, thread x's row being its row x; it has the scale of the m beside it.
constexpr int kFold = 512;
__device__ __forceinline__ float fold_factor(float before, float m) { return before == m ? 1.f : ex2(before - m); }
__device__ __forceinline__ PagedChunkPartial* fold_place(void* workspace) {
    return static_cast<PagedChunkPartial*>(workspace) + 2 * blockIdx.x + 1;
}
template <int D>
__device__ __noinline__ void fold_o(void* workspace, uint32_t o_tmem, float m, bool first) {
    PagedChunkPartial* to = fold_place(workspace);
    const int r2 = threadIdx.x;
    const float f = first ? 0.f : fold_factor(to->m[r2], m);
    to->m[r2] = m;
#pragma unroll 1
    for (int cc = 0; cc < D; cc += 32) {
        uint32_t o[32];
        tmem_ld32(o_tmem + cc, o);
        tmem_wait_ld();
        float4* at = to->o + (cc / 4) * (2 * kTile) + r2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float4 y = first ? make_float4(0.f, 0.f, 0.f, 0.f) : at[i * (2 * kTile)];
            y.x = __fmaf_rn(y.x, f, __uint_as_float(o[4 * i]));
            y.y = __fmaf_rn(y.y, f, __uint_as_float(o[4 * i + 1]));
            y.z = __fmaf_rn(y.z, f, __uint_as_float(o[4 * i + 2]));
            y.w = __fmaf_rn(y.w, f, __uint_as_float(o[4 * i + 3]));
            at[i * (2 * kTile)] = y;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0u;
        tmem_st32(o_tmem + cc, o);
    }
}

__device__ __forceinline__ void unfold_o(void* workspace, int cc, float m, float (&o)[32]) {
    const PagedChunkPartial* from = fold_place(workspace);
    const int r2 = threadIdx.x;
    const float f = fold_factor(from->m[r2], m);
    const float4* at = from->o + (cc / 4) * (2 * kTile) + r2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 y = at[i * (2 * kTile)];
        o[4 * i] = __fmaf_rn(y.x, f, o[4 * i]);
        o[4 * i + 1] = __fmaf_rn(y.y, f, o[4 * i + 1]);
        o[4 * i + 2] = __fmaf_rn(y.z, f, o[4 * i + 2]);
        o[4 * i + 3] = __fmaf_rn(y.w, f, o[4 * i + 3]);
    }
}

template <int D, bool E4M3, bool ALONE>
__device__ void softmax_role(const PagedAttnParams& p, int x, Bars& b, const Part* parts, uint32_t tmem,
                             const volatile int* poison, const WaitCtl& wc) {
    using C = Cfg<D, E4M3, ALONE>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t o_tmem = tmem + lane_off + C::kOCol + x * D;
    const int tok_in = row / p.g;
    uint32_t sit[2] = {0, 0}, pvs = 0, iit = 0;  // uses of s_full (one unit alone: of both) and pv_done; items
    // The issuer waits for P where it cannot give up, so these warps hold on to every S that it queued:
    // their waits end with the barrier or with their own time limit (a second at least, far above
    // what a queued MMA takes), never because another role has given up.
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_noabort(bar, parity, wc));
    };
    take_parts(b, parts, wait, [&](const Part& q) -> bool {
        if (x >= units_of<ALONE>(p, q.c)) return true;
        const bool two = ahead_of<ALONE>(q) == 2;  // scores in both units' S columns in turn
        const int t_row = q.c.ta + x * p.unit_tokens + tok_in;  // the row's token; none if not below tb
        const int pos = q.c.s.base + t_row;
        // keys this row sees: below hi, and from lo on or below the sinks
        const int hi = p.causal ? min(pos + 1, q.c.s.L) : q.c.s.L;
        const int lo = p.window > 0 ? pos - p.window + 1 : 0;
        // the rows of the unit all see a tile that lies in [., u_hi) and from u_lo on
        const int t0 = q.c.ta + x * p.unit_tokens, t1 = min(t0 + p.unit_tokens, q.c.tb);
        const int u_hi = p.causal ? q.c.s.base + t0 + 1 : q.c.s.L;
        const int u_lo = p.window > 0 ? q.c.s.base + t1 - p.window : 0;
        float m = -INFINITY, l = 0.f, lr = 0.f;
        for (int t = q.ta; t < q.tb; ++t) {
            const int j0 = q.c.key(t);
            const int y = ALONE ? (two ? (t - q.ta) & 1 : 0) : x;
            const uint32_t s_tmem = tmem + lane_off + y * kTile, p_tmem = s_tmem + 64;
            if (!wait(&b.s_full[y], (ALONE && y ? sit[1] : sit[0]) & 1u)) return false;
            if (ALONE && y) ++sit[1];
            else ++sit[0];
            tc_fence_after();
            if (j0 + kTile > u_hi || (j0 < u_lo && j0 + kTile > p.sinks))  // not every row of the unit sees it whole
                mask_scores(s_tmem, hi - j0, lo - j0, p.window > 0 ? p.sinks - j0 : 0);
            float s[kTile];
            float pm0, pm1, pm2, pm3;
            {
                uint32_t r0[32], r1[32], r2[32], r3[32];
                tmem_ld32_max(s_tmem + 0, r0, pm0);
                tmem_ld32_max(s_tmem + 32, r1, pm1);
                tmem_ld32_max(s_tmem + 64, r2, pm2);
                tmem_ld32_max(s_tmem + 96, r3, pm3);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    s[i] = __uint_as_float(r0[i]);
                    s[32 + i] = __uint_as_float(r1[i]);
                    s[64 + i] = __uint_as_float(r2[i]);
                    s[96 + i] = __uint_as_float(r3[i]);
                }
            }
            const float mx = fmaxf(fmaxf(pm0, pm1), fmaxf(pm2, pm3));
            const float m_new = fmaxf(m, mx * kLog2e);
            float f = 1.f;
            bool need = false;
            if (t == q.ta) {
                m = m_new;
            } else if (m_new > m + kRescaleLog2 || (m == -INFINITY && m_new > m)) {
                need = true;
                f = ex2(m - m_new);
                l *= f;
                lr *= f;
                m = m_new;
            }
            const float nmu = (m == -INFINITY) ? 0.f : -m;
            float se[2] = {}, sr[2] = {};
#pragma unroll
            for (int qq = 0; qq < 4; ++qq) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float t0, t1;
                    ffma2(t0, t1, s[qq * 32 + 2 * i], s[qq * 32 + 2 * i + 1], kLog2e, kLog2e, nmu, nmu);
                    const float a = ex2(t0), c2 = ex2(t1);
                    fadd2(se[0], se[1], se[0], se[1], a, c2);
                    pk[i] = pack_bf16x2(a, c2);
                    add_bf16x2_f32(sr[0], sr[1], pk[i]);
                }
                tmem_st16(p_tmem + qq * 16, pk);  // every score is in registers: P may overwrite S's upper half
            }
            // O is stable here: the commit that signalled this S covered the previous P V (one unit alone:
            // only the one before it), and the next one waits for this tile's arrivals
            const bool fold = t > q.ta && (t - q.ta) % kFold == 0, rescale = __any_sync(0xffffffffu, need);
            if (rescale || fold) {
                if (ALONE) {  // tile t is the part's (t - ta)th; its predecessor's P V is use pvs + t - ta - 1
                    if (!wait(&b.pv_done, (pvs + (t - q.ta) - 1) & 1u)) return false;
                    tc_fence_after();
                }
                if (rescale) scale_o<D>(o_tmem, f);
                if (fold) fold_o<D>(p.workspace, o_tmem, m, t - q.ta == kFold);
            }
            l += se[0] + se[1];
            lr += sr[0] + sr[1];
            tmem_wait_st();
            tc_fence_before();
            named_bar_arrive(kPBar + y, kPBarThreads);
        }
        pvs += q.tb - q.ta;
        if (!wait(&b.o_done[x], iit & 1u)) return false;
        ++iit;
        tc_fence_after();
        const bool cut = q.ta > 0 || q.tb < q.c.n;
        const bool live = row < p.unit_tokens * p.g && t_row < q.c.tb &&
                          RA_CHECKED(paged_row_ok(p.kv, p.hq, q.c.s.q0 + t_row, q.h * p.g + row - tok_in * p.g), p.err, kSitePagedOut) &&
                          RA_CHECKED(q.slot == 0 || q.slot == 1, p.err, kSitePagedPartial);
        const bool sick = poison[q.k % kPoison] == q.k + 1;
        const float inv = lr == 0.f ? 0.f : 1.f / lr;
        const int tok = q.c.s.q0 + t_row, head = q.h * p.g + row - tok_in * p.g;
        PagedChunkPartial* part = static_cast<PagedChunkPartial*>(p.workspace) + 2 * blockIdx.x + q.slot;
        const int r2 = x * kTile + row;
        if (!cut && !sick && !p.out_f32 && q.tb - q.ta <= kFold) {  // the usual end, with all loads in flight at once
            uint32_t o[D / 32][32];
#pragma unroll
            for (int c = 0; c < D / 32; ++c) tmem_ld32(o_tmem + c * 32, o[c]);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&b.o_free[x]);
            if (live) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[i] = pack_bf16x2(__uint_as_float(o[c][2 * i]) * inv, __uint_as_float(o[c][2 * i + 1]) * inv);
                    store_row(static_cast<uint16_t*>(p.out) + tok * p.o_ts + head * p.o_hs + c * 32, w, p.out_wide);
                }
                paged_store_lse(p, tok, head, m, l);
            }
            return true;
        }
        // (rolled, as the mask: a quarter of the code to fetch)
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
            float o[32];
            {
                uint32_t r[32];
                tmem_ld32(o_tmem + cc, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(r[i]);
            }
            if (cc + 32 == D) {
                tc_fence_before();
                mbar_arrive(&b.o_free[x]);
            }
            if (q.tb - q.ta > kFold) unfold_o(p.workspace, cc, m, o);
            if (sick && live) {  // (copies, so that only this rare call keeps anything in memory)
                const Chunk c = q.c;
                float o2[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) o2[i] = o[i];
                add_sick<E4M3, D>(p, c, q.h, q.ta, q.tb, hi, lo, cc, o2);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = o2[i];
            }
            if (cut && live) {
                float4* dst = part->o + (cc / 4) * (2 * kTile) + r2;
#pragma unroll
                for (int i = 0; i < 8; ++i) dst[i * (2 * kTile)] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
            if (!cut) {
                if (p.out_f32) {
                    float* dst = static_cast<float*>(p.out) + tok * p.o_ts + head * p.o_hs + cc;
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[16 * h2 + i] * inv);
                        if (live) store_row(dst + 16 * h2, w, p.out_wide);
                    }
                } else {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
                    if (live) store_row(static_cast<uint16_t*>(p.out) + tok * p.o_ts + head * p.o_hs + cc, w, p.out_wide);
                }
            }
        }
        if (cut) {
            if (live) {
                part->m[r2] = m;
                part->l[r2] = l;
                part->lr[r2] = lr;
            }
            if (x == 0 && row == 0 && live) {
                part->b = q.c.b;
                part->pair = q.c.pair;
                part->h = q.h;
                part->begins = q.ta == 0;
            }
        } else if (live) {
            paged_store_lse(p, tok, head, m, l);
        }
        return true;
    });
}

template <int D, bool E4M3, bool ALONE>
__global__ void __launch_bounds__(Cfg<D, E4M3, ALONE>::kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ PagedAttnParams p, const __grid_constant__ CUtensorMap tq,
                       const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
    using C = Cfg<D, E4M3, ALONE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) Shared sh;
    Bars& b = sh.b;
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&b.q_full[x], 1);
            mbar_init(&b.q_empty[x], 1);
            mbar_init(&b.s_full[x], 1);
            mbar_init(&b.o_done[x], 1);
            mbar_init(&b.o_free[x], 128);
            mbar_init(&b.drain[x], 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&b.kv_full[s], E4M3 ? 256 : 1);
            mbar_init(&b.kv_empty[s], ALONE ? 1 : 2);  // the issuers
        }
        for (int s = 0; s < 8; ++s) {
            mbar_init(&b.raw_full[s], 1);
            mbar_init(&b.raw_empty[s], 256);
        }
        mbar_init(&b.pv_done, 1);
        for (int s = 0; s < kParts; ++s) {
            mbar_init(&b.part_full[s], 1);
            mbar_init(&b.part_empty[s], (ALONE ? 6 : 11) + (E4M3 ? 8 : 0));  // softmax warps, issuers, loader, expanding warps
        }
        for (int s = 0; s < kFixes; ++s) {
            mbar_init(&b.fix_req[s], 1);
            mbar_init(&b.fixed[s], 4);
        }
        sh.abort_flag = 0;
        sh.turn = 0;
        for (int i = 0; i < kPoison; ++i) sh.poison[i] = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem, C::kTmemCols);
        tmem_relinquish();
    }
    launch_dependents();
    wait_primary();  // the list of items
    if (threadIdx.x < 2) {  // no partial results yet; and a block without a filling is no link between two
        const Plan plan = plan_at(p);
        const bool none = threadIdx.x == 0 && plan.fill[blockIdx.x] == plan.fill[blockIdx.x + 1];
        (static_cast<PagedChunkPartial*>(p.workspace) + 2 * blockIdx.x + threadIdx.x)->b = none ? -2 : -1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const WaitCtl wc{&sh.abort_flag, p.err, p.timeout_ns};
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
        if (!ALONE || warp < 4) softmax_role<D, E4M3, ALONE>(p, warp / 4, b, sh.part, tmem, sh.poison, wc);
    } else if (warp >= kExpandWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kExpandRegs));
        if constexpr (E4M3) expand_role<D, ALONE>(p, smem_u32(smem), b, sh.part, sh.poison, wc);
        else fix_role<D, ALONE>(p, smem_u32(smem), b, sh.fix, sh.poison, &sh.turn, wc);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            if (!ALONE || warp == kMmaWarp)
                mma_role<D, E4M3, ALONE>(p, warp - kMmaWarp, smem_u32(smem), b, sh.part, tmem, &sh.turn, wc);
        } else if (warp == kLoadWarp) {
            load_role<D, E4M3, ALONE>(p, &tq, &tk, &tv, smem_u32(smem), b, sh.fix, sh.part, wc);
        } else {
            list_role(p, b, sh.part, &sh.turn, wc);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, C::kTmemCols);
}

// Joins the parts of items that were cut: block (x, y) takes rows [8 y, 8 y + 8) of the item that
// begins in block x of the first kernel and goes on in the next ones, a thread 4 columns of a row.  The
// weights of all parts come first, the threads side by side: an item may lie in all blocks, and
// with one look at a part after the other its 76 parts took 40 us, 20 so.
constexpr int kJoinRows = 8;
template <int D>
__global__ void __launch_bounds__(kJoinRows * D / 4) paged_chunk_join_kernel(const __grid_constant__ PagedAttnParams p, int shares) {
    constexpr int kThreads = kJoinRows * D / 4, kLanes = kThreads / kJoinRows, kWarps = kThreads / 32;
    __shared__ float weight[kPagedMaxShares][kJoinRows], red[kWarps][kJoinRows];
    wait_primary();
    const PagedChunkPartial* parts = static_cast<const PagedChunkPartial*>(p.workspace);
    const int x = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const PagedChunkPartial* p0 = parts + 2 * x + (parts[2 * x + 1].b >= 0 ? 1 : 0);
    const int b = p0->b, pair = p0->pair, h = p0->h;
    if (b < 0 || !p0->begins) return;
    if (!RA_CHECKED(b < p.kv.batch && pair >= 0 && h >= 0 && h < p.kv.hkv, p.err, kSitePagedPartial)) return;
    const Chunk c = make_chunk(p, b, pair, paged_seq(p.kv, b));
    int n = 1;  // parts: p0, then the first ones of the blocks up to x + n - 1 (that have a filling)
    while (x + n < shares) {
        const int y = x + n + lane;
        const PagedChunkPartial* q = parts + 2 * y;
        const bool on = y < shares && (q->b == -2 || (q->b == b && q->pair == pair && q->h == h && !q->begins));
        const uint32_t v = __ballot_sync(0xffffffffu, on);
        n += v == 0xffffffffu ? 32 : __ffs(~v) - 1;
        if (v != 0xffffffffu) break;
    }
    const int r0 = blockIdx.y * kJoinRows, row8 = threadIdx.x % kJoinRows, r = r0 + row8;  // row of the two units
    const int col = threadIdx.x / kJoinRows;                                               // group of 4 columns
    const int unit = r0 / kTile, ru = r - unit * kTile, rows = p.unit_tokens * p.g;
    if (r0 - unit * kTile >= rows || c.ta + unit * p.unit_tokens + (r0 - unit * kTile) / p.g >= c.tb) return;
    auto part = [&](int k) { return k ? parts + 2 * (x + k) : p0; };
    float M = -INFINITY;
    for (int k = col; k < n; k += kLanes) {
        const float m = part(k)->b >= 0 ? part(k)->m[r] : NAN;  // (a block without a filling left nothing)
        weight[k][row8] = m;
        M = fmaxf(M, m);
    }
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
    if (lane < kJoinRows) red[warp][lane] = M;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red[w][row8]);
    float l = 0.f, lr = 0.f, acc[4] = {};
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
        const float m = weight[k][row8];
        if (m != m) continue;
        const PagedChunkPartial* q = part(k);
        const float f = paged_weight(m, M);
        const float4 v = q->o[col * (2 * kTile) + r];
        l = paged_add_weighted(l, f, q->l[r]);
        lr = paged_add_weighted(lr, f, q->lr[r]);
        acc[0] = paged_add_weighted(acc[0], f, v.x);
        acc[1] = paged_add_weighted(acc[1], f, v.y);
        acc[2] = paged_add_weighted(acc[2], f, v.z);
        acc[3] = paged_add_weighted(acc[3], f, v.w);
    }
    const int t = c.ta + unit * p.unit_tokens + ru / p.g;
    if (ru >= rows || t >= c.tb) return;
    const int tok = c.s.q0 + t, head = h * p.g + ru % p.g;
    paged_store4(p, tok, head, 4 * col, acc, lr == 0.f ? 0.f : 1.f / lr);
    if (col == 0) paged_store_lse(p, tok, head, M, l);
}

template <class... Args>
cudaError_t launch_dependent(void (*kern)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, bool E4M3, bool ALONE>
int launch_t(const PagedAttnParams& p, const PagedMaps& m, int shares, cudaStream_t stream) {
    using C = Cfg<D, E4M3, ALONE>;
    auto kern = paged_chunk_kernel<D, E4M3, ALONE>;
    static std::atomic<unsigned long long> ready{0};
    if (!once_a_device(ready, [&] {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess) return false;
            // the register split adds up only if the block starts with as many as it counts on (the build has checked it)
            cudaFuncAttributes a;
            return cudaFuncGetAttributes(&a, kern) == cudaSuccess && a.numRegs == C::kStartRegs;
        }))
        return -4;
    paged_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, shares);
    if (cudaGetLastError() != cudaSuccess) return -4;
    if (launch_dependent(kern, dim3(shares), C::kThreads, C::kSmemBytes, stream, p, m.q, m.k, m.v) != cudaSuccess) return -4;
    return launch_dependent(paged_chunk_join_kernel<D>, dim3(shares, 2 * kTile / kJoinRows), kJoinRows * D / 4, 0, stream, p,
                            shares) ==
                   cudaSuccess
               ? 0
               : -4;
}

}  // namespace

int launch_paged_chunk(const PagedAttnParams& p, const PagedMaps& m, int shares, cudaStream_t stream) {
    // (item_tokens: api.cu gave items one unit when no sequence has more than a unit's tokens)
    const bool alone = p.item_tokens == p.unit_tokens;
    if (p.kv.d == 128) {
        if (p.kv.e4m3) return alone ? launch_t<128, true, true>(p, m, shares, stream) : launch_t<128, true, false>(p, m, shares, stream);
        return alone ? launch_t<128, false, true>(p, m, shares, stream) : launch_t<128, false, false>(p, m, shares, stream);
    }
    if (p.kv.e4m3) return alone ? launch_t<64, true, true>(p, m, shares, stream) : launch_t<64, true, false>(p, m, shares, stream);
    return alone ? launch_t<64, false, true>(p, m, shares, stream) : launch_t<64, false, false>(p, m, shares, stream);
}

}  // namespace ra
