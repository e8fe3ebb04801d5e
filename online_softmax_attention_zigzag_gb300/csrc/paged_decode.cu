// paged_decode.cu -- attention of few rows over a paged K/V cache: the rows of one sequence and KV
// head (n_b tokens times g query heads) fill at most one 16-row matrix tile.
//
//     s_j = q . k_j,  out = sum_j 2^(c s_j - m) v_j / l,  l = sum_j 2^(c s_j - m),  c = log2 e
// Every K and V row is read once for at most 16 query rows: 16 * 4 * d FLOP for 4 * d bytes (2 * d
// in 8 bits), so HBM bounds it by far and everything else only has to keep out of the way:
//   * one persistent block an SM, of two or four groups of warps that have nothing to do with each other;
//     the tiles of 128 keys of all (sequence, KV head) pairs, in one line, are dealt out to the
//     groups in equal contiguous shares, so that one long context or a thousand
//     short ones load every SM alike.  A pair whose tiles lie in several shares leaves
//     partial results (O, m, l) in the workspace, which a second small kernel joins; a share
//     has at most two of these (its first and its last pair), so the workspace does not grow
//     with the lengths.
//   * a group's loading warp streams K and V tiles through its slots of shared memory with TMA, box
//     by box as the pages come (a box is gcd(page, 128) rows of one page), and runs on into the
//     next pair while the others finish the last.
//   * a group's two or four other warps compute, 64 or 32 keys of every tile each, with mma.sync: 8 rows
//     are a sixteenth of a tcgen05 tile, and S and P stay in registers between the two products.
//     Both products are transposed, S^T = K Q^T and O^T = V^T P^T, so that the keys and the elements
//     fill the 16 rows of the instruction and the query rows its 8 columns: up to 8 rows, the usual
//     case, then cost half the instructions and registers of S = Q K^T.  Each warp keeps its own
//     running max, sum and output; they meet once a pair.
// What a tile takes is a chain of latencies (copy, barrier, S, max, exponentials, P V), and so is what
// a pair takes (q, the meeting, the output): groups hide them behind one another.  One group of eight
// warps with the same 128 KB of slots, and four that took one line's tiles in turn, were slower:
//     64 x 16k keys of 8 heads, bf16             323 us, now 313 (6.5 TB/s)
//     8 x 128k keys, e4m3                        293 us, now 280 (7.0 TB/s)
//     48 windows of 4096 of 3k - 32k keys, e4m3   78 us, now  74
//     512 x 20 - 300 keys, e4m3                  181 us, now  76; bf16 173 and 127
//     32 x 16k keys of d = 64, e4m3              129 us, now  99; bf16 165 and 162 (6.6 TB/s)
//     one sequence of 777 keys                  13.0 us, now 11.7
// (Boxes that no row sees, behind sinks and before windows, are not loaded: windows 77.3 us with them, 76.0 without; in
// bf16 139.1 and 136.5.)
// The tensor cores truncate every addend of a sum, always towards zero, so a warp's sums end after kFold tiles at
// the latest: a longer part of a share goes in stretches, which are added up in fp32, rounded to nearest.
// bf16 cache: P goes into its product as two bf16 halves (p = hi + lo to 2^-15): the second product costs
// nothing here, the loads take longer.  hi is p cut off and lo a trifle above the rest, so that both are above
// zero where p is, and an infinite v makes out that infinity: infinity * 0, and infinities of both
// signs where lo is negative, would be no numbers.
// e4m3 cache: codes become fp16 (one instruction for two, exact), q is brought to fp16's range by
// a power of two per row (elements below 2^-28 of the row's largest lose bits), the K scale
// multiplies the score, and the V scale enters the exponent: with v_j = 2^(a_j) u_j,
//     p'_j = 2^(c s_j + a_j - m),  out = 2^m sum p'_j u_j / (2^ms l),  l = sum 2^(c s_j - ms)
// where m is the running max of c s_j + a_j and ms that of c s_j.  So p' fits fp16 whatever the
// scales are and keeps 11 bits down to 2^-20 of the largest contribution, and l loses nothing.
#include <cuda_bf16.h>

#include "paged.h"
#include "ptx_paged.cuh"

namespace ra {
namespace {

constexpr int kTile = kPagedTile;         // keys of a tile
constexpr int kRows = 16;
constexpr int kBar = 1;                   // named barrier of the computing warps
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;          // the running max moves when it is exceeded by more (log2)
constexpr float kAbove = 1.f + 0x1p-20f;  // keeps p - hi above zero where hi is p (2^-20 of p, far below lo's rounding)
// Tiles of a stretch.  With unequal weights and values of one sign 2^22 keys in one sum came out 0.7 % low in
// bf16 and 1.4 % in e4m3; in stretches of 256 tiles 0.005 % and 0.007 %, however many there are.  (Shares of
// ordinary calls are shorter: 8 x 128k keys in 8 bits are 108 tiles.)
constexpr int kFold = 256;
constexpr float kF16Up = 6.0f;            // p' is kept 2^6 times larger: at most 2^(8 + 6 + 1) in fp16

// NT: 8 query rows each
template <int D, bool E4M3, int NT>
struct Cfg {
    static constexpr int kSlotBytes = kTile * D * (E4M3 ? 1 : 2);
    // In 8 bits four groups of two warps, with 64 keys of a tile each (two groups with twice the tiles: 32 x 16k keys
    // 171 us instead of 174, 512 short sequences 95 instead of 76, d = 64 130 instead of 103); in bf16 two groups
    // of four (d = 64 with four: 165 us instead of 160; d = 128 has slots for two).
    static constexpr int kGroups = E4M3 ? 4 : 2;
    static constexpr int kDepth = D == 128 ? 1 : 2;           // tiles of a group in shared memory, 128 KB in all
    static constexpr int kGroupSlots = 2 * kDepth;            // a K and a V slot each
    static constexpr int kSlots = kGroups * kGroupSlots;
    static constexpr int kWarps = 8;                          // that compute
    static constexpr int kThreads = (kWarps + kGroups) * 32;  // and one that loads for every group
    static constexpr int kGroupWarps = kWarps / kGroups;
    static constexpr int kKeys = kTile / kGroupWarps;  // of a tile, for a warp
    static constexpr int kOStride = D + 4;             // keeps the fragments' stores off each other's banks
    static constexpr int kScaleBytes = kTile * 4;  // of a slot
    static constexpr int kScaleOff = kSlots * kSlotBytes;
    static constexpr int kOOff = kScaleOff + (E4M3 ? kSlots * kScaleBytes : 0);
    // the warps' results meet in a buffer of 8 rows a warp, rows 0-7 and then rows 8-15
    static constexpr int kMlOff = kOOff + kWarps * 8 * kOStride * 4;  // m, ms, l of every warp and row; bad values
    static constexpr int kPreOff = kMlOff + (3 * kWarps * kRows + kWarps) * 4;
    static constexpr int kFixedBytes = kPreOff + 1024;  // and 4 * (batch + 1) for the shares
};

// The key tiles of a sequence that some row sees: tiles [0, ns) hold the sinks, tiles from lo on the
// window (or everything).  At least one tile where there are rows, so that every row is
// written.
struct Tiles {
    int ns, lo, n;
};
__device__ __forceinline__ Tiles key_tiles(const PagedAttnParams& p, const PagedSeq& s) {
    Tiles t;
    const int first = p.window > 0 ? max(0, s.base - p.window + 1) : 0;
    const int hi = (s.L + kTile - 1) / kTile;
    t.lo = min(first / kTile, hi);
    t.ns = p.window > 0 ? min((min(p.sinks, s.L) + kTile - 1) / kTile, t.lo) : 0;
    t.n = s.T > 0 ? max(1, t.ns + hi - t.lo) : 0;
    return t;
}

// One share's part of one (sequence, head) pair: tiles [ta, tb) of its n.
struct Part {
    int b, h, ta, tb, n;
};

// Shares of the tiles, found by every block for itself: pre[b] = tiles of the sequences before b
// (of one head).  Returns their sum.
template <int kThreads>
__device__ int share_tiles(const PagedAttnParams& p, int* pre, int* scratch) {
    const int B = p.kv.batch, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    int base = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const int n = b < B ? key_tiles(p, paged_seq(p.kv, b)).n : 0;
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scratch[warp] = x;
        __syncthreads();
        int before = base, all = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            const int y = scratch[w];
            if (w < warp) before += y;
            all += y;
        }
        if (b < B) pre[b] = before + x - n;
        base += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) pre[B] = base;
    __syncthreads();
    return base;
}

// Walks the parts of a share [w0, w1): f(part) until it returns false.
template <class F>
__device__ __forceinline__ void for_each_part(const PagedAttnParams& p, const int* pre, long long w0, long long w1,
                                              F&& f) {
    if (w0 >= w1) return;
    const int H = p.kv.hkv;
    int lo = 0, hi = p.kv.batch;  // pre[lo] * H <= w0 < pre[hi] * H
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<long long>(pre[mid]) * H <= w0) lo = mid;
        else hi = mid;
    }
    Part q;
    q.b = lo;
    q.n = pre[lo + 1] - pre[lo];
    const long long in = w0 - static_cast<long long>(pre[lo]) * H;
    q.h = static_cast<int>(in / q.n);
    q.ta = static_cast<int>(in - static_cast<long long>(q.h) * q.n);
    long long w = w0;
    while (true) {
        q.tb = static_cast<int>(min(static_cast<long long>(q.n), q.ta + (w1 - w)));
        if (!RA_CHECKED(q.b >= 0 && q.b < p.kv.batch && q.h >= 0 && q.h < H && q.ta >= 0 && q.ta < q.tb && q.tb <= q.n, p.err, kSitePagedShare))
            return;
        if (!f(q)) return;
        w += q.tb - q.ta;
        if (w >= w1) return;
        q.ta = 0;
        if (++q.h == H) {
            q.h = 0;
            do ++q.b; while (pre[q.b + 1] == pre[q.b]);
            q.n = pre[q.b + 1] - pre[q.b];
        }
    }
}

// ------------------------------------------------------------------ the loading warp
template <int D, bool E4M3, int NT>
__device__ void load_role(const PagedAttnParams& p, const CUtensorMap* tk, const CUtensorMap* tv, uint32_t ring,
                          uint32_t scales, uint64_t* full, uint64_t* empty, const int* pre, long long w0, long long w1, const WaitCtl& wc) {
    using C = Cfg<D, E4M3, NT>;
    const PagedKV& kv = p.kv;
    const int lane = threadIdx.x & 31;
    const int rows = p.box_rows;          // of a box; a lane loads one
    const int boxes = kTile / rows;       // at most 8: pages are multiples of 16 rows
    const uint64_t policy = make_policy_evict_first();
    const int log_rows = 31 - __clz(rows);
    uint32_t n = 0;  // tiles so far
    int half = 0;
    bool ok = true;
    for_each_part(p, pre, w0, w1, [&](const Part& q) -> bool {
        const PagedSeq s = paged_seq(kv, q.b);
        const Tiles kt = key_tiles(p, s);
        // q on its way to L1 for the warps that compute, who come here later
        for (int i = lane; i < min(s.T, p.max_q) * p.g * (D / 32); i += 32) {
            const int r = i / (D / 32), t = r / p.g;
            if (!RA_CHECKED(paged_row_ok(kv, p.hq, s.q0 + t, q.h * p.g + r - t * p.g), p.err, kSitePagedToken)) continue;
            const uint16_t* src = static_cast<const uint16_t*>(p.q) + (s.q0 + t) * p.q_ts + (q.h * p.g + r - t * p.g) * p.q_hs;
            asm volatile("prefetch.global.L1 [%0];" ::"l"(src + (i % (D / 32)) * 32));
        }
        // the page of this lane's box, asked for a tile ahead and looked at only when it is needed
        int entry = -1, row = 0;
        const int first = p.window > 0 ? s.base - p.window + 1 : 0;
        auto look = [&](int t) {  // no page (so zeros, and no traffic) behind the last key and where no row looks
            const int pos = (t < kt.ns ? t : kt.lo + t - kt.ns) * kTile + lane * rows;
            entry = -1;
            row = 0;
            if (lane < boxes && pos < s.L && (pos + rows > first || pos < p.sinks)) entry = paged_entry(kv, q.b, pos, row);
        };
        look(q.ta);
        for (int t = q.ta; t < q.tb; ++t, ++n) {
            int pg = paged_checked(kv, entry);
            if (pg >= 0 && !RA_CHECKED(paged_place_ok(kv, pg, q.h, row, rows), p.err, kSitePagedBox)) pg = -1;
            const int y = q.h * kv.page + row;
            if (t + 1 < q.tb) look(t + 1);
#pragma unroll
            for (half = 0; half < 2; ++half) {  // K, then V
                const uint32_t slot = n % C::kDepth * 2 + half;
                ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], ((n / C::kDepth) & 1u) ^ 1u, wc, 20));
                if (!ok) return false;
                if (lane == 0) mbar_arrive_expect_tx(&full[slot], C::kSlotBytes);
                __syncwarp();
                if (lane < boxes) {
                    const CUtensorMap* map = half ? tv : tk;
                    const uint32_t dst = ring + slot * C::kSlotBytes;
                    if constexpr (E4M3) {
                        tma_load_3d(dst + lane * rows * D, map, &full[slot], 0, y, pg, policy);
                    } else {
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load_3d(dst + x * kTile * 128 + lane * rows * 128, map, &full[slot], x * 64, y, pg, policy);
                    }
                }
                if constexpr (E4M3) {  // four rows' scales a lane: TMA boxes take 45 ns each, and pages of 16 rows have 8
                    const int of = __shfl_sync(0xffffffffu, pg, (4 * lane) >> log_rows);
                    const int at = __shfl_sync(0xffffffffu, y, (4 * lane) >> log_rows) + ((4 * lane) & (rows - 1));
                    const float* src = half ? kv.v_scale : kv.k_scale;
                    const bool on = of >= 0 && RA_CHECKED(paged_place_ok(kv, of, q.h, at - q.h * kv.page, 4), p.err, kSitePagedPlace);
                    copy16_async(scales + slot * C::kScaleBytes + lane * 16, on ? src + of * (half ? kv.vs_ps : kv.ks_ps) + at : src, on);
                    copies_arrive(&full[slot]);
                }
            }
        }
        return true;
    });
    if (!ok && lane == 0) {  // let the copies in flight land before the block ends
        const uint32_t all = 2 * n + half;  // tiles asked for, K and V
        for (uint32_t i = all > C::kGroupSlots ? all - C::kGroupSlots : 0; i < all; ++i)
            drain_wait(&full[i % C::kGroupSlots], (i / C::kGroupSlots) & 1u, wc.timeout_ns);
    }
}

// ------------------------------------------------------------------ the computing warps
// Byte offset of the 16-byte chunk `c` of key row r in a tile as TMA stored it (128-byte swizzle;
// 64-byte for rows of 64 bytes).
template <int D, bool E4M3>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if constexpr (!E4M3) return (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    else if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
    else return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// What turns sum p' u into out.
template <bool E4M3>
__device__ __forceinline__ float out_factor(float M, float Ms, float L) {
    if (L == 0.f) return 0.f;
    return (E4M3 && M != -INFINITY) ? ex2(M - kF16Up - Ms) / L : 1.f / L;
}

// Largest of this lane's scores of its row e of row group x.
template <int NB, int NT>
__device__ __forceinline__ float lane_max(const float (&sc)[NB][NT][4], int x, int e) {
    float m = fmaxf(sc[0][x][e], sc[0][x][2 + e]);
#pragma unroll
    for (int n = 1; n < NB; ++n) m = fmaxf(m, fmaxf(sc[n][x][e], sc[n][x][2 + e]));
    return m;
}

__device__ __forceinline__ float bf16_add_nonfinite(float acc, uint16_t bits) {
    return (bits & 0x7f80u) == 0x7f80u ? acc + __uint_as_float(static_cast<uint32_t>(bits) << 16) : acc;
}

// Joins the group's warps' results for tiles [ta, tb) of part q, which is all of it or a stretch: rows 8 round .. + 8 of
// the pair, in turn.  Into the outputs, or, if others have tiles of the pair too or more stretches
// follow, into the workspace, where the stretches before this one are.
template <int D, bool E4M3, int NT>
__device__ __forceinline__ void join_rows(const PagedAttnParams& p, const uint8_t* smem, Part q, int ta, int tb, int slot, int round) {
    using C = Cfg<D, E4M3, NT>;
    constexpr int kWarps = C::kGroupWarps;
    const PagedKV& kv = p.kv;
    const int warp = threadIdx.x / 32 % kWarps, lane = threadIdx.x & 31, w0 = threadIdx.x / 32 - warp;
    const float* so = reinterpret_cast<const float*>(smem + C::kOOff) + w0 * 8 * C::kOStride;
    const float* sm = reinterpret_cast<const float*>(smem + C::kMlOff) + w0 * kRows;
    const float* sms = sm + C::kWarps * kRows;
    const float* sl = sms + C::kWarps * kRows;
    const int* sbad = reinterpret_cast<const int*>(smem + C::kMlOff) + 3 * C::kWarps * kRows + w0;
    const PagedSeq s = paged_seq(kv, q.b);
    const int T = min(s.T, p.max_q), R = T * p.g;
    const bool cut = q.ta > 0 || q.tb < q.n, keep = cut || tb < q.tb, more = ta > q.ta;
    if (!RA_CHECKED(slot >= 0 && slot < 2 * C::kGroups * static_cast<int>(gridDim.x) && R <= kRows, p.err, kSitePagedPartial)) return;
    PagedPartial* part = static_cast<PagedPartial*>(p.workspace) + slot;
    if (cut && warp == 0 && lane == 0) {
        part->b = q.b;
        part->h = q.h;
        part->begins = q.ta == 0;
    }
    for (int row8 = warp; row8 < 8; row8 += kWarps) {
        const int r = row8 + 8 * round;
        if (r >= R) break;
        float M = -INFINITY, Ms = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            M = fmaxf(M, sm[w * kRows + r]);
            Ms = fmaxf(Ms, sms[w * kRows + r]);
        }
        float f[kWarps], L = 0.f, f0 = 0.f;
        if (more) {
            M = fmaxf(M, part->m[r]);
            Ms = fmaxf(Ms, part->ms[r]);
            f0 = paged_weight(part->m[r], M);
            L = paged_add_weighted(L, paged_weight(part->ms[r], Ms), part->l[r]);
        }
        bool any_bad = false;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            f[w] = paged_weight(sm[w * kRows + r], M);
            L = paged_add_weighted(L, paged_weight(sms[w * kRows + r], Ms), sl[w * kRows + r]);
            any_bad |= sbad[w] != 0;
        }
        const int t = r / p.g, head = q.h * p.g + r - t * p.g, tok = s.q0 + t;
        for (int d = 4 * lane; d < D; d += 128) {
            float acc[4] = {};
            if (more) {
                const float4 v = *reinterpret_cast<const float4*>(&part->o[r * kPagedMaxD + d]);
                acc[0] = f0 * v.x;
                acc[1] = f0 * v.y;
                acc[2] = f0 * v.z;
                acc[3] = f0 * v.w;
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 v = *reinterpret_cast<const float4*>(so + (w * 8 + row8) * C::kOStride + d);
                acc[0] = fmaf(f[w], v.x, acc[0]);
                acc[1] = fmaf(f[w], v.y, acc[1]);
                acc[2] = fmaf(f[w], v.z, acc[2]);
                acc[3] = fmaf(f[w], v.w, acc[3]);
            }
            if (!E4M3 && any_bad) {  // values that are no numbers, of the keys this row sees
                const Tiles kt = key_tiles(p, s);
                const int see_lo = s.base + T - p.window;
                const int i = s.base + t, rhi = p.causal ? i + 1 : s.L, rlo = p.window > 0 ? i - p.window + 1 : 0;
                for (int tt = ta; tt < tb; ++tt) {
                    const int j0 = (tt < kt.ns ? tt : kt.lo + tt - kt.ns) * kTile;
                    if (j0 + kTile <= (p.causal ? s.base + 1 : s.L) && (p.window == 0 || j0 >= see_lo || j0 + kTile <= p.sinks))
                        continue;  // its values went into the product as they are
                    for (int j = j0; j < min(j0 + kTile, rhi); ++j) {
                        if (p.window > 0 && j < rlo && j >= p.sinks) continue;
                        int in;
                        const int pg = paged_page(kv, q.b, j, in);
                        if (pg < 0 || !RA_CHECKED(paged_place_ok(kv, pg, q.h, in), p.err, kSitePagedPlace)) continue;
                        const uint16_t* v = static_cast<const uint16_t*>(kv.v) + pg * kv.v_ps + (static_cast<long long>(q.h) * kv.page + in) * D + d;
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[e] = bf16_add_nonfinite(acc[e], v[e]);
                    }
                }
            }
            if (keep) *reinterpret_cast<float4*>(&part->o[r * kPagedMaxD + d]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            else paged_store4(p, tok, head, d, acc, out_factor<E4M3>(M, Ms, L));
        }
        __syncwarp();  // all lanes have what the stretches before left
        if (lane == 0) {
            if (keep) {
                part->m[r] = M;
                part->ms[r] = Ms;
                part->l[r] = L;
            } else {
                paged_store_lse(p, tok, head, Ms, L);
            }
        }
    }
}

template <int D, bool E4M3, int NT>
__device__ void compute_role(const PagedAttnParams& p, uint8_t* smem, uint64_t* full, uint64_t* empty, const int* pre,
                             int share, long long w0, long long w1, const WaitCtl& wc) {
    using C = Cfg<D, E4M3, NT>;
    constexpr int kWarps = C::kWarps, NB = C::kKeys / 16;
    const PagedKV& kv = p.kv;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, c4 = lane & 3, r8 = lane >> 2;
    const int grp = warp / C::kGroupWarps, key0 = (warp % C::kGroupWarps) * C::kKeys;  // this warp's keys of a tile
    const uint32_t ring = smem_u32(smem) + grp * C::kGroupSlots * C::kSlotBytes;
    float* so = reinterpret_cast<float*>(smem + C::kOOff);
    float* sm = reinterpret_cast<float*>(smem + C::kMlOff);
    float* sms = sm + kWarps * kRows;
    float* sl = sms + kWarps * kRows;
    int* sbad = reinterpret_cast<int*>(sl + kWarps * kRows);
    const float* scales = reinterpret_cast<const float*>(smem + C::kScaleOff + grp * C::kGroupSlots * C::kScaleBytes) + key0 + r8;  // its
    uint32_t done = 0;  // tiles so far
    bool ok = true;
    int place = 2 * share;  // for a part that is cut: the first one's, then the others'
    auto stretch = [&](const Part& q, int ta, int tb) -> bool {  // tiles [ta, tb) of part q
        const PagedSeq s = paged_seq(kv, q.b);
        const Tiles kt = key_tiles(p, s);
        const int T = min(s.T, p.max_q), R = T * p.g;
        // q as the B operand: this lane has elements of row 8 x + r8
        uint32_t qb[NT][D / 16][2];
        float cs[NT][2];        // e4m3: log2 e times what row 8 x + 2 c4 + e was scaled down by
        int hi[NT][2], lo[NT][2];  // the keys that row sees: below hi, from lo on or sinks
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const int r = 8 * x + r8, t = r / p.g;
            const uint16_t* src = static_cast<const uint16_t*>(p.q) + (s.q0 + t) * p.q_ts + (q.h * p.g + r - t * p.g) * p.q_hs;
            const bool live = r < R && RA_CHECKED(paged_row_ok(kv, p.hq, s.q0 + t, q.h * p.g + r - t * p.g), p.err, kSitePagedToken);
            if constexpr (E4M3) {
                uint2 w[D / 16];
                uint32_t m = 0;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    w[k] = live ? __ldg(reinterpret_cast<const uint2*>(src + 16 * k + 4 * c4)) : make_uint2(0, 0);
                    m = __vmaxu2(m, __vmaxu2(w[k].x & 0x7fff7fffu, w[k].y & 0x7fff7fffu));
                }
                m = max(m & 0xffffu, m >> 16);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                // largest element in [2^13, 2^14): exponent field m >> 7 becomes 127 + 13
                const int e = min(max(static_cast<int>(m >> 7), 16), 254);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 + 127 - e) << 23);
                const float down = kLog2e * __uint_as_float(static_cast<uint32_t>(e - 13) << 23);
                cs[x][0] = __shfl_sync(0xffffffffu, down, 8 * c4);
                cs[x][1] = __shfl_sync(0xffffffffu, down, 8 * c4 + 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qb[x][k][0] = pack_f16x2(__uint_as_float(w[k].x << 16) * up, __uint_as_float(w[k].x & 0xffff0000u) * up);
                    qb[x][k][1] = pack_f16x2(__uint_as_float(w[k].y << 16) * up, __uint_as_float(w[k].y & 0xffff0000u) * up);
                }
            } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qb[x][k][0] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * c4)) : 0u;
                    qb[x][k][1] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 8 + 2 * c4)) : 0u;
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = s.base + (8 * x + 2 * c4 + e) / p.g;
                hi[x][e] = p.causal ? i + 1 : s.L;
                lo[x][e] = p.window > 0 ? i - p.window + 1 : 0;
            }
        }
        float o[D / 16][NT][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][x][e] = 0.f;
        float m[NT][2], ms[NT][2], l[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[x][e] = ms[x][e] = -INFINITY;
                l[x][e] = 0.f;
            }
        bool bad_v = false;  // a value that is no number, in a tile that not every row sees whole
        const int see_lo = s.base + T - p.window;  // the window of the last row begins here
        for (int t = ta; t < tb; ++t, ++done) {
            const int j0 = (t < kt.ns ? t : kt.lo + t - kt.ns) * kTile;
            // does every row see every key of the tile?
            const bool whole = j0 + kTile <= (p.causal ? s.base + 1 : s.L) &&
                               (p.window == 0 || j0 >= see_lo || j0 + kTile <= p.sinks);
            // ---- S^T = K Q^T: element e is key r8 + 8 (e / 2) of the 16, row 2 c4 + e % 2 of the 8
            const uint32_t slot = done % C::kDepth * 2, parity = (done / C::kDepth) & 1u;  // K's, V's is the next
            ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], parity, wc));
            if (!ok) break;
            float sc[NB][NT][4] = {};
            uint32_t base = ring + slot * C::kSlotBytes;
            // matrices: keys 0-7 and 8-15 of a 16-byte chunk, then of the next chunk
            if constexpr (E4M3) {
#pragma unroll
                for (int x = 0; x < D / 32; ++x)
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        uint32_t b[4];
                        ldmatrix4(b, base + chunk_at<D, E4M3>(key0 + 16 * n + (lane & 15), 2 * x + (lane >> 4)));
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t a[4] = {e4m3x2_f16x2(b[2 * y] & 0xffffu), e4m3x2_f16x2(b[2 * y + 1] & 0xffffu),
                                                   e4m3x2_f16x2(b[2 * y] >> 16), e4m3x2_f16x2(b[2 * y + 1] >> 16)};
#pragma unroll
                            for (int z = 0; z < NT; ++z) mma16816<true>(sc[n][z], a, qb[z][2 * x + y][0], qb[z][2 * x + y][1]);
                        }
                    }
                const float* f = scales + slot * kTile;
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const float k0 = f[16 * n], k1 = f[16 * n + 8];
#pragma unroll
                    for (int z = 0; z < NT; ++z) {
                        sc[n][z][0] *= k0 * cs[z][0];
                        sc[n][z][1] *= k0 * cs[z][1];
                        sc[n][z][2] *= k1 * cs[z][0];
                        sc[n][z][3] *= k1 * cs[z][1];
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        uint32_t a[4];
                        ldmatrix4(a, base + chunk_at<D, E4M3>(key0 + 16 * n + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
                        for (int z = 0; z < NT; ++z) mma16816<false>(sc[n][z], a, qb[z][k][0], qb[z][k][1]);
                    }
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int z = 0; z < NT; ++z)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[n][z][e] *= kLog2e;
            }
            // (a slot is handed back when what was loaded from it has been used)
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
            base += C::kSlotBytes;
            const int jk = j0 + key0;  // the warp's first key
            if (!whole) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int z = 0; z < NT; ++z)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = jk + 16 * n + r8 + 8 * (e >> 1);
                            const bool see = j < hi[z][e & 1] && (p.window == 0 || j >= lo[z][e & 1] || j < p.sinks);
                            if (!see) sc[n][z][e] = -INFINITY;
                        }
            }
            // ---- e4m3: l, with a running max of each lane's own
            if constexpr (E4M3) {
#pragma unroll
                for (int z = 0; z < NT; ++z)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mx = lane_max(sc, z, e);
                        if (mx > ms[z][e] + kRescale || (ms[z][e] == -INFINITY && mx > ms[z][e])) {
                            l[z][e] *= ex2(ms[z][e] - mx);
                            ms[z][e] = mx;
                        }
                        const float nm = ms[z][e] == -INFINITY ? 0.f : -ms[z][e];
#pragma unroll
                        for (int n = 0; n < NB; ++n) l[z][e] += ex2(sc[n][z][e] + nm) + ex2(sc[n][z][2 + e] + nm);
                    }
            }
            ok = __all_sync(0xffffffffu, mbar_wait(&full[slot + 1], parity, wc));
            if (!ok) break;
            // ---- e4m3: the V scales join the scores as exponents.  (No number stays none; log2 0 = -inf,
            // for the zeros of a page that is none.)
            if constexpr (E4M3) {
                const float* f = scales + (slot + 1) * kTile;
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const float v0 = lg2(f[16 * n]), v1 = lg2(f[16 * n + 8]);
#pragma unroll
                    for (int z = 0; z < NT; ++z)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float y = sc[n][z][e] + (e < 2 ? v0 : v1);
                            sc[n][z][e] = whole || sc[n][z][e] != -INFINITY ? y : -INFINITY;  // masked stays masked
                        }
                }
            }
            // ---- running max of the row (shared by the eight lanes that hold it), p, sums
            bool raise = false;
            float mx[NT][2];
#pragma unroll
            for (int z = 0; z < NT; ++z)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float y = lane_max(sc, z, e);
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                    mx[z][e] = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                    raise |= mx[z][e] > m[z][e] + kRescale || (m[z][e] == -INFINITY && mx[z][e] > m[z][e]);
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int z = 0; z < NT; ++z)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool up = mx[z][e] > m[z][e];  // (any rise will do once one is due)
                        const float f = up ? ex2(m[z][e] - mx[z][e]) : 1.f;
                        if (up) m[z][e] = mx[z][e];
                        if (!E4M3) l[z][e] *= f;
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) {
                            o[i][z][e] *= f;
                            o[i][z][2 + e] *= f;
                        }
                    }
            }
            // P^T as the B operand: pairs of rows become pairs of keys
            uint32_t pa[NB][NT][2], pb[NB][NT][2];
#pragma unroll
            for (int z = 0; z < NT; ++z) {
                const float n0 = (E4M3 ? kF16Up : 0.f) - (m[z][0] == -INFINITY ? 0.f : m[z][0]);
                const float n1 = (E4M3 ? kF16Up : 0.f) - (m[z][1] == -INFINITY ? 0.f : m[z][1]);
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float a = ex2(sc[n][z][2 * h] + n0), b = ex2(sc[n][z][2 * h + 1] + n1);
                        if constexpr (E4M3) {
                            pa[n][z][h] = transpose8(pack_f16x2(a, b));
                        } else {
                            l[z][0] += a;
                            l[z][1] += b;
                            const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
                            pa[n][z][h] = transpose8(__byte_perm(ua, ub, 0x7632));
                            pb[n][z][h] = transpose8(pack_bf16x2(fmaf(a, kAbove, -__uint_as_float(ua & 0xffff0000u)),
                                                                 fmaf(b, kAbove, -__uint_as_float(ub & 0xffff0000u))));
                        }
                    }
            }
            // ---- O^T += V^T P^T; values of keys that no row sees count as zero, whatever they hold
            uint32_t keep[NB][2];  // of the key pairs 2 c4 of the first and of the second 8
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    keep[n][h] = 0xffffffffu;
                    if (!whole) {
                        const int j = jk + 16 * n + 8 * h + 2 * c4;
                        const int wlo = p.window > 0 ? s.base - p.window + 1 : 0;
                        const bool a = j < s.L && (j >= wlo || j < p.sinks);
                        const bool b = j + 1 < s.L && (j + 1 >= wlo || j + 1 < p.sinks);
                        keep[n][h] = (a ? 0xffffu : 0u) | (b ? 0xffff0000u : 0u);
                    }
                }
            if constexpr (E4M3) {
                // matrices: keys 0-7 and 8-15 of a chunk of 16 elements, then of the next; the operand's rows
                // 0-7 are a chunk's even elements, 8-15 its odd ones
#pragma unroll
                for (int x = 0; x < D / 32; ++x)
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        uint32_t b[4];
                        ldmatrix4_t(b, base + chunk_at<D, E4M3>(key0 + 16 * n + (lane & 15), 2 * x + (lane >> 4)));
                        if (!whole) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) b[e] &= keep[n][e & 1];
                        }
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t u = __byte_perm(b[2 * y], 0, 0x3120), v = __byte_perm(b[2 * y + 1], 0, 0x3120);
                            const uint32_t a[4] = {e4m3x2_f16x2(u & 0xffffu), e4m3x2_f16x2(u >> 16), e4m3x2_f16x2(v & 0xffffu),
                                                   e4m3x2_f16x2(v >> 16)};
#pragma unroll
                            for (int z = 0; z < NT; ++z) mma16816<true>(o[2 * x + y][z], a, pa[n][z][0], pa[n][z][1]);
                        }
                    }
            } else {
                // matrices: elements 0-7 and 8-15 of 16 for keys 0-7, then for keys 8-15
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        uint32_t a[4];
                        ldmatrix4_t(a, base + chunk_at<D, E4M3>(key0 + 16 * n + (lane & 7) + ((lane >> 4) << 3), 2 * x + ((lane >> 3) & 1)));
                        if (!whole) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                a[e] &= keep[n][e >> 1];
                                if (T > 1) {
                                    const uint32_t bad = ((a[e] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
                                                         ((a[e] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
                                    if (bad) bad_v = true;
                                    a[e] &= ~bad;
                                }
                            }
                        }
#pragma unroll
                        for (int z = 0; z < NT; ++z) {
                            mma16816<false>(o[x][z], a, pa[n][z][0], pa[n][z][1]);
                            mma16816<false>(o[x][z], a, pb[n][z][0], pb[n][z][1]);
                        }
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot + 1]);
        }
        // ---- the group's warps' results meet: rows 0-7, then rows 8-15
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if constexpr (E4M3) {  // the lanes' sums to one max
                    float top = fmaxf(ms[x][e], __shfl_xor_sync(0xffffffffu, ms[x][e], 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    if (ms[x][e] != -INFINITY) l[x][e] *= ex2(ms[x][e] - top);
                    ms[x][e] = top;
                } else {
                    ms[x][e] = m[x][e];
                }
                l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], 4);
                l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], 8);
                l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], 16);
                if (r8 == 0) {
                    sm[warp * kRows + 8 * x + 2 * c4 + e] = m[x][e];
                    sms[warp * kRows + 8 * x + 2 * c4 + e] = ms[x][e];
                    sl[warp * kRows + 8 * x + 2 * c4 + e] = l[x][e];
                }
            }
        if (lane == 0) sbad[warp] = 0;
        __syncwarp();
        if (bad_v) sbad[warp] = 1;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            float* dst = so + (warp * 8 + 2 * c4) * C::kOStride;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if constexpr (E4M3) {
                        *reinterpret_cast<float2*>(dst + e * C::kOStride + 16 * i + 2 * r8) = make_float2(o[i][x][e], o[i][x][2 + e]);
                    } else {
                        dst[e * C::kOStride + 16 * i + r8] = o[i][x][e];
                        dst[e * C::kOStride + 16 * i + 8 + r8] = o[i][x][2 + e];
                    }
                }
            // (a warp that gave up still comes here, so that none waits for it)
            if (!named_bar_and(kBar + grp, C::kGroupWarps * 32, ok)) return false;
            join_rows<D, E4M3, NT>(p, smem, q, ta, tb, place, x);
            named_bar_sync(kBar + grp, C::kGroupWarps * 32);  // the buffer is free again
        }
        return true;
    };
    for_each_part(p, pre, w0, w1, [&](const Part& q) -> bool {
        for (int ta = q.ta; ta < q.tb; ta += kFold)
            if (!stretch(q, ta, min(q.tb, ta + kFold))) return false;
        place = 2 * share + 1;
        return true;
    });
}

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(Cfg<D, E4M3, NT>::kThreads, 1)
    paged_decode_kernel(const __grid_constant__ PagedAttnParams p, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv) {
    using C = Cfg<D, E4M3, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[C::kSlots];
    __shared__ __align__(8) uint64_t empty[C::kSlots];
    __shared__ int scratch[C::kThreads / 32];
    __shared__ int abort_flag;
    int* pre = reinterpret_cast<int*>(smem + C::kPreOff);
    launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(&full[s], E4M3 ? 1 + 32 : 1);  // the tile's bytes, and every lane's scales
            mbar_init(&empty[s], C::kGroupWarps);
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    const long long W = static_cast<long long>(share_tiles<C::kThreads>(p, pre, scratch)) * p.kv.hkv;
    // Every group has a share; the first W % shares take one tile more, those without any are the last
    // ones, so share i is group i / grid's of block i % grid: a few tiles go to as many SMs.
    const int warp = threadIdx.x / 32;
    const bool loads = warp >= C::kWarps;
    const int grp = loads ? warp - C::kWarps : warp / C::kGroupWarps, share = grp * gridDim.x + blockIdx.x;
    const int slot0 = grp * C::kGroupSlots;
    const long long each = W / (C::kGroups * gridDim.x), more = W % (C::kGroups * gridDim.x);
    const long long w0 = share * each + min(static_cast<long long>(share), more), w1 = w0 + each + (share < more ? 1 : 0);
    PagedPartial* parts = static_cast<PagedPartial*>(p.workspace);
    if (loads && (threadIdx.x & 31) < 2) parts[2 * share + (threadIdx.x & 31)].b = -1;  // until a cut pair says otherwise
    __syncthreads();
    const WaitCtl wc{&abort_flag, p.err, p.timeout_ns};
    if (loads)
        load_role<D, E4M3, NT>(p, &tk, &tv, smem_u32(smem) + slot0 * C::kSlotBytes, smem_u32(smem) + C::kScaleOff + slot0 * C::kScaleBytes,
                               full + slot0, empty + slot0, pre, w0, w1, wc);
    else
        compute_role<D, E4M3, NT>(p, smem, full + slot0, empty + slot0, pre, share, w0, w1, wc);
}

// Joins the parts of pairs that were cut.  Block (x, r): if a pair begins in share x and goes on in share
// x + 1, row r of that pair.
template <int D, bool E4M3>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedAttnParams p, int shares) {
    constexpr int kSub = 8;
    __shared__ float so[kSub][D], sl[kSub];
    wait_primary();
    const PagedPartial* parts = static_cast<const PagedPartial*>(p.workspace);
    const int x = blockIdx.x, r = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int i0 = parts[2 * x + 1].b >= 0 ? 2 * x + 1 : 2 * x;  // the pair of x that goes on: its last cut part
    const int b = parts[i0].b, h = parts[i0].h;
    if (b < 0 || !parts[i0].begins) return;
    if (!RA_CHECKED(b < p.kv.batch && h >= 0 && h < p.kv.hkv, p.err, kSitePagedPartial)) return;
    int n = 1;  // parts: i0, then the first of every share up to x + n - 1
    while (x + n < shares) {
        const int y = x + n + lane;
        const PagedPartial* q = parts + 2 * y;
        const bool on = y < shares && q->b == b && q->h == h && !q->begins;
        const uint32_t v = __ballot_sync(0xffffffffu, on);
        n += v == 0xffffffffu ? 32 : __ffs(~v) - 1;
        if (v != 0xffffffffu) break;
    }
    const PagedSeq s = paged_seq(p.kv, b);
    const int R = min(s.T, p.max_q) * p.g;
    auto part = [&](int k) { return parts + (k == 0 ? i0 : 2 * (x + k)); };
    if (gridDim.y == 1) {
        // a row a warp, a part a lane for the weights; the launch says so where pairs have few parts on average
        for (int r = warp; r < R; r += kSub) {
            float M = -INFINITY, Ms = -INFINITY;
            for (int k = lane; k < n; k += 32) {
                M = fmaxf(M, part(k)->m[r]);
                Ms = fmaxf(Ms, part(k)->ms[r]);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                Ms = fmaxf(Ms, __shfl_xor_sync(0xffffffffu, Ms, o));
            }
            float l = 0.f, acc[4] = {};
#pragma unroll 8
            for (int k = 0; k < n; ++k) {
                const PagedPartial* q = part(k);
                const float f = paged_weight(q->m[r], M);
                l = paged_add_weighted(l, paged_weight(q->ms[r], Ms), q->l[r]);
                if (4 * lane < D) {
                    const float4 v = *reinterpret_cast<const float4*>(&q->o[r * kPagedMaxD + 4 * lane]);
                    acc[0] = fmaf(f, v.x, acc[0]);
                    acc[1] = fmaf(f, v.y, acc[1]);
                    acc[2] = fmaf(f, v.z, acc[2]);
                    acc[3] = fmaf(f, v.w, acc[3]);
                }
            }
            const int t = r / p.g, head = h * p.g + r - t * p.g, tok = s.q0 + t;
            if (4 * lane < D) paged_store4(p, tok, head, 4 * lane, acc, out_factor<E4M3>(M, Ms, l));
            if (lane == 0) paged_store_lse(p, tok, head, Ms, l);
        }
        return;
    }
    const int t = r / p.g;
    if (r >= R) return;
    float M = -INFINITY, Ms = -INFINITY;
    for (int k = lane; k < n; k += 32) {
        const PagedPartial* q = part(k);
        M = fmaxf(M, q->m[r]);
        Ms = fmaxf(Ms, q->ms[r]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        Ms = fmaxf(Ms, __shfl_xor_sync(0xffffffffu, Ms, o));
    }
    float l = 0.f, acc[4] = {};
#pragma unroll 4
    for (int k = warp; k < n; k += kSub) {
        const PagedPartial* q = part(k);
        const float f = paged_weight(q->m[r], M);
        l = paged_add_weighted(l, paged_weight(q->ms[r], Ms), q->l[r]);
        if (4 * lane < D) {
            const float4 v = *reinterpret_cast<const float4*>(&q->o[r * kPagedMaxD + 4 * lane]);
            acc[0] = fmaf(f, v.x, acc[0]);
            acc[1] = fmaf(f, v.y, acc[1]);
            acc[2] = fmaf(f, v.z, acc[2]);
            acc[3] = fmaf(f, v.w, acc[3]);
        }
    }
    if (4 * lane < D) *reinterpret_cast<float4*>(&so[warp][4 * lane]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if (lane == 0) sl[warp] = l;
    __syncthreads();
    if (warp != 0) return;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kSub; ++w) l += sl[w];
    const int head = h * p.g + r - t * p.g, tok = s.q0 + t;
    if (4 * lane < D) {
        float v[4] = {};
#pragma unroll
        for (int w = 0; w < kSub; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += so[w][4 * lane + e];
        paged_store4(p, tok, head, 4 * lane, v, out_factor<E4M3>(M, Ms, l));
    }
    if (lane == 0) paged_store_lse(p, tok, head, Ms, l);
}

template <int D, bool E4M3, int NT>
int launch_t(const PagedAttnParams& p, const PagedMaps& m, int blocks, cudaStream_t stream) {
    using C = Cfg<D, E4M3, NT>;
    const int shares = blocks * C::kGroups;
    static_assert(C::kGroups <= kPagedMaxGroups, "room for their results");
    auto kern = paged_decode_kernel<D, E4M3, NT>;
    const int bytes = C::kFixedBytes + 4 * (p.kv.batch + 1);
    static std::atomic<unsigned long long> ready{0};
    if (!once_a_device(ready, [&] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        C::kFixedBytes + 4 * (kPagedMaxBatch + 1)) == cudaSuccess;
        }))
        return -4;
    kern<<<blocks, C::kThreads, bytes, stream>>>(p, m.k, m.v);
    if (cudaGetLastError() != cudaSuccess) return -4;
    cudaLaunchConfig_t cfg = {};
    // Fewer than 8 parts a pair on average: one block for all rows of a pair; else one for each row.  (All rows against
    // a row a block: 64 x 16k keys of 8 heads 314 and 319 us, 48 windows in e4m3 76 and 84, one
    // sequence of 128k keys 102 and 94, in e4m3 77 and 59; near the border level: 6 x 16k 73 and 73.)
    cfg.gridDim = dim3(shares, 8LL * p.kv.batch * p.kv.hkv >= shares ? 1 : p.max_q * p.g);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, E4M3>, p, shares) == cudaSuccess ? 0 : -4;
}

}  // namespace

int launch_paged_decode(const PagedAttnParams& p, const PagedMaps& m, int blocks, cudaStream_t stream) {
    const bool one = p.max_q * p.g <= 8;
    if (p.kv.d == 128) {
        if (p.kv.e4m3) return one ? launch_t<128, true, 1>(p, m, blocks, stream) : launch_t<128, true, 2>(p, m, blocks, stream);
        return one ? launch_t<128, false, 1>(p, m, blocks, stream) : launch_t<128, false, 2>(p, m, blocks, stream);
    }
    if (p.kv.e4m3) return one ? launch_t<64, true, 1>(p, m, blocks, stream) : launch_t<64, true, 2>(p, m, blocks, stream);
    return one ? launch_t<64, false, 1>(p, m, blocks, stream) : launch_t<64, false, 2>(p, m, blocks, stream);
}

}  // namespace ra
