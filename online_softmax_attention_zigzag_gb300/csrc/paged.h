// paged.h -- parameter block, launchers and index arithmetic of the paged K/V cache
// (ringattn_cache_append, ringattn_cache_read, ringattn_fwd_paged).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "fastdiv.h"
#include "internal.h"

namespace ra {

// Sets a kernel up once a device (at most 64 of them, as everywhere): f() returns whether it worked.
template <class F>
bool once_a_device(std::atomic<unsigned long long>& done, F&& f) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (!f()) return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

// Sites of the check build (internal.h): every index that the paged kernels derive from the batch's arrays
// and their own division of the work.
enum PagedCheckSite : int {
    kSitePagedToken = 51,  // a row of the caller's k, v or q, and of cache_read's output
    kSitePagedPlace = 52,  // a row of the pool and its scale
    kSitePagedBox = 53,    // a TMA box of the pool
    kSitePagedShare = 54,  // a block's or group's part of the work
    kSitePagedPartial = 55,  // its place among the partial results
    kSitePagedOut = 56       // a row of out and lse
};

constexpr int kPagedMaxBatch = 4096;  // RINGATTN_PAGED_MAX_BATCH
constexpr int kPagedTile = 128;       // keys of a tile
constexpr int kPagedMaxD = 128;
constexpr int kPagedMaxShares = 160;  // most blocks of an attention kernel
constexpr int kPagedMaxGroups = 4;    // of a few-row block, with a share each
constexpr int kPagedFewRows = 16;     // rows of one sequence and KV head that the few-row kernel takes

// What a share of the few-row kernel's work leaves of a (sequence, KV head) pair that others have tiles
// of too: row r's sum of p v with weights 2^(x - m), and sum of p with weights 2^(x - ms).
struct PagedPartial {
    int b, h, begins, pad;  // b < 0: none; begins: the pair's first tile is in it
    float m[kPagedFewRows], ms[kPagedFewRows], l[kPagedFewRows];
    float o[kPagedFewRows * kPagedMaxD];
};

// The cache and the batch that uses it (ra_paged_kv, checked).  Strides are in elements.
struct PagedKV {
    void* k;
    void* v;
    float* k_scale;  // null for bf16
    float* v_scale;
    long long k_ps, v_ps, ks_ps, vs_ps;  // from page to page
    const int* table;                    // [batch, max_pages], rows table_stride apart
    const int* cu;                       // [batch + 1]
    const int* len;                      // [batch]
    long long table_stride;
    int n_pages, page, hkv, d, e4m3, batch, max_pages;
    int total;       // rows of the caller's token tensors
    FastDiv by_page;
};

// The same of an item (two units of 128 rows) of the chunk kernel: l sums the exact p, lr the p as
// rounded for the product with V.
struct PagedChunkPartial {
    int b, pair, h, begins;
    float m[2 * 128], l[2 * 128], lr[2 * 128];
    float4 o[kPagedMaxD / 4 * 2 * 128];  // [group of 4 columns][row]
};

struct PagedCopyParams {  // append: token-major rows in; read: [Hkv, total, d] out
    PagedKV kv;
    const void* k_in;
    const void* v_in;
    long long k_ts, k_hs, v_ts, v_hs;  // token and head strides of k_in, v_in
    void* k_out;
    void* v_out;
    int* err;    // device error word (check build)
    int tokens;  // of a block (set by the launcher, with the two divisions)
    FastDiv by_heads, by_tokens;
};

struct PagedAttnParams {
    PagedKV kv;
    const void* q;
    void* out;
    float* lse;
    long long q_ts, q_hs, o_ts, o_hs, l_ts, l_hs;
    int hq, g, max_q, causal, window, sinks, out_f32;
    bool out_wide;  // rows of out are 32-byte aligned
    // chunk kernel: tokens of a unit (128 / g) and of an item (one unit or two), most items of one
    // head, and where the list of items lies in the workspace (behind the partial results)
    int unit_tokens, item_tokens, max_pairs;
    long long plan_off;
    int box_rows;  // gcd(page, 128): rows of a TMA box, all on one page
    void* workspace;
    int* err;
    unsigned long long timeout_ns;
};

struct PagedMaps {  // of the pool; q for chunks
    CUtensorMap k, v, q;
};

int launch_cache_append(const PagedCopyParams& p, int sms, cudaStream_t stream);
int launch_cache_read(const PagedCopyParams& p, int sms, cudaStream_t stream);
// max_q * g <= kPagedFewRows; `blocks` at most kPagedMaxShares, the workspace 2 * kPagedMaxGroups
// PagedPartial for each
int launch_paged_decode(const PagedAttnParams& p, const PagedMaps& m, int blocks, cudaStream_t stream);
// any number of rows, g <= 128; the workspace 2 * shares PagedChunkPartial and the list of items
int launch_paged_chunk(const PagedAttnParams& p, const PagedMaps& m, int shares, cudaStream_t stream);

#ifdef __CUDACC__
// One sequence of the batch: rows [q0, q0 + T) of the token tensors, row t at position
// base + t, L positions in all.  Whatever the device arrays hold, the rows lie inside the
// tensors and the positions inside the block table.
struct PagedSeq {
    int q0, T, L, base;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedKV& kv, int b) {
    PagedSeq s;
    s.q0 = min(max(__ldg(kv.cu + b), 0), kv.total);
    s.T = min(max(__ldg(kv.cu + b + 1), s.q0), kv.total) - s.q0;
    s.L = min(max(__ldg(kv.len + b), 0), kv.max_pages * kv.page);
    s.base = s.L - s.T;
    return s;
}

// Page of position pos (0 <= pos < max_pages * page) of sequence b; -1 when the table's entry
// is no page of the pool.
__device__ __forceinline__ int paged_page(const PagedKV& kv, int b, int pos, int& row) {
    const int i = static_cast<int>(fdiv(static_cast<unsigned>(pos), kv.by_page));
    row = pos - i * kv.page;
    const int pg = __ldg(kv.table + b * kv.table_stride + i);
    return (pg >= 0 && pg < kv.n_pages) ? pg : -1;
}

// The same in two steps, for loops that load the table's entry well before they need it.
__device__ __forceinline__ int paged_entry(const PagedKV& kv, int b, int pos, int& row) {
    const int i = static_cast<int>(fdiv(static_cast<unsigned>(pos), kv.by_page));
    row = pos - i * kv.page;
    return __ldg(kv.table + b * kv.table_stride + i);
}
__device__ __forceinline__ int paged_checked(const PagedKV& kv, int entry) {
    return (entry >= 0 && entry < kv.n_pages) ? entry : -1;
}

// What the check build asks of an index: row `row` of page pg and head h; rows of one page; a row of a call's tokens.
__device__ __forceinline__ bool paged_place_ok(const PagedKV& kv, int pg, int h, int row, int rows = 1) {
    return pg >= 0 && pg < kv.n_pages && h >= 0 && h < kv.hkv && row >= 0 && row + rows <= kv.page;
}
__device__ __forceinline__ bool paged_row_ok(const PagedKV& kv, int heads, long long t, int h) {
    return t >= 0 && t < kv.total && h >= 0 && h < heads;
}

// The sequence whose rows hold row t (cu[b] <= t < cu[b + 1]), -1 if none does.  cu may be in
// shared memory.
__device__ __forceinline__ int paged_find(const int* cu, int batch, int t) {
    if (t < cu[0] || t >= cu[batch]) return -1;
    int lo = 0, hi = batch;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Weight of a partial result with running max m when the joint one is M.  All -inf: nothing was
// seen (sums are 0), or only scores that are no numbers, which have to come through.
__device__ __forceinline__ float paged_weight(float m, float M) {
    if (m == -INFINITY) return M == -INFINITY ? 1.f : 0.f;
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(m - M));
    return w;
}
__device__ __forceinline__ float paged_add_weighted(float sum, float w, float x) {
    return (w == 0.f && x == x) ? sum : fmaf(w, x, sum);
}

// Four elements of an output row, times inv, in the caller's type.
__device__ __forceinline__ void paged_store4(const PagedAttnParams& p, int tok, int head, int d, const float (&x)[4],
                                             float inv) {
    if (!RA_CHECKED(paged_row_ok(p.kv, p.hq, tok, head) && d >= 0 && d + 4 <= p.kv.d, p.err, kSitePagedOut)) return;
    const long long at = tok * p.o_ts + head * p.o_hs + d;
    if (p.out_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) =
            make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    } else {
        uint2 w;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(x[1] * inv), "f"(x[0] * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(x[3] * inv), "f"(x[2] * inv));
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = w;
    }
}

// lse of an output row: M + log2 l, in natural units; no key at all has l = 0.
__device__ __forceinline__ void paged_store_lse(const PagedAttnParams& p, int tok, int head, float M, float l) {
    if (!RA_CHECKED(paged_row_ok(p.kv, p.hq, tok, head), p.err, kSitePagedOut)) return;
    p.lse[tok * p.l_ts + head * p.l_hs] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
}
#endif

}  // namespace ra
