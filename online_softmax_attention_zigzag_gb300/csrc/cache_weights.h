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

struct WeightsParams {
    PagedKV kv;
    const void* q;
    const float* lse;
    float* w;
    long long q_ts, q_hs, l_ts, l_hs, w_ps;
    float decay;
    int hq, g, max_q, causal, window, sinks;
    FastDiv by_g;
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

int launch_cache_weights(const WeightsParams& p, int sms, cudaStream_t stream);
int launch_cache_evict(const EvictParams& p, int sms, cudaStream_t stream);

}  // namespace ra
