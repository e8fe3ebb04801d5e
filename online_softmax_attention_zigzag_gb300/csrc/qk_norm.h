// qk_norm.h -- parameter block and launchers of the norm and rotation of q and k rows
// (ringattn_qk_norm_rope, ringattn_qk_norm_rope_bwd).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace ra {

// Sites of the check build (internal.h).
enum NormCheckSite : int {
    kSiteNormRow = 61,      // a row of q, k and of what goes with them
    kSiteNormTable = 62,    // a row of the table of cosines and sines
    kSiteNormPartial = 63   // a block's sums for the weights' gradients
};

constexpr int kNormThreads = 256;
constexpr int kNormHeads = 4;          // heads of a group: rows that a thread has in flight
constexpr int kNormBlocksPerSm = 8;    // most blocks of the forward pass
// and of the backward pass, whose sums the workspace holds: two rounds of the two that an SM takes (32k tokens: 394 us, 399 with eight)
constexpr int kNormBwdBlocksPerSm = 4;
constexpr int kNormMaxSms = 256;

// Rows of q and of k: [token, head, d], strides in elements.
struct NormRows {
    void* p[2];
    long long ts[2], hs[2];
};

struct NormParams {
    NormRows x, y, g;       // rows in; forward: rows out; backward: y their gradients' source, g the gradients
    const void* w[2];       // [d] of q and of k, or null
    float* dw[2];           // backward: gradients of w, or null
    const float* cos_sin;   // [n_pos, rot]
    const int* position;    // [total]
    float* partial;         // backward: [blocks, d] of q's groups, then of k's
    int total, heads[2], groups[2], d, rot, n_pos, w_f32, interleaved, blocks_x;
    float eps, scale[2];
    int* err;
};

// Blocks along the tokens: all that are needed, at most `most` in all.
int norm_blocks(int total, int groups, int d, int most);
int launch_qk_norm_rope(NormParams p, int sms, cudaStream_t stream);
int launch_qk_norm_rope_bwd(NormParams p, bool dy_f32, bool dx_f32, int sms, cudaStream_t stream);

}  // namespace ra
