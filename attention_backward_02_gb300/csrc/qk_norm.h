// qk_norm.h -- argument bundle of the query / key norm and rotation kernels.
#pragma once

#include "plan.h"

namespace attn {

// One side: the query heads or the key heads.
struct QkSide {
    View x, dy, y;          // input; gradient of the output (backward); output, or gradient of the input
    const void *w;          // [d] weight (NULL: ones)
    float *dw;              // [d] weight gradient (backward; NULL: not wanted)
    float *part;            // [blocks][d] each block's share of it
    int64_t h;
    int blocks;             // blocks of the main kernel that work on this side
};

// Workspace (256-byte aligned):  status uint32[64];  backward: part f32 [kQkBlocks + 2][d]
struct QkNormArgs {
    int dtype, weight_fp32, interleaved;
    int64_t b, s, d, rot, max_pos;
    float eps;
    const float *cos, *sin;
    const int32_t *pos;
    uint32_t *status;
    QkSide side[2];
    int warp_smem;          // bytes of a warp's shared memory (set by the launcher)
};

// Most blocks the kernels are launched with on both sides together; each leaves one row of weight
// gradient shares in the workspace.
constexpr int kQkBlocks = 1216;

cudaError_t launch_qk_norm(const QkNormArgs &a, bool backward, cudaStream_t s);

}  // namespace attn
