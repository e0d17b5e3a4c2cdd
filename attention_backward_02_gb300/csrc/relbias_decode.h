// relbias_decode.h -- argument bundle of the single-token attention kernels.
#pragma once

#include "relbias.h"

namespace attn {

// Workspace (256-byte aligned):  status uint32[64];  with more than one chunk a sequence:
//   part_ml f32 [b][h][chunks][2]   maximum (log2 units) and sum of a chunk
//   part_o  f32 [b][h][chunks][d]   its unnormalised output
struct DecodeArgs {
    int dtype;
    int64_t b, h, h_kv, d, cap;   // cap: keys of the cache a sequence may have
    int64_t chunk;                // keys of a block
    float scale;
    View q, k, v, o;
    const int32_t *lens;          // [b] keys cached, the new token's among them (NULL: cap)
    RelBias bias;
    uint32_t *status;
    float2 *part_ml;
    float *part_o;
};

// Keys of a block: enough blocks to fill the GPU several times over when the cache is full (so that a
// mix of lengths still does), at least one step of every warp, at most 1024.
inline int64_t decode_chunk(int64_t b, int64_t h_kv, int64_t cap)
{
    const int64_t want = 152 * 8;
    int64_t c = 64;
    while (c < 1024 && b * h_kv * ((cap + c - 1) / c) > want) c *= 2;
    return c;
}
inline int64_t decode_chunks(int64_t cap, int64_t chunk) { return cap > chunk ? (cap + chunk - 1) / chunk : 1; }

cudaError_t launch_relbias_decode(const DecodeArgs &a, cudaStream_t s);

}  // namespace attn
