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

// Query heads a block handles: the rows of its products.
inline int64_t decode_rows(int64_t h, int64_t h_kv) { return h / h_kv > 8 ? 16 : 8; }

// Keys of a block.  Two blocks fit an SM at d = 128, four at d = 64; a block's start and end take about the time of
// 128 keys.  Of the chunk counts that fill one, two, .. sixteen waves of blocks when the cache is full, the one with
// the least waves x (keys + 128); a multiple of the 64 keys of a block's step.  (At 32 sequences of 8192 keys, 8 kv
// heads of 128: chunks of 1024 take 188 us, of 2048 196, of 1216, this choice, 183.)  A constant 152 SMs: the
// workspace size must not depend on a CUDA call.
inline int64_t decode_chunk(int64_t b, int64_t h, int64_t h_kv, int64_t cap, int64_t d)
{
    const int64_t rows = decode_rows(h, h_kv), units = b * h_kv * ((h / h_kv + rows - 1) / rows);
    const int64_t slots = 152 * (d == 64 ? 4 : 2);
    int64_t best = cap, best_cost = -1;
    for (int64_t waves = 1; waves <= 16; ++waves) {
        int64_t n = waves * slots / units;
        if (n < 1) n = 1;
        int64_t chunk = ((cap + n - 1) / n + 63) / 64 * 64;
        if (chunk < 64) chunk = 64;
        n = (cap + chunk - 1) / chunk;
        const int64_t cost = (units * n + slots - 1) / slots * (chunk + 128);
        if (best_cost < 0 || cost < best_cost) {
            best = chunk;
            best_cost = cost;
        }
    }
    return best;
}
inline int64_t decode_chunks(int64_t cap, int64_t chunk) { return cap > chunk ? (cap + chunk - 1) / chunk : 1; }

cudaError_t launch_relbias_decode(const DecodeArgs &a, cudaStream_t s);

}  // namespace attn
