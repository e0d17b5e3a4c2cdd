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

// Blocks an SM holds: set by the registers of a lane's K, V, Q and sums.
constexpr int decode_blocks(int64_t d, int64_t rows) { return d == 64 ? 4 : rows == 8 ? 3 : 2; }

// Keys of a block.  A block's start and end take about the time of 128 keys.  Of the chunk counts that fill one, two,
// .. sixteen waves of blocks when the cache is full, the one with the least time of two caches: a full one, whole
// waves x (keys + 128), and one half full with sequences of all lengths, whose blocks spread evenly but for half a block
// at the end; a multiple of the 64 keys of a block's step.  (us, lengths of 1 to 8192 / all 8192, 32 / 8 heads of
// 128; the choice in brackets: 32 sequences, chunks of 640 91 / 176, [1216 93 / 165], 1664 97 / 165, 2048 106 / 186; 8
// sequences, [640 26 / 47], 1216 34 / 43, 2048 44 / 51.)  A constant 152 SMs: the workspace size must not depend on a
// CUDA call.
inline int64_t decode_chunk(int64_t b, int64_t h, int64_t h_kv, int64_t cap, int64_t d)
{
    const int64_t rows = decode_rows(h, h_kv), units = b * h_kv * ((h / h_kv + rows - 1) / rows);
    const int64_t slots = 152 * decode_blocks(d, rows);
    int64_t best = cap, best_cost = -1;
    for (int64_t waves = 1; waves <= 16; ++waves) {
        int64_t n = waves * slots / units;
        if (n < 1) n = 1;
        int64_t chunk = ((cap + n - 1) / n + 63) / 64 * 64;
        if (chunk < 64) chunk = 64;
        n = (cap + chunk - 1) / chunk;
        const int64_t cost = (units * n + slots - 1) / slots * (chunk + 128) +
                             (units * n + slots) * (chunk + 128) / (2 * slots);
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
