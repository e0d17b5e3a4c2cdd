// relbias.h -- the learned relative position bias by buckets: the bucket of a
// distance, and the argument bundle of the kernels that add the bias to the
// scores or sum its gradient.
#pragma once

#include "plan.h"

namespace attn {

constexpr int kRelMaxBuckets = 128;
constexpr int64_t kRelMaxDistance = 65536;
constexpr int kRelCodes = kRelMaxBuckets + 4;  // bucket codes: kRelMaxBuckets is that of causally masked deltas
constexpr float kRelMasked = -1e30f;  // a table entry at or below this masks its bucket

// The caller's bias.  A key delta positions after its query has distance |delta| (both directions) or
// max(-delta, 0) (one direction: the keys after the query share bucket 0).  Of the n buckets of a direction
// the first e are exact; the rest start at the distances thr[0] < thr[1] < ...
struct RelBias {
    const void *table;        // [buckets][h]
    int table_type;           // ATTN_F16, ATTN_BF16 or ATTN_F32
    int buckets, n, e;        // n: buckets of one direction (buckets / 2 or buckets), e = n / 2
    int bidirectional;
    int nthr;                 // n - e - 1
    int lo, hi;               // every delta <= lo is in one bucket, and every delta >= hi
    int32_t thr[kRelMaxBuckets / 2];

    __host__ __device__ int bucket(int64_t delta) const
    {
        const int64_t x = delta < 0 ? -delta : (bidirectional ? delta : 0);
        const int base = bidirectional && delta > 0 ? n : 0;
        if (x < e) return base + int(x);
        int k = 0, m = nthr;  // borders at or below x
        while (k < m) {
            const int mid = (k + m) / 2;
            if (thr[mid] <= x) k = mid + 1;
            else m = mid;
        }
        return base + e + k;
    }
};

// Expanded form, made once per call in the workspace: the bias by delta, in log2 units (-inf where the
// bucket is masked), for each head; the entry of delta is at delta - (lo - kRelPad).  The pad on both sides
// lets the window of any tile that is not wholly in one of the end buckets be read without a clamp.
constexpr int kRelPad = 272;

struct RelArgs {
    RelBias b;
    int64_t h;
    float *rel;               // [h][stride]
    int causal;               // backward under a causal mask: entries of delta > 0 are -inf
    uint32_t *code;           // [stride] bucket | min(31, deltas after this one in its bucket) << 8 | first of it << 16
    int64_t stride;           // hi - lo + 1 + 2 kRelPad, rounded up to 4
    float *part;              // backward: [part_rows][h][8 warps][buckets] shares of the table's gradient
    int64_t part_rows;        // one per key tile: row of tile jt of sequence b = kv_start(b) / 128 + b + jt
    float *dtable;            // [buckets][h]
    uint32_t *status;
};

inline int64_t rel_stride(const RelBias &b) { return (int64_t(b.hi) - b.lo + 1 + 2 * kRelPad + 3) / 4 * 4; }

__device__ __forceinline__ float rel_table_value(const RelBias &b, int64_t at)
{
    float v;
    if (b.table_type == ATTN_F16) v = to_f32(static_cast<const __half *>(b.table)[at]);
    else if (b.table_type == ATTN_BF16) v = to_f32(static_cast<const __nv_bfloat16 *>(b.table)[at]);
    else v = static_cast<const float *>(b.table)[at];
    return v <= kRelMasked ? -INFINITY : v * kLog2e;
}

// dtable[n][head] = the sum of the shares of 32 buckets of one head, in a fixed order: a block of 256 threads;
// warp w sums every 8th share, the warps' sums are added in order.
__device__ __forceinline__ void rel_dtable_block(const RelArgs &a, int unit)
{
    __shared__ float red[8][32];
    const int nb = (a.b.buckets + 31) / 32, w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t head = unit / nb;
    const int n = unit % nb * 32 + lane;
    float v = 0.f;
    if (n < a.b.buckets) {
        const float *p = a.part + (head * 8 + w) * a.b.buckets + n;
#pragma unroll 4
        for (int64_t row = 0; row < a.part_rows; ++row) v += p[row * a.h * 8 * a.b.buckets];
    }
    red[w][lane] = v;
    __syncthreads();
    if (w == 0 && n < a.b.buckets) {
        for (int k = 1; k < 8; ++k) v += red[k][lane];
        a.dtable[int64_t(n) * a.h + head] = v;
    }
}
inline int64_t rel_dtable_blocks(const RelArgs &a) { return a.h * ((a.b.buckets + 31) / 32); }

// Expands the table (and zeroes the status word and the gradient shares, where there are any); dependents
// may start at once and wait for it.
cudaError_t launch_rel_expand(const RelArgs &a, cudaStream_t s);

}  // namespace attn
