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
    int shares;               // backward: CTAs that share the query heads of a (key tile, kv head); more than one:
    float *kv_part;           // [dK, dV][shares][h_kv][t_kv][d] their sums, which the dQ finalize adds up
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
// warp w sums every 8th share, the warps' sums are added in order.  A warp takes the rows one after the other, four
// loads in flight, which shows where the rows are many and the heads few: the finalize takes 81 us where it takes 18
// without a bias at 16 sequences of 4096 keys, 5 heads of 64 (529 rows), and 110 where 48 at 256 packed sequences of 50
// to 350, 12 heads of 64 (667 rows).
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
// dK (scaled) and dV = the sums of the shares, in order: 8 elements a thread, tokens' heads side by side.
template <class T>
__device__ __forceinline__ void rel_sum_shares(const RelArgs &a, const DenseArgs &d, int64_t s_kv, int block, int blocks)
{
    const uint32_t per = uint32_t(d.d / 8), hk = uint32_t(d.h_kv), n = uint32_t(2 * d.t_kv) * hk * per;
    const int64_t share = d.h_kv * d.t_kv * d.d;
    for (uint32_t k = uint32_t(block) * 256 + threadIdx.x; k < n; k += uint32_t(blocks) * 256) {
        const uint32_t c = k % per, x = k / per, head = x % hk, y = x / hk;
        const bool isv = y >= uint32_t(d.t_kv);
        const uint32_t t = isv ? y - uint32_t(d.t_kv) : y;
        const float *p = a.kv_part + (isv ? a.shares * share : 0) + (head * d.t_kv + t) * d.d + c * 8;
        float v[8] = {};
        for (int s = 0; s < a.shares; ++s) {
            const float4 u = *reinterpret_cast<const float4 *>(p + s * share), w = *reinterpret_cast<const float4 *>(p + s * share + 4);
            v[0] += u.x; v[1] += u.y; v[2] += u.z; v[3] += u.w;
            v[4] += w.x; v[5] += w.y; v[6] += w.z; v[7] += w.w;
        }
        const float m = isv ? 1.f : d.scale;
        const View &o = isv ? d.dV : d.dK;
        const uint32_t b = d.packed ? 0 : t / uint32_t(s_kv);
        T *dst = static_cast<T *>(o.ptr) + b * o.sb + head * o.sh + int64_t(d.packed ? t : t - b * uint32_t(s_kv)) * o.ss + c * 8;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<T>(v[0] * m, v[1] * m), pack2<T>(v[2] * m, v[3] * m),
                                                     pack2<T>(v[4] * m, v[5] * m), pack2<T>(v[6] * m, v[7] * m));
    }
}
inline int64_t rel_dtable_blocks(const RelArgs &a) { return a.h * ((a.b.buckets + 31) / 32); }

// Expands the table (and zeroes the status word and the gradient shares, where there are any); dependents
// may start at once and wait for it.
cudaError_t launch_rel_expand(const RelArgs &a, cudaStream_t s);

}  // namespace attn
