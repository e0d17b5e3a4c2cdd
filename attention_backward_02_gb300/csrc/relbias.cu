// relbias.cu -- the table of a learned relative position bias expanded by distance,
// ahead of the attention kernels.
//
// The bias of a score depends on delta = (key position - query position) alone,
// and every delta <= lo, and every delta >= hi, has one bucket.  Expanded over
// lo .. hi a head's table is a line of floats, and the bias of a tile of scores is
// a window of it: element (key row r, query column c) reads window[r - c + const].
// For the backward under a causal mask the entries of keys after their query are
// -inf, which is the mask.
#include <cmath>

#include "relbias.h"

namespace attn {
namespace {

// grid (blocks over the deltas, h).  A few microseconds of latency; at the sizes in use (a few hundred
// deltas a head) it moves kilobytes.
__global__ void __launch_bounds__(256) rel_expand_kernel(const RelArgs a)
{
    pdl_trigger();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0u;
    const int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x, delta = t + a.b.lo - kRelPad;
    // keys after their query are masked like a bucket, of their own where they share one with their query's key
    auto bucket = [&](int64_t x) { return a.causal && !a.b.bidirectional && x > 0 ? kRelMaxBuckets : a.b.bucket(x); };
    const int n = bucket(delta);
    if (t < a.stride)
        for (int64_t h = blockIdx.y; h < a.h; h += gridDim.y)
            a.rel[h * a.stride + t] = a.causal && delta > 0 ? -INFINITY : rel_table_value(a.b, int64_t(n) * a.h + h);
    if (a.code && blockIdx.y == 0) {
        __shared__ int16_t near[256 + 32];  // buckets of delta - 1 .. delta + 31 of the block's deltas
        near[threadIdx.x + 1] = int16_t(n);
        if (threadIdx.x < 31) near[threadIdx.x + 257] = int16_t(bucket(delta + 256));
        if (threadIdx.x == 0) near[0] = int16_t(bucket(delta - 1));
        __syncthreads();
        uint32_t rem = 0;
        while (rem < 31 && near[threadIdx.x + rem + 2] == n) ++rem;
        if (t < a.stride) a.code[t] = uint32_t(n) | rem << 8 | uint32_t(near[threadIdx.x] != n) << 16;
    }
    if (a.part) {
        const int64_t n2 = a.part_rows * a.h * 8 * a.b.buckets / 2;
        const int64_t nthreads = int64_t(gridDim.x) * gridDim.y * 256;
        float2 *p = reinterpret_cast<float2 *>(a.part);
        for (int64_t k = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x; k < n2; k += nthreads)
            p[k] = make_float2(0.f, 0.f);
    }
}

}  // namespace

cudaError_t launch_rel_expand(const RelArgs &a, cudaStream_t s)
{
    const unsigned ny = unsigned(a.h < 65535 ? a.h : 65535);
    return launch_kernel(rel_expand_kernel, dim3(unsigned((a.stride + 255) / 256), ny), dim3(256), 0, s, false, a);
}

}  // namespace attn
