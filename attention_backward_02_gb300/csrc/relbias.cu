// relbias.cu -- the small kernels around attention with a learned relative
// position bias: the table expanded by distance before the attention kernel, and
// the sum of the table's gradient behind the backward one.
//
// The bias of a score depends on delta = (key position - query position) alone,
// and every delta <= lo, and every delta >= hi, has one bucket.  Expanded over
// lo .. hi a head's table is a line of floats, and the bias of a tile of scores is
// a window of it: element (key row r, query column c) reads window[r - c + const].
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
    const int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (t < a.stride) {
        const int64_t delta = t + a.b.lo - kRelPad;
        const int n = a.b.bucket(delta);
        for (int64_t h = blockIdx.y; h < a.h; h += gridDim.y)
            a.rel[h * a.stride + t] = rel_table_value(a.b, int64_t(n) * a.h + h);
        if (a.code && blockIdx.y == 0) {
            uint32_t rem = 0;
            while (rem < 31 && a.b.bucket(delta + rem + 1) == n) ++rem;
            const uint32_t first = a.b.bucket(delta - 1) != n;
            a.code[t] = uint32_t(n) | rem << 8 | first << 16;
        }
    }
    if (a.part) {
        const int64_t n2 = a.part_rows * a.h * 8 * a.b.buckets / 2;
        const int64_t nthreads = int64_t(gridDim.x) * gridDim.y * 256;
        float2 *p = reinterpret_cast<float2 *>(a.part);
        for (int64_t k = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x; k < n2; k += nthreads)
            p[k] = make_float2(0.f, 0.f);
    }
}

// grid (h, blocks of 32 buckets): warp w sums every 32nd share, the warps' sums are added in a fixed order.
__global__ void __launch_bounds__(1024) rel_dtable_kernel(const RelArgs a)
{
    __shared__ float red[32][33];
    pdl_wait();
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n = blockIdx.y * 32 + lane;
    float v = 0.f;
    if (n < a.b.buckets)
        for (int64_t s = w; s < a.part_rows * 8; s += 32)
            v += a.part[(((s >> 3) * a.h + blockIdx.x) * 8 + (s & 7)) * a.b.buckets + n];
    red[w][lane] = v;
    __syncthreads();
    v = red[lane][w];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int nw = blockIdx.y * 32 + w;
    if (lane == 0 && nw < a.b.buckets) a.dtable[int64_t(nw) * a.h + blockIdx.x] = v;
}

}  // namespace

cudaError_t launch_rel_expand(const RelArgs &a, cudaStream_t s)
{
    const unsigned ny = unsigned(a.h < 65535 ? a.h : 65535);
    return launch_kernel(rel_expand_kernel, dim3(unsigned((a.stride + 255) / 256), ny), dim3(256), 0, s, false, a);
}

cudaError_t launch_rel_dtable(const RelArgs &a, cudaStream_t s)
{
    return launch_kernel(rel_dtable_kernel, dim3(unsigned(a.h), unsigned((a.b.buckets + 31) / 32)), dim3(1024), 0, s, true, a);
}

}  // namespace attn
