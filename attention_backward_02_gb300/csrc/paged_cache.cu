// paged_cache.cu -- new tokens' keys and values into a paged cache, and rows of the
// cache back into dense tensors.
//
// A row x (a token's d elements of one head) goes into the cache as it is, or as
// e4m3 numbers with one scale:
//   a = max(max |x|, 2^-110),  code = e4m3(x (448 / a)),  scale = a / 448,  value = code scale,
// the maximum over the finite elements; an infinity becomes the largest code of its sign
// and a NaN stays one.  (2^-110: 448 / a stays finite; smaller rows keep their elements
// relative to it.)  Both factors are rounded fp32 quotients, so a row's codes do not
// depend on how it is shared out.
//
// Bound by HBM: a row is read once and written once.  A lane takes 16 bytes of the 16-bit side (8 elements; 8 of
// the 8-bit side), d / 8 lanes a row.  A block takes a run of rows in the order token, keys and values, head, up to
// eight a lane group; the write's are all loaded before the places in the cache are looked up (cumulative
// counts, length, page id: three dependent loads), the read's behind it.
#include <type_traits>

#include "paged.h"

#include <cuda_fp8.h>

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kMost = 8;           // rows of a lane group in a block
constexpr float kTop = 448.f;
constexpr float kFloor = 0x1p-110f;

__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint16_t x)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(x));
    return unpack2<__half>(h);
}

// Place of new token `row` of the call: sequence, then page id and token in it.  false: it has none.
__device__ bool place_of(const PagedSeqs &s, const PagedCache &c, int row, int *page, int *tok)
{
    bool bad = false;
    int n, first, m;
    if (s.cu) {  // the last sequence that begins at or before the row
        int lo = 0, hi = s.b - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (s.cu[mid] <= row) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
    } else {
        n = row / s.s_q;
    }
    s.rows(n, &first, &m, &bad);
    if (row < first || row >= first + m) return false;
    const int pos = s.len(n, &bad) - m + (row - first);
    if (pos < 0) return false;
    const int id = s.table[n * s.table_stride + (pos >> c.shift)];
    if (id < 0 || id >= c.n_pages) return false;
    *page = id;
    *tok = pos & ((1 << c.shift) - 1);
    return true;
}

// The call's status, by its first block: counts and lengths in range, and the page of every new token.
__device__ void check_call(const PagedSeqs &s, const PagedCache &c, uint32_t *status)
{
    bool bad = false;
    for (int n = threadIdx.x / 32; n < s.b; n += kThreads / 32) {
        int first, m;
        s.rows(n, &first, &m, &bad);
        const int len = s.len(n, &bad), from = len - m > 0 ? len - m : 0;
        if (m > 0 && len > 0)
            for (int p = (from >> c.shift) + threadIdx.x % 32; p <= (len - 1) >> c.shift; p += 32) {
                const int id = s.table[n * s.table_stride + p];
                bad |= id < 0 || id >= c.n_pages;
            }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *status = bad ? ATTN_DEV_INDEX_RANGE : 0u;
}

// T: the dense rows' type; kEight: e4m3 cache (else T); a block takes `most` rows, at most kMost a lane group.
template <class T, bool kEight, int D, bool kWrite>
__global__ void __launch_bounds__(kThreads) paged_copy_kernel(const __grid_constant__ PagedCopyArgs a, int most)
{
    constexpr int LPR = D / 8, GROUPS = kThreads / LPR;
    constexpr int kTokens = GROUPS * kMost / 2 + 1;            // that a block's rows may belong to
    __shared__ int sm_page[kTokens], sm_tok[kTokens];          // page -1: no place; -2: no sequence's row
    const int group = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int per = 2 * a.h_kv, all = a.seqs.tokens * per;     // rows of a token, and of the call
    const int row0 = blockIdx.x * most, rows = all - row0 < most ? all - row0 : most;
    const int token0 = row0 / per, here = rows > 0 ? (row0 + rows - 1) / per - token0 + 1 : 0;

    auto dense = [&](int t, int side, int head) -> T * {
        const View &v = side ? a.v : a.k;
        const int row = token0 + t;
        int64_t at = int64_t(head) * v.sh + l * 8;
        if (a.seqs.cu) at += int64_t(row) * v.ss;
        else at += int64_t(row / a.seqs.s_q) * v.sb + int64_t(row % a.seqs.s_q) * v.ss;
        return static_cast<T *>(v.ptr) + at;
    };
    auto split = [&](int r, int *t, int *side, int *head) {
        const int th = (row0 + r) / a.h_kv;
        *head = row0 + r - th * a.h_kv;
        *t = (th >> 1) - token0;
        *side = th & 1;
    };

    uint4 x[kMost];
    if (kWrite) {
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int r = group + i * GROUPS;
            int t, side, head;
            split(r, &t, &side, &head);
            x[i] = r < rows ? __ldcs(reinterpret_cast<const uint4 *>(dense(t, side, head))) : make_uint4(0, 0, 0, 0);
        }
    }
    if (int(threadIdx.x) < here) {
        const int row = token0 + threadIdx.x;
        int page = -1, tok = 0;
        if (!place_of(a.seqs, a.cache, row, &page, &tok)) page = -1;
        if (!kWrite && a.seqs.cu && (row >= a.seqs.cu[a.seqs.b] || row < a.seqs.cu[0])) page = -2;
        sm_page[threadIdx.x] = page;
        sm_tok[threadIdx.x] = tok;
    }
    __syncthreads();

    auto scale_at = [&](int t, int side, int head) -> float * {
        return (side ? a.cache.v_scale : a.cache.k_scale) + sm_page[t] * a.cache.sc_sp +
               (head * a.cache.sc_sh + sm_tok[t] * a.cache.sc_ss);
    };
    auto cached = [&](int t, int side, int head) -> int64_t {
        return sm_page[t] * a.cache.sp + (head * a.cache.sh + sm_tok[t] * a.cache.ss + l * 8);
    };

    if (kWrite) {
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int r = group + i * GROUPS;
            if (i * GROUPS >= rows) break;  // (the same for the whole block: the shuffles below need all lanes)
            int t, side, head;
            split(r, &t, &side, &head);
            const bool on = r < rows && sm_page[r < rows ? t : 0] >= 0;
            void *pool = side ? a.cache.v : a.cache.k;
            if (!kEight) {
                if (on) *reinterpret_cast<uint4 *>(static_cast<T *>(pool) + cached(t, side, head)) = x[i];
                continue;
            }
            float2 y[4] = {unpack2<T>(x[i].x), unpack2<T>(x[i].y), unpack2<T>(x[i].z), unpack2<T>(x[i].w)};
            float most = kFloor;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float u = fabsf(y[e].x), w = fabsf(y[e].y);
                most = fmaxf(most, u < INFINITY ? u : 0.f);  // (false for NaN too)
                most = fmaxf(most, w < INFINITY ? w : 0.f);
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            const float up = kTop / most;
            uint16_t c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = to_e4m3x2(y[e].x * up, y[e].y * up);
            if (on) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(pool) + cached(t, side, head)) =
                    make_uint2(c[0] | uint32_t(c[1]) << 16, c[2] | uint32_t(c[3]) << 16);
                if (l == 0) *scale_at(t, side, head) = most / kTop;
            }
        }
    } else {
        uint2 c[kMost];
        float size[kMost];
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int r = group + i * GROUPS;
            int t, side, head;
            split(r, &t, &side, &head);
            const bool on = r < rows && sm_page[r < rows ? t : 0] >= 0;
            const void *pool = side ? a.cache.v : a.cache.k;
            if (kEight) {
                c[i] = on ? __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(pool) + cached(t, side, head)))
                          : make_uint2(0, 0);
                size[i] = on ? *scale_at(t, side, head) : 0.f;
            } else {
                x[i] = on ? __ldcs(reinterpret_cast<const uint4 *>(static_cast<const T *>(pool) + cached(t, side, head)))
                          : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int r = group + i * GROUPS;
            if (r >= rows) break;
            int t, side, head;
            split(r, &t, &side, &head);
            if (sm_page[t] == -2) continue;
            if (kEight) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 y = from_e4m3x2(uint16_t((e < 2 ? c[i].x : c[i].y) >> (16 * (e & 1))));
                    w[e] = pack2<T>(y.x * size[i], y.y * size[i]);
                }
                x[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4 *>(dense(t, side, head)) = x[i];
        }
    }
    if (blockIdx.x == 0) check_call(a.seqs, a.cache, a.status);  // the call's only status writer
}

template <class T, bool kEight, int D> cudaError_t run(const PagedCopyArgs &a, bool write, cudaStream_t s)
{
    // as many rows a lane group as leave four blocks an SM
    constexpr int GROUPS = kThreads / (D / 8);
    const int all = a.seqs.tokens * 2 * a.h_kv, share = (all + 4 * kPagedCtas - 1) / (4 * kPagedCtas);
    int most = (share + GROUPS - 1) / GROUPS;
    most = (most < 1 ? 1 : most > kMost ? kMost : most) * GROUPS;
    const int blocks = all > 0 ? (all + most - 1) / most : 1;
    return launch_kernel(write ? paged_copy_kernel<T, kEight, D, true> : paged_copy_kernel<T, kEight, D, false>,
                         dim3(unsigned(blocks)), dim3(kThreads), 0, s, false, a, most);
}

template <class T> cudaError_t pick(const PagedCopyArgs &a, bool write, cudaStream_t s)
{
    const bool eight = a.cache.type == ATTN_E4M3;
    if (a.d == 64) return eight ? run<T, true, 64>(a, write, s) : run<T, false, 64>(a, write, s);
    return eight ? run<T, true, 128>(a, write, s) : run<T, false, 128>(a, write, s);
}

}  // namespace

cudaError_t launch_paged_copy(const PagedCopyArgs &a, bool write, cudaStream_t s)
{
    return a.dtype == ATTN_F16 ? pick<__half>(a, write, s) : pick<__nv_bfloat16>(a, write, s);
}

}  // namespace attn
