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
// Bound by HBM: a row is read once and written once; what has to be kept low for that is
// the instructions a row takes (with 8 elements a lane 116 for two rows, 75 % of the issue
// slots).  A lane takes two pieces of a row, 16 bytes of the 16-bit side each (8 elements;
// 8 bytes of the 8-bit side), d / 16 lanes a row.  A block takes a run of rows in the order
// token, keys and values, head, up to four a lane group; the write's are all loaded before
// the places in the cache are looked up (cumulative counts, length, page id: three
// dependent loads), the read's behind it.  131104 tokens of 8 heads of 128 read from e4m3:
// 124 us, 0.96 of the measured copy rate; 17408 tokens written: 25 us, 0.64 (the start and
// end of the run).
#include <cstring>
#include <type_traits>

#include "paged.h"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kMost = 4;           // rows of a lane group in a block
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

// The largest |x| of a lane's eight elements, NaN left out (the two-element maximum does that); kFinite: infinities too.
template <class T, bool kFinite> __device__ __forceinline__ float most_of(const uint4 &x)
{
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const uint32_t u[4] = {x.x & 0x7fff7fffu, x.y & 0x7fff7fffu, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu};
    float most = 0.f;
    if (kFinite) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 y = unpack2<T>(u[e]);
            most = fmaxf(most, fmaxf(y.x < INFINITY ? y.x : 0.f, y.y < INFINITY ? y.y : 0.f));  // (false for NaN too)
        }
        return most;
    }
    T2 v[4];
    memcpy(v, u, sizeof v);
    const T2 m = __hmax2(__hmax2(v[0], v[1]), __hmax2(v[2], v[3]));
    uint32_t w;
    memcpy(&w, &m, sizeof w);
    const float2 y = unpack2<T>(w);
    return fmaxf(fmaxf(y.x, y.y), 0.f);
}

// T: the dense rows' type; kEight: e4m3 cache (else T); a block takes `most` rows, at most kMost a lane group.  A lane
// group's rows are kThreads / (D / 16) apart, which is step_t tokens and step_r rows of one.
template <class T, bool kEight, int D, bool kWrite>
__global__ void __launch_bounds__(kThreads) paged_copy_kernel(const __grid_constant__ PagedCopyArgs a, int most, int step_t, int step_r)
{
    constexpr int LPR = D / 16, GROUPS = kThreads / LPR, HALF = D / 2;
    constexpr int kTokens = GROUPS * kMost / 2 + 1;            // that a block's rows may belong to
    constexpr int kNone = -1, kNotOurs = -2;                   // page: no place; no sequence's row
    __shared__ int64_t sm_dense[2][kTokens], sm_place[kTokens], sm_scale[kTokens];  // element offsets of head 0
    __shared__ int sm_page[kTokens];
    const int group = threadIdx.x / LPR, l = threadIdx.x % LPR;
    const int per = 2 * a.h_kv, all = a.seqs.tokens * per;     // rows of a token, and of the call
    const int row0 = blockIdx.x * most, rows = all - row0 < most ? all - row0 : most;
    const int token0 = row0 / per, here = rows > 0 ? (row0 + rows - 1) / per - token0 + 1 : 0;
    if (int(threadIdx.x) < here) {
        const int row = token0 + threadIdx.x;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const View &v = e ? a.v : a.k;
            sm_dense[e][threadIdx.x] = a.seqs.cu ? row * v.ss : (row / a.seqs.s_q) * v.sb + (row % a.seqs.s_q) * v.ss;
        }
    }
    __syncthreads();

    // this lane group's rows: token, and row of the token (keys, then values; heads)
    struct At {
        int t, r;
    };
    At at0;
    at0.t = (row0 + group) / per;
    at0.r = row0 + group - at0.t * per;
    at0.t -= token0;
    auto next = [&](At &at) {
        at.t += step_t;
        at.r += step_r;
        if (at.r >= per) {
            at.r -= per;
            ++at.t;
        }
    };
    auto dense = [&](const At &at) -> T * {
        const bool side = at.r >= a.h_kv;
        const View &v = side ? a.v : a.k;
        return static_cast<T *>(v.ptr) + sm_dense[side][at.t] + (side ? at.r - a.h_kv : at.r) * v.sh + l * 8;
    };
    const int count = rows > group ? (rows - group + GROUPS - 1) / GROUPS : 0;

    uint4 x[kMost][2];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (kWrite) {
        At at = at0;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            x[i][0] = x[i][1] = zero;
            if (i < count) {
                const T *src = dense(at);
                x[i][0] = __ldcs(reinterpret_cast<const uint4 *>(src));
                x[i][1] = __ldcs(reinterpret_cast<const uint4 *>(src + HALF));
            }
            next(at);
        }
    }
    if (int(threadIdx.x) < here) {
        const int row = token0 + threadIdx.x;
        int page = kNone, tok = 0;
        if (!place_of(a.seqs, a.cache, row, &page, &tok)) page = kNone;
        if (!kWrite && a.seqs.cu && (row >= a.seqs.cu[a.seqs.b] || row < a.seqs.cu[0])) page = kNotOurs;
        sm_page[threadIdx.x] = page;
        sm_place[threadIdx.x] = page * a.cache.sp + tok * a.cache.ss;
        if (kEight) sm_scale[threadIdx.x] = page * a.cache.sc_sp + tok * a.cache.sc_ss;
    }
    __syncthreads();

    struct Place {
        int64_t at, scale;
        bool side;
    };
    auto place = [&](const At &at) -> Place {
        Place p;
        p.side = at.r >= a.h_kv;
        const int head = p.side ? at.r - a.h_kv : at.r;
        p.at = sm_place[at.t] + head * a.cache.sh + l * 8;
        p.scale = kEight ? sm_scale[at.t] + head * a.cache.sc_sh : 0;
        return p;
    };

    At at = at0;
    if (kWrite) {
#pragma unroll
        for (int i = 0; i < kMost; ++i, next(at)) {
            if (i * GROUPS >= rows) break;  // (the same for the whole block: the shuffles below need all lanes)
            const bool on = i < count && sm_page[i < count ? at.t : 0] >= 0;
            if (!kEight) {
                if (on) {
                    const Place p = place(at);
                    T *dst = static_cast<T *>(p.side ? a.cache.v : a.cache.k) + p.at;
                    *reinterpret_cast<uint4 *>(dst) = x[i][0];
                    *reinterpret_cast<uint4 *>(dst + HALF) = x[i][1];
                }
                continue;
            }
            float top = fmaxf(most_of<T, false>(x[i][0]), most_of<T, false>(x[i][1]));
            if (__any_sync(0xffffffffu, top == INFINITY)) top = fmaxf(most_of<T, true>(x[i][0]), most_of<T, true>(x[i][1]));
            top = fmaxf(top, kFloor);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float up = kTop / top;
            uint32_t c[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 y = unpack2<T>(e ? x[i][h].z : x[i][h].x), z = unpack2<T>(e ? x[i][h].w : x[i][h].y);
                    c[h][e] = to_e4m3x2(y.x * up, y.y * up) | uint32_t(to_e4m3x2(z.x * up, z.y * up)) << 16;
                }
            if (on) {
                const Place p = place(at);
                uint8_t *dst = static_cast<uint8_t *>(p.side ? a.cache.v : a.cache.k) + p.at;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0][0], c[0][1]);
                *reinterpret_cast<uint2 *>(dst + HALF) = make_uint2(c[1][0], c[1][1]);
                if (l == 0) (p.side ? a.cache.v_scale : a.cache.k_scale)[p.scale] = top / kTop;
            }
        }
    } else {
        uint2 c[kMost][2];
        float size[kMost];
#pragma unroll
        for (int i = 0; i < kMost; ++i, next(at)) {
            const bool on = i < count && sm_page[i < count ? at.t : 0] >= 0;
            x[i][0] = x[i][1] = zero;
            c[i][0] = c[i][1] = make_uint2(0, 0);
            size[i] = 0.f;
            if (!on) continue;
            const Place p = place(at);
            const void *pool = p.side ? a.cache.v : a.cache.k;
            if (kEight) {
                const uint8_t *src = static_cast<const uint8_t *>(pool) + p.at;
                c[i][0] = __ldcs(reinterpret_cast<const uint2 *>(src));
                c[i][1] = __ldcs(reinterpret_cast<const uint2 *>(src + HALF));
                size[i] = __ldg((p.side ? a.cache.v_scale : a.cache.k_scale) + p.scale);
            } else {
                const T *src = static_cast<const T *>(pool) + p.at;
                x[i][0] = __ldcs(reinterpret_cast<const uint4 *>(src));
                x[i][1] = __ldcs(reinterpret_cast<const uint4 *>(src + HALF));
            }
        }
        at = at0;
#pragma unroll
        for (int i = 0; i < kMost; ++i, next(at)) {
            if (i >= count) break;
            if (sm_page[at.t] == kNotOurs) continue;
            T *dst = dense(at);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (kEight) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y = from_e4m3x2(uint16_t((e < 2 ? c[i][h].x : c[i][h].y) >> (16 * (e & 1))));
                        w[e] = pack2<T>(y.x * size[i], y.y * size[i]);
                    }
                    x[i][h] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                __stcs(reinterpret_cast<uint4 *>(dst + h * HALF), x[i][h]);
            }
        }
    }
    if (blockIdx.x == 0) check_call(a.seqs, a.cache, a.status);  // the call's only status writer
}

template <class T, bool kEight, int D> cudaError_t run(const PagedCopyArgs &a, bool write, cudaStream_t s)
{
    // as many rows a lane group as leave four blocks an SM
    constexpr int GROUPS = kThreads / (D / 16);
    const int all = a.seqs.tokens * 2 * a.h_kv, share = (all + 4 * kPagedCtas - 1) / (4 * kPagedCtas);
    int most = (share + GROUPS - 1) / GROUPS;
    most = (most < 1 ? 1 : most > kMost ? kMost : most) * GROUPS;
    const int blocks = all > 0 ? (all + most - 1) / most : 1;
    return launch_kernel(write ? paged_copy_kernel<T, kEight, D, true> : paged_copy_kernel<T, kEight, D, false>,
                         dim3(unsigned(blocks)), dim3(kThreads), 0, s, false, a, most, GROUPS / (2 * a.h_kv), GROUPS % (2 * a.h_kv));
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
