// paged_decode.cu -- attention of a few new tokens per sequence over a paged key /
// value cache, 16-bit or e4m3, and the join of the partial results of both paged
// attention kernels.
//
// A unit (paged_sched.cuh) is up to ROWS rows: as many tokens as fit with the query
// heads that share a kv head, or one token with ROWS of them.  Row (token i, head x):
//   s_j = scale q.k_j over the keys j <= its position,  O = sum_j exp(s_j) v_j / sum_j exp(s_j).
//
// Bound by HBM: every cached key and value is read once a row block against 4 d ROWS
// operations.  A CTA takes its range of keys, four warps striding over it 16 keys (e4m3:
// 2 x 16) at a time.  Both products are mma.sync m16n8k16, which keeps the operations off
// the critical path; the tcgen05 path would need the tile staged through shared memory.
// S = Q K^T has the rows as its rows; its accumulator is, as it stands, the second operand
// of O^T = V^T P^T, whose rows are head dims and whose eight columns are rows of S.  K and V
// go from global memory to registers as 16-byte loads that are operand fragments as they
// stand: the order of the contraction over d is free, so a lane's 16 bytes of a key serve
// several steps, and V's key pairs are joined by byte permutes.
//
// e4m3: a number is a half-precision number exactly, one conversion a pair, so both products
// are of that type whatever the queries' is.  bf16 queries are scaled by a power of two per row that
// brings their largest element to 2^14 .. 2^15 (exact but for elements 2^-38 below it);
// a key's scale and that power multiply its score; a value's scale multiplies its weight,
// relative to a running power of two of the warp (the largest value scale so far), so that the
// weights are at most 1 and those of 16 bits.
//
// The weights P are rounded to the 16-bit type of the product with V, after their sum is taken: its
// operands are 16-bit, and a weight is off by half a step of that type.
#include <type_traits>

#include "paged.h"
#include "paged_sched.cuh"

namespace attn {
namespace {

using namespace paged;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 16;        // keys of a warp's product
constexpr int kUnitCost = 128;   // what a unit's start and end take, in keys

__device__ __forceinline__ float ex2f(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 (8) bytes of the cache: read once, not kept in L1
__device__ __forceinline__ uint4 load16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 load8(const void *p)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// two e4m3 numbers as half-precision ones
__device__ __forceinline__ uint32_t to_half2(uint32_t e4m3x2)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(e4m3x2)));
    return h;
}

// c += a b for a 16 x 16 a (rows lane / 4 and lane / 4 + 8) and a 16 x 8 b
template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    if (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t part(const uint4 &u, int k) { return k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w; }

// Registers of a lane (K and V in flight, Q, sums) set the CTAs an SM holds.
constexpr int decode_blocks(int d, int rows) { return d == 64 ? 4 : rows == 8 ? 3 : 2; }

// A power of two that brings |x| <= most to 2^14 .. 2^15.
__device__ __forceinline__ float half_range(float most)
{
    const uint32_t e = __float_as_uint(fminf(fmaxf(most, 0x1p-100f), 0x1p+127f)) >> 23;
    return __uint_as_float((127u + 14u + 127u - e) << 23);
}

// ROWS: rows of a unit, 8 (the second half of S's rows is zero and never looked at) or 16.
template <class T, bool kEight, int D, int ROWS>
__global__ void __launch_bounds__(kThreads, decode_blocks(D, ROWS)) paged_decode_kernel(const __grid_constant__ PagedAttnArgs a)
{
    using M = typename std::conditional<kEight, __half, T>::type;  // the products' type
    constexpr int NQ = D / 8;                // 32-bit words of a query row in a lane
    constexpr int NE = D / 16;               // products of O^T
    constexpr int NR = ROWS / 8;             // rows of a lane
    constexpr int SUB = kEight ? 2 : 1;      // blocks of 16 keys a step
    constexpr int KL = kEight ? D / 64 : D / 32, VL = kEight ? 1 : D / 64;  // loads of a key, of a value
    constexpr int kStep = kWarps * kKeys * SUB;
    __shared__ float sm_m[kWarps][ROWS], sm_l[kWarps][ROWS];
    __shared__ float sm_o[kWarps][ROWS][D];
    __shared__ int64_t scratch[kWarps + 5];

    pdl_trigger();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
    const int G = a.h / a.h_kv, hb = G < ROWS ? G : ROWS, nrb = (G + ROWS - 1) / ROWS;
    const Sched<kUnitCost> sched = {a.seqs, ROWS / hb, a.h_kv * nrb, a.causal};
    bool bad = false;
    const Range range = sched.range<kThreads, kStep, kStep, 2 * kUnitCost>(blockIdx.x, gridDim.x, scratch, &bad);
    if (blockIdx.x != 0) bad = false;  // one CTA reports the lengths
    const float sc = a.scale * kLog2e;
    const PagedCache &cache = a.cache;
    const int esize = kEight ? 1 : 2;

    int4 named[2] = {unit_name(0, 0, 0, kNone), unit_name(0, 0, 0, kNone)};
    Walk<kUnitCost> w(sched, range);
    while (w.next()) {
        const int kvh = w.x / nrb, rb = w.x - kvh * nrb;
        // ---- the lane's rows: query words, last visible key, factor of the scores
        uint32_t qa[NR][NQ];
        int lim[NR];
        float fs[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = g + 8 * i, tok = r / hb, ti = w.t * sched.tokens + tok, head = kvh * G + rb * ROWS + r - tok * hb;
            const bool on = tok < sched.tokens && ti < w.u.m && rb * ROWS + r - tok * hb < G;
            lim[i] = !on ? -1 : a.causal ? w.u.len - w.u.m + ti : w.u.len - 1;
            const int64_t row = a.seqs.cu ? int64_t(w.u.first + ti) * a.q.ss : w.n * a.q.sb + ti * a.q.ss;
            const T *p = static_cast<const T *>(a.q.ptr) + row + head * a.q.sh;
            // 16-bit caches: 8 elements from 32 n + 8 q on; e4m3: 16 from 64 n + 16 q on
#pragma unroll
            for (int n = 0; n < NQ / 4; ++n) {
                const int at = kEight ? 64 * (n / 2) + 16 * q + 8 * (n % 2) : 32 * n + 8 * q;
                const uint4 v = on ? *reinterpret_cast<const uint4 *>(p + at) : make_uint4(0, 0, 0, 0);
                qa[i][4 * n] = v.x; qa[i][4 * n + 1] = v.y; qa[i][4 * n + 2] = v.z; qa[i][4 * n + 3] = v.w;
            }
            fs[i] = sc;
            if (kEight && !std::is_same<T, __half>::value) {
                float most = 0.f;
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const float2 y = unpack2<T>(qa[i][n]);
                    most = fmaxf(most, fmaxf(fabsf(y.x), fabsf(y.y)));
                }
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                const float up = half_range(most);
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const float2 y = unpack2<T>(qa[i][n]);
                    qa[i][n] = pack2<__half>(y.x * up, y.y * up);
                }
                fs[i] = sc / up;
            }
        }

        float m[NR], l[NR], vmax = 0x1p-120f;  // vmax: a power of two, at least every value scale so far
        float acc[NR][NE][4];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < NE; ++e) acc[i][e][0] = acc[i][e][1] = acc[i][e][2] = acc[i][e][3] = 0.f;
        }
        const int32_t *table = a.seqs.table + w.n * a.seqs.table_stride;
        const char *kp = static_cast<const char *>(cache.k) + int64_t(kvh) * cache.sh * esize;
        const char *vp = static_cast<const char *>(cache.v) + int64_t(kvh) * cache.sh * esize;
        const float *sp = lane < 16 ? cache.k_scale : cache.v_scale;
        auto page_of = [&](int key) -> int { return key < w.k1 ? table[key >> cache.shift] : -1; };

        int base = w.k0 + warp * kKeys * SUB;
        int id[SUB];
#pragma unroll
        for (int u = 0; u < SUB; ++u) id[u] = page_of(base + u * kKeys);
        for (; base < w.k1; base += kStep) {
            uint4 kr[SUB][2][KL], vr[SUB][4][VL];
            float size[SUB];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                const int kb = base + u * kKeys, tok = kb & ((1 << cache.shift) - 1);
                int left = w.k1 - kb < kKeys ? w.k1 - kb : kKeys;
                if (id[u] < 0 || id[u] >= cache.n_pages) {  // such a page reads as zeros
                    bad |= left > 0;
                    left = 0;
                }
                const int64_t page = id[u] * cache.sp;
                const char *kb0 = kp + (page + (tok + g) * cache.ss) * esize;
                const char *vb0 = vp + (page + (tok + 2 * q) * cache.ss) * esize;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int n = 0; n < KL; ++n)
                        kr[u][t][n] = 8 * t + g < left ? load16(kb0 + 8 * t * cache.ss * esize + 64 * n + 16 * q) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = (i & 1) + 8 * (i >> 1);
#pragma unroll
                    for (int j = 0; j < VL; ++j) {
                        const char *p = vb0 + key * cache.ss * esize;
                        vr[u][i][j] = !(2 * q + key < left) ? make_uint4(0, 0, 0, 0)
                                      : !kEight            ? load16(p + 128 * j + 16 * g)
                                      : D == 128           ? load16(p + 16 * g)
                                                           : load8(p + 8 * g);
                    }
                }
                size[u] = 0.f;
                if (kEight && lane % 16 < left)
                    size[u] = __ldg(sp + id[u] * cache.sc_sp + (kvh * cache.sc_sh + (tok + lane % 16) * cache.sc_ss));
            }
#pragma unroll
            for (int u = 0; u < SUB; ++u) id[u] = page_of(base + kStep + u * kKeys);
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                const int kb = base + u * kKeys;
                if (u > 0 && kb >= w.k1) break;
                // scores: lane (g, q) gets rows g, g + 8 and keys 2q, 2q + 1 of both tiles
                float s[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
                    for (int n = 0; n < NQ / 2; ++n) {
                        uint32_t b0, b1;
                        if (kEight) {
                            const uint32_t x = part(kr[u][t][n / 4], n % 4);
                            b0 = to_half2(x);
                            b1 = to_half2(x >> 16);
                        } else {
                            b0 = part(kr[u][t][n / 2], 2 * (n % 2));
                            b1 = part(kr[u][t][n / 2], 2 * (n % 2) + 1);
                        }
                        mma16816<M>(s[t], qa[0][2 * n], NR > 1 ? qa[NR - 1][2 * n] : 0u, qa[0][2 * n + 1],
                                    NR > 1 ? qa[NR - 1][2 * n + 1] : 0u, b0, b1);
                    }
                }
                float ks[4], vs[4];  // scales of the lane's keys
                if (kEight) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = 8 * (e >> 1) + 2 * q + (e & 1);
                        ks[e] = __shfl_sync(0xffffffffu, size[u], key);
                        vs[e] = __shfl_sync(0xffffffffu, size[u], 16 + key);
                    }
                }
                float x[NR][4], mx[NR];
                bool raise = false;
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    mx[i] = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = kb + 8 * (e >> 1) + 2 * q + (e & 1);
                        const float f = kEight ? fs[i] * ks[e] : fs[i];
                        // (behind k1 the keys are another CTA's, or hidden from all rows)
                        x[i][e] = key <= lim[i] && key < w.k1 ? s[e >> 1][2 * i + (e & 1)] * f : -INFINITY;
                        mx[i] = fmaxf(mx[i], x[i][e]);
                    }
                    mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                    mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
                    raise |= mx[i] > m[i];
                }
                float vm = 0.f;
                if (kEight) {
                    vm = fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]));
                    raise |= vm > vmax;
                }
                if (__any_sync(0xffffffffu, raise)) {
                    float fv = 1.f;
                    if (kEight) {
                        vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 1));
                        vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 2));
                        if (vm > vmax) {  // the next power of two
                            const float up = __uint_as_float((__float_as_uint(fminf(vm, 0x1p+126f)) + 0x7fffffu) & 0xff800000u);
                            fv = vmax / up;
                            vmax = up;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        const float nm = fmaxf(m[i], mx[i]);
                        const float f = nm == -INFINITY ? 1.f : ex2f(m[i] - nm);
                        m[i] = nm;
                        l[i] *= f;
                        // (the accumulator holds rows 2 q and 2 q + 1 of the eight)
                        const float f0 = __shfl_sync(0xffffffffu, f, 8 * q) * fv, f1 = __shfl_sync(0xffffffffu, f, 8 * q + 4) * fv;
#pragma unroll
                        for (int e = 0; e < NE; ++e) {
                            acc[i][e][0] *= f0;
                            acc[i][e][1] *= f1;
                            acc[i][e][2] *= f0;
                            acc[i][e][3] *= f1;
                        }
                    }
                }
                // P, rounded (see above) for the product with V; its sum is taken before
                uint32_t pa[2][2] = {{0u, 0u}, {0u, 0u}};  // [key tile][row]
                if (kEight) {
                    const float down = 1.f / vmax;
#pragma unroll
                    for (int e = 0; e < 4; ++e) vs[e] *= down;
                }
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const float ref = m[i] == -INFINITY ? 0.f : m[i];
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = ex2f(x[i][e] - ref);
                        l[i] += p[e];
                        if (kEight) p[e] *= vs[e];
                    }
                    pa[0][i] = pack2<M>(p[0], p[1]);
                    pa[1][i] = pack2<M>(p[2], p[3]);
                }
#pragma unroll
                for (int e = 0; e < NE; ++e) {  // keys 2 q, 2 q + 1 (and + 8) of two head dims
                    uint32_t a0, a1, a2, a3;
                    if (kEight) {
                        const uint32_t sel = e % 2 ? 0x7362 : 0x5140;
                        const uint32_t x0 = __byte_perm(part(vr[u][0][0], e / 2), part(vr[u][1][0], e / 2), sel);
                        const uint32_t x1 = __byte_perm(part(vr[u][2][0], e / 2), part(vr[u][3][0], e / 2), sel);
                        a0 = to_half2(x0);
                        a1 = to_half2(x0 >> 16);
                        a2 = to_half2(x1);
                        a3 = to_half2(x1 >> 16);
                    } else {
                        const uint32_t u0 = part(vr[u][0][e / 4 % VL], e % 4), u1 = part(vr[u][1][e / 4 % VL], e % 4);
                        const uint32_t u2 = part(vr[u][2][e / 4 % VL], e % 4), u3 = part(vr[u][3][e / 4 % VL], e % 4);
                        a0 = __byte_perm(u0, u1, 0x5410);
                        a1 = __byte_perm(u0, u1, 0x7632);
                        a2 = __byte_perm(u2, u3, 0x5410);
                        a3 = __byte_perm(u2, u3, 0x7632);
                    }
#pragma unroll
                    for (int i = 0; i < NR; ++i) mma16816<M>(acc[i][e], a0, a1, a2, a3, pa[0][i], pa[1][i]);
                }
            }
        }

        // ---- join the warps: lane (g, q) holds the sums of row g (+ 8 i), and dims of rows 2 q and 2 q + 1
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (q == 0) {
                sm_m[warp][g + 8 * i] = m[i];
                sm_l[warp][g + 8 * i] = l[i];
            }
            // (a lane's rows 2 q, 2 q + 1 are of the same warp: one vmax)
            const float f = kEight ? vmax : 1.f;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    const int dim = kEight ? D / 8 * g + 2 * e : 64 * (e / 4) + 8 * g + 2 * (e % 4);
                    *reinterpret_cast<float2 *>(&sm_o[warp][2 * q + c + 8 * i][dim]) =
                        make_float2(acc[i][e][c] * f, acc[i][e][2 + c] * f);
                }
        }
        __syncthreads();
        const bool whole = w.begins() && w.ends();
        const int slot = w.begins() ? 1 : 0;
        if (!whole) named[slot] = unit_name(w.n, w.x, w.t, w.ends() ? kEnds : kGoesOn);
        for (int t = threadIdx.x; t < ROWS * (D / 8); t += kThreads) {
            const int r = t / (D / 8), c = t % (D / 8) * 8;
            const int tok = r / hb, ti = w.t * sched.tokens + tok, head = kvh * G + rb * ROWS + r - tok * hb;
            if (tok >= sched.tokens || ti >= w.u.m || rb * ROWS + r - tok * hb >= G) continue;
            float mm = -INFINITY, ll = 0.f, o[8] = {};
            for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, sm_m[k][r]);
            const float ref = mm == -INFINITY ? 0.f : mm;
            for (int k = 0; k < kWarps; ++k) {
                const float f = ex2f(sm_m[k][r] - ref);
                ll += f * sm_l[k][r];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = fmaf(f, sm_o[k][r][c + e], o[e]);
            }
            if (whole) {
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                const int64_t row = a.seqs.cu ? int64_t(w.u.first + ti) * a.o.ss : w.n * a.o.sb + ti * a.o.ss;
                T *dst = static_cast<T *>(a.o.ptr) + row + head * a.o.sh + c;
                *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                                                             pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
                if (a.lse && c == 0)
                    a.lse[a.seqs.cu ? int64_t(head) * a.seqs.tokens + w.u.first + ti
                                    : (int64_t(w.n) * a.h + head) * a.seqs.s_q + ti] =
                        ll == 0.f ? INFINITY : (mm + __log2f(ll)) / kLog2e;
            } else {
                const int64_t row = (int64_t(blockIdx.x) * 2 + slot) * ROWS + r;
                if (c == 0) a.part_ml[row] = make_float2(mm, ll);
                float4 *dst = reinterpret_cast<float4 *>(a.part_o + row * D + c);
                dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                dst[1] = make_float4(o[4], o[5], o[6], o[7]);
            }
        }
        __syncthreads();
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        a.flags[blockIdx.x] = bad ? ATTN_DEV_INDEX_RANGE : 0u;
        a.rec[2 * blockIdx.x] = named[0];
        a.rec[2 * blockIdx.x + 1] = named[1];
    }
}

// Outputs of the units that several shares hold, a block for every share that holds a unit's first piece and every 16
// rows: the pieces' maxima, then their sums in order of the shares, D / 8 lanes a row.  The first block gathers the
// call's status.
template <class T, int D>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const __grid_constant__ PagedAttnArgs a, const PagedShape shape)
{
    constexpr int LPR = D / 8, NG = kThreads / LPR;
    const int c0 = blockIdx.x, shares = shape.shares, rows = shape.rows;
    pdl_wait();
    if (c0 == 0 && blockIdx.y == 0) {
        uint32_t flags = 0;
        for (int k = threadIdx.x; k < shares; k += kThreads) flags |= a.flags[k];
        const int range = __syncthreads_or(flags & ATTN_DEV_INDEX_RANGE), timeout = __syncthreads_or(flags & ATTN_DEV_TIMEOUT);
        if (threadIdx.x == 0) *a.status = (range ? ATTN_DEV_INDEX_RANGE : 0u) | (timeout ? ATTN_DEV_TIMEOUT : 0u);
    }
    const int4 name = a.rec[2 * c0 + 1];
    if (name.w == kNone) return;
    // the shares that hold the rest: up to the one whose first piece ends the unit
    int end = c0 + 1;
    while (end < shares && a.rec[2 * end].w != kEnds) ++end;
    const int G = a.h / a.h_kv, kvh = name.y / shape.row_blocks, block = name.y - kvh * shape.row_blocks;
    bool none = false;
    int first, m;
    a.seqs.rows(name.x, &first, &m, &none);
    const int g = threadIdx.x / LPR, c = threadIdx.x % LPR * 8, group_rows = rows / shape.groups;
    for (int r = blockIdx.y * 16 + g; r < int(blockIdx.y) * 16 + 16 && r < rows; r += NG) {
        const int grp = r / group_rows, in = r - grp * group_rows, tok = in / shape.heads;
        const int x = block * shape.heads + in - tok * shape.heads, head = kvh * G + x;
        const int ti = (name.z * shape.groups + grp) * shape.tokens + tok;
        if (tok >= shape.tokens || ti >= m || x >= G) continue;
        float mm = -INFINITY;
        for (int k = c0; k <= end && k < shares; ++k)
            if (k == c0 || a.rec[2 * k].w != kNone) mm = fmaxf(mm, a.part_ml[(int64_t(k) * 2 + (k == c0)) * rows + r].x);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f, o[8] = {};
        for (int k = c0; k <= end && k < shares; ++k) {
            if (k != c0 && a.rec[2 * k].w == kNone) continue;
            const int64_t row = (int64_t(k) * 2 + (k == c0)) * rows + r;
            const float2 x = a.part_ml[row];
            const float4 *src = reinterpret_cast<const float4 *>(a.part_o + row * D + c);
            const float4 u = src[0], v = src[1];
            const float f = ex2f(x.x - ref);
            ll = fmaf(f, x.y, ll);
            o[0] = fmaf(f, u.x, o[0]); o[1] = fmaf(f, u.y, o[1]); o[2] = fmaf(f, u.z, o[2]); o[3] = fmaf(f, u.w, o[3]);
            o[4] = fmaf(f, v.x, o[4]); o[5] = fmaf(f, v.y, o[5]); o[6] = fmaf(f, v.z, o[6]); o[7] = fmaf(f, v.w, o[7]);
        }
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        const int64_t row = a.seqs.cu ? int64_t(first + ti) * a.o.ss : name.x * a.o.sb + ti * a.o.ss;
        T *dst = static_cast<T *>(a.o.ptr) + row + head * a.o.sh + c;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                                                     pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
        if (a.lse && c == 0)
            a.lse[a.seqs.cu ? int64_t(head) * a.seqs.tokens + first + ti : (int64_t(name.x) * a.h + head) * a.seqs.s_q + ti] =
                ll == 0.f ? INFINITY : (mm + __log2f(ll)) / kLog2e;
    }
}

template <class T, bool kEight, int D, int ROWS> cudaError_t run(const PagedAttnArgs &a, const PagedShape &p, cudaStream_t s)
{
    return launch_kernel(paged_decode_kernel<T, kEight, D, ROWS>, dim3(unsigned(p.shares)), dim3(kThreads), 0, s, false, a);
}

template <class T, bool kEight> cudaError_t pick(const PagedAttnArgs &a, const PagedShape &p, cudaStream_t s)
{
    if (a.d == 64) return p.rows == 16 ? run<T, kEight, 64, 16>(a, p, s) : run<T, kEight, 64, 8>(a, p, s);
    return p.rows == 16 ? run<T, kEight, 128, 16>(a, p, s) : run<T, kEight, 128, 8>(a, p, s);
}

}  // namespace

PagedShape paged_decode_shape(int64_t h, int64_t h_kv, int64_t d, int64_t s_q)
{
    const int group = int(h / h_kv);
    PagedShape p;
    p.chunk = false;
    p.rows = group * (s_q < 16 ? s_q : 16) > 8 ? 16 : 8;
    p.shares = kPagedCtas * decode_blocks(int(d), p.rows);
    p.groups = 1;
    p.heads = group < p.rows ? group : p.rows;
    p.tokens = p.rows / p.heads;
    p.row_blocks = (group + p.rows - 1) / p.rows;
    return p;
}

cudaError_t launch_paged_decode(const PagedAttnArgs &a, const PagedShape &p, cudaStream_t s)
{
    if (a.cache.type == ATTN_E4M3) return a.dtype == ATTN_F16 ? pick<__half, true>(a, p, s) : pick<__nv_bfloat16, true>(a, p, s);
    return a.dtype == ATTN_F16 ? pick<__half, false>(a, p, s) : pick<__nv_bfloat16, false>(a, p, s);
}

cudaError_t launch_paged_join(const PagedAttnArgs &a, const PagedShape &p, cudaStream_t s)
{
    auto k = a.d == 64 ? (a.dtype == ATTN_F16 ? paged_join_kernel<__half, 64> : paged_join_kernel<__nv_bfloat16, 64>)
                       : (a.dtype == ATTN_F16 ? paged_join_kernel<__half, 128> : paged_join_kernel<__nv_bfloat16, 128>);
    return launch_kernel(k, dim3(unsigned(p.shares), unsigned((p.rows + 15) / 16)), dim3(kThreads), 0, s, true, a, p);
}

}  // namespace attn
