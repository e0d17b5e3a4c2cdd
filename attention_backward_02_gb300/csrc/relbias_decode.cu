// relbias_decode.cu -- attention of one new token per sequence over a key / value
// cache, with the learned relative position bias.
//
// For query head x of sequence b, whose L = lens[b] cached keys end with the new
// token's own (delta of key j = j - (L - 1)):
//   s_j = scale q.k_j + table[bucket(delta)][x],  O = sum_j exp(s_j) v_j / sum_j exp(s_j).
//
// Bound by HBM: every cached key and value is read once (4 d bytes a key and kv
// head) against 4 d G operations for the G query heads that share it.  A block
// takes one (sequence, kv head) and a chunk of its keys, four warps striding over
// it 16 keys at a time; chunks past a sequence's length end at once, so sequences
// of any mix of lengths load the GPU by their keys.  Both products are mma.sync
// m16n8k16, which keeps the operations off the critical path at every G: the tensor
// cores idle either way, and the tcgen05 path would need the tile staged through
// shared memory.  S = Q K^T has the query heads of a group as its rows (8 of 16 used
// up to G = 8; more than 16: several blocks); its accumulator is, as it stands, the
// second operand of O^T = V^T P^T, whose rows are head dims and whose eight columns
// are heads, so O takes D / 4 registers a lane for eight heads (with O = P V, half
// of whose rows were empty, a lane held 212 registers, two blocks an SM, and 32
// sequences took 104 us where three blocks take 93).  K and V go from global memory
// to registers as 16-byte loads that are operand fragments as they stand: the order
// of the contraction over d is free, so a lane's 16 bytes of a key serve two steps,
// and V's key pairs are joined by byte permutes, head dims taken in the order that
// makes a lane's 16 bytes four row pairs.
// Each warp keeps a running maximum and sum (log2 units); the warps of a block join
// through shared memory, the chunks of a sequence through fp32 partial results in
// the workspace and a second kernel that adds them in order.
// The weights P are rounded to the 16-bit type for the product with V, after their sum
// is taken: the operands of that product are 16-bit, and a weight is off by half a step of V's own
// type, as in the training forward (against the 64-bit form 0.00073 of the largest output for
// bf16, where fp32 weights give 0.00065: O's own rounding is most of both).
// 32 sequences of 1 to 8192 keys, 32 / 8 heads of 128: 93 us for 537 MB, 0.86 of the
// measured copy rate, and 0.97 with all of 8192 (K and V through a ring of asynchronous
// copies in shared memory: 112 against 107 as loads at the time; kv heads as the
// grid's fastest index: 111; K a step ahead in registers: no gain); one sequence of 1000
// keys, 12 heads of 64: 7 us, two launches' latency.
#include <cmath>
#include <type_traits>

#include "relbias_decode.h"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 16;  // keys of a warp's step

__device__ __forceinline__ float ex2f(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 bytes of the cache: read once, not kept in L1
__device__ __forceinline__ uint4 load_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
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

// Length of sequence b, brought into [0, cap].
__device__ __forceinline__ int64_t cached_len(const DecodeArgs &a, int64_t b)
{
    if (!a.lens) return a.cap;
    const int64_t n = a.lens[b];
    return n < 0 ? 0 : (n > a.cap ? a.cap : n);
}

// grid (chunks, kv heads x row blocks of ROWS query heads, sequences).  ROWS: query heads of a group handled, 8
// (the second half of S's rows is zero and never looked at) or 16.
template <class T, int D, int ROWS>
__global__ void __launch_bounds__(32 * kWarps, decode_blocks(D, ROWS)) relbias_decode_kernel(const __grid_constant__ DecodeArgs a)
{
    constexpr int NP = D / 32;   // 64-byte pieces of a key
    constexpr int NJ = D / 64;   // 128-byte pieces of a value
    constexpr int NR = ROWS / 8; // rows of a lane
    __shared__ float sm_m[kWarps][ROWS], sm_l[kWarps][ROWS];
    __shared__ float sm_o[kWarps][ROWS][D];

    pdl_trigger();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && warp == 0) {  // the call's only status writer
        bool bad = false;
        if (a.lens)
            for (int64_t n = lane; n < a.b; n += 32) bad |= a.lens[n] < 0 || a.lens[n] > a.cap;
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) *a.status = bad ? ATTN_DEV_INDEX_RANGE : 0u;
    }
    const int64_t b = blockIdx.z, G = a.h / a.h_kv;
    const int64_t nrb = (G + ROWS - 1) / ROWS, kvh = blockIdx.y / nrb, rb = blockIdx.y - kvh * nrb;
    const int64_t h0 = kvh * G + rb * ROWS;                 // first query head of the block
    const int rows = int(G - rb * ROWS < ROWS ? G - rb * ROWS : ROWS);
    const int64_t len = cached_len(a, b);
    const int64_t k0 = int64_t(blockIdx.x) * a.chunk, k1 = k0 + a.chunk < len ? k0 + a.chunk : len;
    const bool direct = gridDim.x == 1;                     // no second kernel behind
    if (k0 >= len && !(direct && len == 0)) return;

    // the query rows as the first operand, and each row's bias of the end bucket
    uint4 qa[NR][NP];
    float past[NR];
    int64_t head[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const bool on = g + 8 * i < rows;
        head[i] = h0 + (on ? g + 8 * i : 0);
        const T *p = static_cast<const T *>(a.q.ptr) + b * a.q.sb + head[i] * a.q.sh;
#pragma unroll
        for (int n = 0; n < NP; ++n)
            qa[i][n] = on ? *reinterpret_cast<const uint4 *>(p + 32 * n + 8 * q) : make_uint4(0, 0, 0, 0);
        past[i] = rel_table_value(a.bias, int64_t(a.bias.n - 1) * a.h + head[i]);
    }
    const T *kp = static_cast<const T *>(a.k.ptr) + b * a.k.sb + kvh * a.k.sh;
    const T *vp = static_cast<const T *>(a.v.ptr) + b * a.v.sb + kvh * a.v.sh;
    const float sc = a.scale * kLog2e;

    float m[NR], l[NR];
    float acc[NR][NJ][4][4];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e][0] = acc[i][j][e][1] = acc[i][j][e][2] = acc[i][j][e][3] = 0.f;

    for (int64_t base = k0 + warp * kKeys; base < k1; base += kWarps * kKeys) {
        const int left = int(k1 - base < kKeys ? k1 - base : kKeys);
        uint4 kr[2][NP], vr[4][NJ];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int n = 0; n < NP; ++n)
                kr[t][n] = 8 * t + g < left ? load_stream(kp + (base + 8 * t + g) * a.k.ss + 32 * n + 8 * q) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = 2 * q + (i & 1) + 8 * (i >> 1);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                vr[i][j] = key < left ? load_stream(vp + (base + key) * a.v.ss + 64 * j + 8 * g) : make_uint4(0, 0, 0, 0);
        }
        // scores: lane (g, q) gets rows g, g + 8 and keys 2q, 2q + 1 of both tiles
        float s[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                const uint4 x = qa[0][n], y = NR > 1 ? qa[NR - 1][n] : make_uint4(0, 0, 0, 0);
                mma16816<T>(s[t], x.x, y.x, x.y, y.y, kr[t][n].x, kr[t][n].y);
                mma16816<T>(s[t], x.z, y.z, x.w, y.w, kr[t][n].z, kr[t][n].w);
            }
        }
        const bool far = base + kKeys - 1 - (len - 1) <= a.bias.lo;
        float x[NR][4], mx[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            mx[i] = -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = 8 * (e >> 1) + 2 * q + (e & 1);
                float bias = past[i];
                if (!far) bias = rel_table_value(a.bias, int64_t(a.bias.bucket(base + key - (len - 1))) * a.h + head[i]);
                x[i][e] = key < left ? fmaf(s[e >> 1][2 * i + (e & 1)], sc, bias) : -INFINITY;
                mx[i] = fmaxf(mx[i], x[i][e]);
            }
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        }
        bool raise = false;
#pragma unroll
        for (int i = 0; i < NR; ++i) raise |= mx[i] > m[i];
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const float nm = fmaxf(m[i], mx[i]);
                const float f = nm == -INFINITY ? 1.f : ex2f(m[i] - nm);
                m[i] = nm;
                l[i] *= f;
                // (the accumulator holds heads 2 q and 2 q + 1 of the eight)
                const float f0 = __shfl_sync(0xffffffffu, f, 8 * q), f1 = __shfl_sync(0xffffffffu, f, 8 * q + 4);
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[i][j][e][0] *= f0;
                        acc[i][j][e][1] *= f1;
                        acc[i][j][e][2] *= f0;
                        acc[i][j][e][3] *= f1;
                    }
            }
        }
        // P, rounded to the 16-bit type (see above) for the product with V; its sum is taken before
        uint32_t pa[2][2] = {{0u, 0u}, {0u, 0u}};  // [key tile][row]
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float ref = m[i] == -INFINITY ? 0.f : m[i];
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[e] = ex2f(x[i][e] - ref);
                l[i] += p[e];
            }
            pa[0][i] = pack2<T>(p[0], p[1]);
            pa[1][i] = pack2<T>(p[2], p[3]);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // columns 64 j + 8 g + 2 e (and + 1), keys 2 q, 2 q + 1 (and + 8)
                const uint32_t u0 = part(vr[0][j], e), u1 = part(vr[1][j], e), u2 = part(vr[2][j], e), u3 = part(vr[3][j], e);
                const uint32_t a0 = __byte_perm(u0, u1, 0x5410), a1 = __byte_perm(u0, u1, 0x7632);
                const uint32_t a2 = __byte_perm(u2, u3, 0x5410), a3 = __byte_perm(u2, u3, 0x7632);
#pragma unroll
                for (int i = 0; i < NR; ++i) mma16816<T>(acc[i][j][e], a0, a1, a2, a3, pa[0][i], pa[1][i]);
            }
    }

    // join the warps: lane (g, q) holds the sums of head g (+ 8 i), and columns 64 j + 8 g + .. of heads 2 q and 2 q + 1
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if (q == 0) {
            sm_m[warp][g + 8 * i] = m[i];
            sm_l[warp][g + 8 * i] = l[i];
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<float2 *>(&sm_o[warp][2 * q + c + 8 * i][64 * j + 8 * g + 2 * e]) =
                        make_float2(acc[i][j][e][c], acc[i][j][e][2 + c]);
    }
    __syncthreads();
    for (int t = threadIdx.x; t < rows * (D / 8); t += 32 * kWarps) {
        const int r = t / (D / 8), c = t % (D / 8) * 8;
        float mm = -INFINITY, ll = 0.f, o[8] = {};
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][r]);
        const float ref = mm == -INFINITY ? 0.f : mm;
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2f(sm_m[w][r] - ref);
            ll += f * sm_l[w][r];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf(f, sm_o[w][r][c + e], o[e]);
        }
        if (direct) {
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            T *dst = static_cast<T *>(a.o.ptr) + b * a.o.sb + (h0 + r) * a.o.sh + c;
            *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                                                         pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
        } else {
            const int64_t row = (b * a.h + h0 + r) * gridDim.x + blockIdx.x;
            if (c == 0) a.part_ml[row] = make_float2(mm, ll);
            float4 *dst = reinterpret_cast<float4 *>(a.part_o + row * D + c);
            dst[0] = make_float4(o[0], o[1], o[2], o[3]);
            dst[1] = make_float4(o[4], o[5], o[6], o[7]);
        }
    }
}

// O of a (sequence, head) from its chunks' results: a block a row.  The threads take the chunks' maxima side by
// side; then groups of D / 8 lanes (8 columns each) every NG-th chunk, and the groups' sums are added in order.
// (A chunk after the other cost 35 us at 128 chunks.)
template <class T, int D>
__global__ void __launch_bounds__(128) relbias_decode_join_kernel(const __grid_constant__ DecodeArgs a, int chunks)
{
    constexpr int LPR = D / 8, NG = 128 / LPR;
    __shared__ float sm_m[4], sm_l[NG], sm_o[NG][D];
    const int64_t row = blockIdx.x, b = row / a.h, hq = row - b * a.h;
    const int t = threadIdx.x, g = t / LPR, c = t % LPR * 8;
    pdl_wait();
    const int n = int((cached_len(a, b) + a.chunk - 1) / a.chunk);
    const float2 *ml = a.part_ml + row * chunks;
    float m = -INFINITY;
    for (int k = t; k < n; k += 128) m = fmaxf(m, ml[k].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (t % 32 == 0) sm_m[t / 32] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[8] = {};
#pragma unroll 4
    for (int k = g; k < n; k += NG) {
        const float2 x = ml[k];
        const float4 *src = reinterpret_cast<const float4 *>(a.part_o + (row * chunks + k) * D + c);
        const float4 u = src[0], v = src[1];
        const float f = ex2f(x.x - ref);
        l = fmaf(f, x.y, l);
        o[0] = fmaf(f, u.x, o[0]); o[1] = fmaf(f, u.y, o[1]); o[2] = fmaf(f, u.z, o[2]); o[3] = fmaf(f, u.w, o[3]);
        o[4] = fmaf(f, v.x, o[4]); o[5] = fmaf(f, v.y, o[5]); o[6] = fmaf(f, v.z, o[6]); o[7] = fmaf(f, v.w, o[7]);
    }
    if (c == 0) sm_l[g] = l;
#pragma unroll
    for (int e = 0; e < 8; ++e) sm_o[g][c + e] = o[e];
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int k = 1; k < NG; ++k) {
        l = k == 1 ? sm_l[0] + sm_l[1] : l + sm_l[k];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += sm_o[k][c + e];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T *dst = static_cast<T *>(a.o.ptr) + b * a.o.sb + hq * a.o.sh + c;
    *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                                                 pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
}

template <class T, int D, int ROWS> cudaError_t run(const DecodeArgs &a, cudaStream_t s)
{
    const int64_t chunks = decode_chunks(a.cap, a.chunk), G = a.h / a.h_kv;
    const dim3 grid(unsigned(chunks), unsigned(a.h_kv * ((G + ROWS - 1) / ROWS)), unsigned(a.b));
    cudaError_t e = launch_kernel(relbias_decode_kernel<T, D, ROWS>, grid, dim3(32 * kWarps), 0, s, false, a);
    if (e != cudaSuccess || chunks == 1) return e;
    return launch_kernel(relbias_decode_join_kernel<T, D>, dim3(unsigned(a.b * a.h)), dim3(128), 0, s, true, a, int(chunks));
}

template <class T> cudaError_t pick(const DecodeArgs &a, cudaStream_t s)
{
    const bool wide = decode_rows(a.h, a.h_kv) == 16;
    if (a.d == 64) return wide ? run<T, 64, 16>(a, s) : run<T, 64, 8>(a, s);
    return wide ? run<T, 128, 16>(a, s) : run<T, 128, 8>(a, s);
}

}  // namespace

cudaError_t launch_relbias_decode(const DecodeArgs &a, cudaStream_t s)
{
    return a.dtype == ATTN_F16 ? pick<__half>(a, s) : pick<__nv_bfloat16>(a, s);
}

}  // namespace attn
