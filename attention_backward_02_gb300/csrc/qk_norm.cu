// qk_norm.cu -- RMS norm of every query and key head with the rotary position
// embedding in the same pass, and the gradient of both.
//
// Forward, for the d elements x of one (token, head) row:
//   r = 1 / sqrt(mean(x^2) + eps),  z = w x r,  y = Rot(position) z.
// Backward, with xh = x r and dz = Rot(-position) dy (Rot is orthogonal):
//   dw = sum over rows of dz xh,  g = dz w,  dx = r (g - xh mean(g xh)).
// r is computed again from x: the row is read anyway, so nothing is saved.
//
// Bound by HBM: forward 4 bytes an element, backward 6, against about 10 and 25
// operations.  Eight lanes hold a row in chunks of 8 elements (16 bytes), chunk
// l + 8 k on lane l, so a warp reads four rows at once, each 128 bytes
// contiguous per load, and a row's sums take three shuffles.  The partner of a
// rotated element lies rotary_dim / 2 away, on another lane for most sizes: z
// (backward: dy) goes through shared memory once, which serves every
// rotary_dim that is a multiple of 16.  A work item is four heads of a token; each
// warp takes a run of items.  The rows of the next items, and the cos and sin rows of
// their tokens, come through a ring of asynchronous copies in shared memory that is
// the warp's own: HBM needs about 40 KB of loads in flight an SM, more than the
// registers hold (one item ahead in registers: 104 us where this takes 74 at
// 20442 tokens x 40 heads x 128, 0.84 of the measured copy rate; the backward there
// 107 us, 0.87).  A lane reads back its own 16 bytes.  Blocks work
// on one side (query or key heads) each, so weights and weight-gradient sums stay in
// registers.  The other end of the range is few heads: items of four heads are padded, and
// one block's look over all positions (the status word) outlasts the rest; 163536
// tokens of 5 + 5 heads of 64 take 182 us, 0.34 of the copy rate, and the backward 253, 0.37.
#include <cstdint>

#include "qk_norm.h"
#include "tc_util.cuh"

namespace attn {
namespace {
using tc::add2;
using tc::fma2;
using tc::mul2;

constexpr int kWarps = 4;
constexpr int kItemHeads = 4;  // rows a warp works on side by side

// 8 elements as pairs
template <class T> __device__ __forceinline__ void unpack8(const uint4 &u, float2 (&f)[4])
{
    f[0] = unpack2<T>(u.x);
    f[1] = unpack2<T>(u.y);
    f[2] = unpack2<T>(u.z);
    f[3] = unpack2<T>(u.w);
}

template <class T> __device__ __forceinline__ uint4 pack8(const float2 (&f)[4])
{
    return make_uint4(pack2<T>(f[0].x, f[0].y), pack2<T>(f[1].x, f[1].y), pack2<T>(f[2].x, f[2].y), pack2<T>(f[3].x, f[3].y));
}

__device__ __forceinline__ void load8(const float *p, float2 (&f)[4])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y);
    f[3] = make_float2(b.z, b.w);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// sum over the 8 lanes of a row
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// How the pairs of a rotation lie: none; (i, i + rotary_dim / 2) through shared memory; the same with
// rotary_dim = 128, where both halves are chunks of one lane; (2i, 2i + 1).
enum { kNoRope = 0, kHalves = 1, kHalves128 = 2, kPairs = 3 };

// Blocks an SM holds: set so that the registers of a lane (its row, weights, cos and sin, backward the
// weight-gradient sums) fit without spills.
template <int NC, bool BWD> constexpr int kBlocksPerSm = BWD ? (NC == 1 ? 4 : NC == 2 ? 3 : 2) : (NC == 1 ? 6 : NC == 2 ? 4 : 3);
// Items a warp has in flight.  More is worse where the copies bound it (forward, 20442 tokens x 40 heads x 128: 2
// items 73 us, 3 75, 4 82; 8192 tokens: 31.8, 30.6, 30.8), and makes no difference at d = 64 and 192.
template <int NC, bool BWD> constexpr int kDepth = NC == 2 ? 3 : 4;

// Shared memory of a warp: rows [depth][x, dy][chunk][lane] of 16 bytes; cos and sin rows [depth + 1][rot]
// floats; the exchange of the turn [4 rows][D] floats.
template <int NC, int ROPE, bool BWD> int warp_smem(int64_t rot)
{
    return kDepth<NC, BWD> * (BWD ? 2 : 1) * NC * 512 + (ROPE != kNoRope ? (kDepth<NC, BWD> + 1) * int(rot) * 4 : 0) +
           (ROPE == kHalves ? kItemHeads * NC * 64 * 4 : 0);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on)  // zeros where off
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// NC = d / 64 chunks a lane.
template <class T, int NC, int ROPE, bool BWD>
__global__ void __launch_bounds__(32 * kWarps, kBlocksPerSm<NC, BWD>) qk_norm_kernel(const __grid_constant__ QkNormArgs a)
{
    constexpr int D = NC * 64, DEPTH = kDepth<NC, BWD>, ROWS16 = (BWD ? 2 : 1) * NC;
    extern __shared__ uint4 ring_mem[];
    if (blockIdx.x == 0) {  // the status word: one block looks over the positions beside the others' work
        bool bad = false;
        if (ROPE != kNoRope && a.pos)
            for (int64_t t = threadIdx.x; t < a.b * a.s; t += 32 * kWarps) bad |= a.pos[t] < 0 || a.pos[t] >= a.max_pos;
        if (ROPE != kNoRope && !a.pos) bad = a.s > a.max_pos;
        bad = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.status = bad ? ATTN_DEV_INDEX_RANGE : 0u;
        return;
    }
    const int bid = int(blockIdx.x) - 1;
    const int sd = bid >= a.side[0].blocks;
    const QkSide &s = a.side[sd];
    const int cta = bid - (sd ? a.side[0].blocks : 0);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, grp = lane / 8, l = lane % 8;
    uint8_t *const ring = reinterpret_cast<uint8_t *>(ring_mem) + warp * a.warp_smem;
    float *const angles = reinterpret_cast<float *>(ring + DEPTH * ROWS16 * 512);
    float *const mine = angles + (DEPTH + 1) * a.rot + grp * D;  // kHalves: this row's exchange

    // this warp's items, a run of them: 4 heads of a token each, heads fastest
    const uint32_t nhb = uint32_t((s.h + kItemHeads - 1) / kItemHeads);
    const uint64_t items = uint64_t(a.b * a.s) * nhb, warps = uint64_t(s.blocks) * kWarps, w_id = uint64_t(cta) * kWarps + warp;
    const uint32_t first = uint32_t(items * w_id / warps), end = uint32_t(items * (w_id + 1) / warps);
    const int shift = ROPE == kHalves128 ? 8 : int(a.rot) / 16;  // chunks between the halves of a rotated pair

    // ---- the item whose copies go out next: its token t = (b, i), head block, this lane's place in its row;
    // positions of 32 tokens, one a lane; tokens begun, and which of them (mod 32) have a valid position
    uint32_t t = first / nhb, hb = first - t * nhb;
    uint32_t b = t / uint32_t(a.s), i = t - b * uint32_t(a.s);
    const T *xp = nullptr, *dp = nullptr;
    uint32_t pos_base = t, begun = 0, valid_bits = 0;
    int32_t pos_lane = 0;
    auto load_positions = [&]() {
        pos_base = t;
        const int64_t u = int64_t(t) + lane;
        if (u < a.b * a.s) pos_lane = a.pos ? a.pos[u] : int32_t(u % a.s);
    };
    auto issue = [&](uint32_t n) {  // copies of item n, the next one in order
        if (n < end) {
            if (n == first || hb == 0) {  // a new token
                const int64_t h = int64_t(hb) * kItemHeads + grp;
                xp = static_cast<const T *>(s.x.ptr) + b * s.x.sb + h * s.x.sh + i * s.x.ss + l * 8;
                if (BWD) dp = static_cast<const T *>(s.dy.ptr) + b * s.dy.sb + h * s.dy.sh + i * s.dy.ss + l * 8;
                if (ROPE != kNoRope) {
                    if (n == first || t - pos_base == 32) load_positions();
                    const int32_t p = __shfl_sync(0xffffffffu, pos_lane, int(t - pos_base));
                    const bool ok = p >= 0 && p < a.max_pos;
                    valid_bits = (valid_bits & ~(1u << (begun & 31))) | uint32_t(ok) << (begun & 31);
                    const float *cr = a.cos + int64_t(ok ? p : 0) * (a.rot / 2), *sr = a.sin + int64_t(ok ? p : 0) * (a.rot / 2);
                    const uint32_t dst = tc::smem_u32(angles + (begun % (DEPTH + 1)) * a.rot);
                    const int half = int(a.rot) / 8;  // 16-byte pieces of a cos or sin row
                    for (int k = lane; k < 2 * half; k += 32) copy16(dst + k * 16, k < half ? cr + 4 * k : sr + 4 * (k - half), ok);
                }
                ++begun;
            }
            const bool on = int64_t(hb) * kItemHeads + grp < s.h;
            const uint32_t dst = tc::smem_u32(ring + (n - first) % DEPTH * ROWS16 * 512 + lane * 16);
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                copy16(dst + k * 512, on ? xp + 64 * k : s.x.ptr, on);
                if (BWD) copy16(dst + (NC + k) * 512, on ? dp + 64 * k : s.dy.ptr, on);
            }
            xp += kItemHeads * s.x.sh;
            if (BWD) dp += kItemHeads * s.dy.sh;
            if (++hb == nhb) {
                hb = 0;
                ++t;
                if (++i == uint32_t(a.s)) {
                    i = 0;
                    ++b;
                }
            }
        }
        copy_commit();  // one group an item, empty ones behind the last
    };
    // ---- the item being worked on: its head block, this lane's place in its output row, and its token's number
    uint32_t c_hb = hb, c_b = b, c_i = i, c_token = 0;
    T *yp = nullptr;
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) issue(first + k);

    float2 w[NC][4], dw[NC][4];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dw[k][e] = both(0.f);
            w[k][e] = both(1.f);
        }
        if (s.w) {
            const int c = (l + 8 * k) * 8;
            if (a.weight_fp32) load8(static_cast<const float *>(s.w) + c, w[k]);
            else unpack8<T>(*reinterpret_cast<const uint4 *>(static_cast<const T *>(s.w) + c), w[k]);
        }
    }
    float2 cs[NC][4], sn[NC][4];
    bool valid = true;
    auto load_angles = [&]() {  // cos and sin of this lane's elements (sin with the sign of the turn)
        valid = valid_bits >> (c_token & 31) & 1u;
        const float *cr = angles + (c_token % (DEPTH + 1)) * a.rot, *sr = cr + a.rot / 2;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = l + 8 * k;
            if (c < 2 * shift) {
                if (ROPE == kPairs) {
                    const float4 c4 = *reinterpret_cast<const float4 *>(cr + 4 * c), s4 = *reinterpret_cast<const float4 *>(sr + 4 * c);
                    const float cv[4] = {c4.x, c4.y, c4.z, c4.w}, sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        cs[k][e] = both(cv[e]);
                        sn[k][e] = BWD ? make_float2(sv[e], -sv[e]) : make_float2(-sv[e], sv[e]);
                    }
                } else {
                    const bool lo = c < shift;
                    load8(cr + 8 * (lo ? c : c - shift), cs[k]);
                    load8(sr + 8 * (lo ? c : c - shift), sn[k]);
                    const float2 sign = both(lo != BWD ? -1.f : 1.f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sn[k][e] = mul2(sn[k][e], sign);
                }
            }
        }
    };
    // a row turned by the token's angle, in place
    auto turn = [&](float2 (&z)[NC][4]) {
        if (ROPE == kNoRope) return;
        if (ROPE == kHalves) {
            __syncwarp();  // the previous row's partners have been read
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float4 *dst = reinterpret_cast<float4 *>(mine + (l + 8 * k) * 8);
                dst[0] = make_float4(z[k][0].x, z[k][0].y, z[k][1].x, z[k][1].y);
                dst[1] = make_float4(z[k][2].x, z[k][2].y, z[k][3].x, z[k][3].y);
            }
            __syncwarp();
        }
        if (ROPE == kHalves128) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 lo = z[0][e], hi = z[NC > 1 ? 1 : 0][e];
                z[0][e] = fma2(lo, cs[0][e], mul2(hi, sn[0][e]));
                z[NC > 1 ? 1 : 0][e] = fma2(hi, cs[NC > 1 ? 1 : 0][e], mul2(lo, sn[NC > 1 ? 1 : 0][e]));
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int c = l + 8 * k;
            if (c < 2 * shift) {
                float2 q[4];
                if (ROPE == kHalves) load8(mine + 8 * (c < shift ? c + shift : c - shift), q);
                else
#pragma unroll
                    for (int e = 0; e < 4; ++e) q[e] = make_float2(z[k][e].y, z[k][e].x);
#pragma unroll
                for (int e = 0; e < 4; ++e) z[k][e] = fma2(z[k][e], cs[k][e], mul2(q[e], sn[k][e]));
            }
        }
    };

    for (uint32_t item = first; item < end; ++item) {
        copy_wait<DEPTH - 1>();  // this item's copies have landed (this lane's; with the barrier, the warp's)
        if (ROPE != kNoRope) __syncwarp();
        uint4 xr[NC], yr[NC];
        const uint8_t *slot = ring + (item - first) % DEPTH * ROWS16 * 512 + lane * 16;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            xr[k] = *reinterpret_cast<const uint4 *>(slot + k * 512);
            if (BWD) yr[k] = *reinterpret_cast<const uint4 *>(slot + (NC + k) * 512);
        }
        if (item == first || c_hb == 0) {
            const int64_t h = int64_t(c_hb) * kItemHeads + grp;
            yp = static_cast<T *>(s.y.ptr) + c_b * s.y.sb + h * s.y.sh + c_i * s.y.ss + l * 8;
            if (ROPE != kNoRope) {
                load_angles();
                __syncwarp();  // read before the copies of a later token
            }
        }
        issue(item + DEPTH);
        if (ROPE != kNoRope && !valid) {  // a token out of range: with a row and angles of zeros it adds nothing to the
                                          // weights' gradient, and its outputs are zeros whatever the weights hold
#pragma unroll
            for (int k = 0; k < NC; ++k) xr[k] = yr[k] = make_uint4(0, 0, 0, 0);
        }
        float2 x[NC][4], z[NC][4];
        float2 sq = both(0.f);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            unpack8<T>(xr[k], x[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) sq = fma2(x[k][e], x[k][e], sq);
        }
        const float r = rsqrtf(fmaf(row_sum(sq.x + sq.y), 1.f / D, a.eps));
        if (!BWD) {  // the norm's factor is common to a row: it goes on last
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[k][e] = mul2(x[k][e], w[k][e]);
            turn(z);
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[k][e] = mul2(z[k][e], both(r));
        } else {
#pragma unroll
            for (int k = 0; k < NC; ++k) unpack8<T>(yr[k], z[k]);
            turn(z);
            float2 dot = both(0.f);
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[k][e] = mul2(x[k][e], both(r));
                    dw[k][e] = fma2(z[k][e], x[k][e], dw[k][e]);
                    z[k][e] = mul2(z[k][e], w[k][e]);
                    dot = fma2(z[k][e], x[k][e], dot);
                }
            const float mean = row_sum(dot.x + dot.y) * (-1.f / D);
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[k][e] = mul2(fma2(x[k][e], both(mean), z[k][e]), both(r));
        }
        if (int64_t(c_hb) * kItemHeads + grp < s.h) {
#pragma unroll
            for (int k = 0; k < NC; ++k)
                *reinterpret_cast<uint4 *>(yp + 64 * k) = ROPE == kNoRope || valid ? pack8<T>(z[k]) : make_uint4(0, 0, 0, 0);
        }
        yp += kItemHeads * s.y.sh;
        if (++c_hb == nhb) {
            c_hb = 0;
            ++c_token;
            if (++c_i == uint32_t(a.s)) {
                c_i = 0;
                ++c_b;
            }
        }
    }
    copy_wait<0>();
    if (BWD && s.dw) {  // this block's share of the weight gradient: rows of a warp, then the warps in order
        __shared__ float red[kWarps][D];
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = e & 1 ? dw[k][e / 2].y : dw[k][e / 2].x;
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (grp == 0) red[warp][(l + 8 * k) * 8 + e] = v;
            }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += 32 * kWarps) {
            float v = 0.f;
            for (int k = 0; k < kWarps; ++k) v += red[k][c];
            s.part[int64_t(cta) * D + c] = v;
        }
    }
    if (BWD) pdl_trigger();
}

// Weight gradients: the blocks' shares, summed in a fixed order.  One block per side and 32 columns;
// warp k of 32 takes every 32nd share.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const QkNormArgs a)
{
    __shared__ float red[32][33];
    const QkSide &s = a.side[blockIdx.y];
    pdl_wait();
    if (!s.dw) return;
    const int k = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.f;
    for (int p = k; p < s.blocks; p += 32) v += s.part[int64_t(p) * a.d + c];
    red[k][lane] = v;
    __syncthreads();
    v = red[lane][k];  // transposed: warp k sums column k
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) s.dw[blockIdx.x * 32 + k] = v;
}

template <class T, int NC, int ROPE, bool BWD> cudaError_t run(QkNormArgs a, cudaStream_t st)
{
    // one wave of blocks, or fewer when that gives every warp an item, shared out by the sides' rows
    static const int sms = []() {
        int dev = 0, n = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) n = 0;
        return n > 0 ? n : 1;
    }();
    const int64_t wave = sms * kBlocksPerSm<NC, BWD> - 1 < kQkBlocks ? sms * kBlocksPerSm<NC, BWD> - 1 : kQkBlocks;
    const int64_t t = a.b * a.s;
    int64_t want[2], total = 0;
    for (int k = 0; k < 2; ++k) {
        const int64_t nhb = (a.side[k].h + kItemHeads - 1) / kItemHeads;
        want[k] = (t * nhb + kWarps - 1) / kWarps;
        total += want[k];
    }
    for (int k = 0; k < 2; ++k) {
        int64_t n = want[k];
        if (total > wave) {
            n = want[k] * wave / total;
            if (n < 1 && want[k] > 0) n = 1;
        }
        a.side[k].blocks = int(n);
    }
    const int grid = 1 + a.side[0].blocks + a.side[1].blocks;
    if (BWD) a.side[1].part = a.side[0].part + int64_t(a.side[0].blocks) * a.d;
    a.warp_smem = warp_smem<NC, ROPE, BWD>(a.rot);
    const int smem = kWarps * a.warp_smem;
    auto k = qk_norm_kernel<T, NC, ROPE, BWD>;
    cudaError_t e = cudaSuccess;
    if (smem > 40 * 1024) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_kernel(k, dim3(grid), dim3(32 * kWarps), size_t(smem), st, false, a);
    if (e == cudaSuccess && BWD && (a.side[0].dw || a.side[1].dw))
        e = launch_kernel(qk_norm_dw_kernel, dim3(unsigned(a.d / 32), 2), dim3(1024), 0, st, true, a);
    return e;
}

template <class T, int NC, bool BWD> cudaError_t pick_rope(const QkNormArgs &a, cudaStream_t s)
{
    if (a.rot == 0) return run<T, NC, kNoRope, BWD>(a, s);
    if (a.interleaved) return run<T, NC, kPairs, BWD>(a, s);
    if constexpr (NC > 1)
        if (a.rot == 128) return run<T, NC, kHalves128, BWD>(a, s);
    return run<T, NC, kHalves, BWD>(a, s);
}

template <class T, bool BWD> cudaError_t pick_dim(const QkNormArgs &a, cudaStream_t s)
{
    return a.d == 64 ? pick_rope<T, 1, BWD>(a, s) : a.d == 128 ? pick_rope<T, 2, BWD>(a, s) : pick_rope<T, 3, BWD>(a, s);
}

}  // namespace

cudaError_t launch_qk_norm(const QkNormArgs &a, bool backward, cudaStream_t s)
{
    if (a.dtype == ATTN_F16) return backward ? pick_dim<__half, true>(a, s) : pick_dim<__half, false>(a, s);
    return backward ? pick_dim<__nv_bfloat16, true>(a, s) : pick_dim<__nv_bfloat16, false>(a, s);
}

}  // namespace attn
