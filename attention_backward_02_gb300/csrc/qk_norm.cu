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
// rotary_dim that is a multiple of 16.  A work item is a token and a few of its
// heads, so a lane loads its cos and sin values once for them.  Blocks work on
// one side (query or key heads) each, so weights and weight-gradient sums stay
// in registers.
#include <cstdint>

#include "qk_norm.h"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kItemHeads = 4;  // rows a warp works on side by side

template <class T> __device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 p = unpack2<T>(w[e]);
        f[2 * e] = p.x;
        f[2 * e + 1] = p.y;
    }
}

template <class T> __device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
}

__device__ __forceinline__ void load8(const float *p, float (&f)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// sum over the 8 lanes of a row
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

enum { kNoRope = 0, kHalves = 1, kPairs = 2 };

// NC = d / 64 chunks a lane; U rows of a lane in flight at once.
template <class T, int NC, int ROPE, bool BWD, int U>
__global__ void __launch_bounds__(32 * kWarps) qk_norm_kernel(const QkNormArgs a)
{
    constexpr int D = NC * 64;
    __shared__ float xch[ROPE == kHalves ? kWarps * kItemHeads * D : 1];
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
    float *const mine = xch + (ROPE == kHalves ? (warp * kItemHeads + grp) * D : 0);

    float w[NC][8], dw[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = (l + 8 * k) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw[k][e] = 0.f;
            w[k][e] = 1.f;
        }
        if (s.w) {
            if (a.weight_fp32) load8(static_cast<const float *>(s.w) + c, w[k]);
            else unpack8<T>(*reinterpret_cast<const uint4 *>(static_cast<const T *>(s.w) + c), w[k]);
        }
    }
    const int shift = int(a.rot) / 16;  // chunks between the halves of a rotated pair
    const uint32_t nhb = uint32_t((s.h + kItemHeads * U - 1) / (kItemHeads * U));
    const uint32_t items = uint32_t(a.b * a.s) * nhb;
    for (uint32_t item = cta * kWarps + warp; item < items; item += uint32_t(s.blocks) * kWarps) {
        const uint32_t t = item / nhb, hb = item - t * nhb;
        const uint32_t b = t / uint32_t(a.s), i = t - b * uint32_t(a.s);
        uint4 xr[U][NC], yr[U][NC];
        int64_t off_y[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t h = int64_t(hb) * (kItemHeads * U) + u * kItemHeads + grp;
            on[u] = h < s.h;
            off_y[u] = b * s.y.sb + h * s.y.sh + i * s.y.ss;
            const T *x = static_cast<const T *>(s.x.ptr) + b * s.x.sb + h * s.x.sh + i * s.x.ss;
            const T *dy = static_cast<const T *>(s.dy.ptr) + b * s.dy.sb + h * s.dy.sh + i * s.dy.ss;
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                xr[u][k] = yr[u][k] = make_uint4(0, 0, 0, 0);
                if (on[u]) {
                    xr[u][k] = *reinterpret_cast<const uint4 *>(x + (l + 8 * k) * 8);
                    if (BWD) yr[u][k] = *reinterpret_cast<const uint4 *>(dy + (l + 8 * k) * 8);
                }
            }
        }
        // cos and sin of this lane's elements (sin with the sign of the turn)
        float cs[NC][8], sn[NC][8];
        bool valid = true;
        if (ROPE != kNoRope) {
            const int32_t p = a.pos ? a.pos[t] : int32_t(i);
            valid = p >= 0 && p < a.max_pos;
            const float *cr = a.cos + int64_t(valid ? p : 0) * (a.rot / 2), *sr = a.sin + int64_t(valid ? p : 0) * (a.rot / 2);
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const int c = l + 8 * k;
                if (c < 2 * shift) {
                    if (ROPE == kHalves) {
                        const bool lo = c < shift;
                        load8(cr + 8 * (lo ? c : c - shift), cs[k]);
                        load8(sr + 8 * (lo ? c : c - shift), sn[k]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) sn[k][e] = (lo != BWD) ? -sn[k][e] : sn[k][e];
                    } else {
                        const float4 c4 = *reinterpret_cast<const float4 *>(cr + 4 * c), s4 = *reinterpret_cast<const float4 *>(sr + 4 * c);
                        const float cv[4] = {c4.x, c4.y, c4.z, c4.w}, sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            cs[k][2 * e] = cs[k][2 * e + 1] = cv[e];
                            sn[k][2 * e] = BWD ? sv[e] : -sv[e];
                            sn[k][2 * e + 1] = -sn[k][2 * e];
                        }
                    }
                }
            }
        }
        // z (backward: dy) turned by the token's angle, in place
        auto turn = [&](float (&z)[NC][8]) {
            if (ROPE == kNoRope) return;
            if (ROPE == kHalves) {
                __syncwarp();  // the previous row's partners have been read
#pragma unroll
                for (int k = 0; k < NC; ++k) {
                    float4 *dst = reinterpret_cast<float4 *>(mine + (l + 8 * k) * 8);
                    dst[0] = make_float4(z[k][0], z[k][1], z[k][2], z[k][3]);
                    dst[1] = make_float4(z[k][4], z[k][5], z[k][6], z[k][7]);
                }
                __syncwarp();
            }
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                const int c = l + 8 * k;
                if (c < 2 * shift) {
                    float q[8];
                    if (ROPE == kHalves) load8(mine + 8 * (c < shift ? c + shift : c - shift), q);
                    else
#pragma unroll
                        for (int e = 0; e < 8; ++e) q[e] = z[k][e ^ 1];
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[k][e] = fmaf(z[k][e], cs[k][e], q[e] * sn[k][e]);
                }
            }
        };
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[NC][8];
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                unpack8<T>(xr[u][k], x[k]);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[k][e], x[k][e], ss);
            }
            const float r = rsqrtf(fmaf(row_sum(ss), 1.f / D, a.eps));
            float z[NC][8];
            if (!BWD) {
#pragma unroll
                for (int k = 0; k < NC; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[k][e] = x[k][e] * r * w[k][e];
                turn(z);
            } else {
#pragma unroll
                for (int k = 0; k < NC; ++k) unpack8<T>(yr[u][k], z[k]);
                turn(z);
                float dot = 0.f;
#pragma unroll
                for (int k = 0; k < NC; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[k][e] *= r;
                        if (valid && on[u]) dw[k][e] = fmaf(z[k][e], x[k][e], dw[k][e]);
                        z[k][e] *= w[k][e];
                        dot = fmaf(z[k][e], x[k][e], dot);
                    }
                dot = row_sum(dot) * (1.f / D);
#pragma unroll
                for (int k = 0; k < NC; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[k][e] = r * fmaf(-x[k][e], dot, z[k][e]);
            }
            if (on[u]) {
                T *y = static_cast<T *>(s.y.ptr) + off_y[u];
#pragma unroll
                for (int k = 0; k < NC; ++k)
                    *reinterpret_cast<uint4 *>(y + (l + 8 * k) * 8) = valid ? pack8<T>(z[k]) : make_uint4(0, 0, 0, 0);
            }
        }
    }
    if (BWD && s.dw) {  // this block's share of the weight gradient: rows of a warp, then the warps in order
        __shared__ float red[kWarps][D];
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = dw[k][e];
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
    constexpr int U = NC == 1 ? 4 : (BWD ? 1 : 2);
    // blocks: one a few items of each warp, at most kQkBlocks, shared out by the sides' rows
    const int64_t t = a.b * a.s;
    int64_t want[2], total = 0;
    for (int k = 0; k < 2; ++k) {
        const int64_t nhb = (a.side[k].h + kItemHeads * U - 1) / (kItemHeads * U);
        want[k] = (t * nhb + kWarps - 1) / kWarps;
        total += want[k];
    }
    for (int k = 0; k < 2; ++k) {
        int64_t n = want[k];
        if (total > kQkBlocks) {
            n = want[k] * kQkBlocks / total;
            if (n < 1 && want[k] > 0) n = 1;
        }
        a.side[k].blocks = int(n);
    }
    const int grid = 1 + a.side[0].blocks + a.side[1].blocks;
    if (BWD) a.side[1].part = a.side[0].part + int64_t(a.side[0].blocks) * a.d;
    cudaError_t e = launch_kernel(qk_norm_kernel<T, NC, ROPE, BWD, U>, dim3(grid), dim3(32 * kWarps), 0, st, false, a);
    if (e == cudaSuccess && BWD && (a.side[0].dw || a.side[1].dw))
        e = launch_kernel(qk_norm_dw_kernel, dim3(unsigned(a.d / 32), 2), dim3(1024), 0, st, true, a);
    return e;
}

template <class T, int NC, bool BWD> cudaError_t pick_rope(const QkNormArgs &a, cudaStream_t s)
{
    if (a.rot == 0) return run<T, NC, kNoRope, BWD>(a, s);
    return a.interleaved ? run<T, NC, kPairs, BWD>(a, s) : run<T, NC, kHalves, BWD>(a, s);
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
