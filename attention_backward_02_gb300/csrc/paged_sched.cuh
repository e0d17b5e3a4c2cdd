// paged_sched.cuh -- how the attention over a paged cache is shared out among the
// CTAs of a launch, on the device, from lengths that only the device has.
//
// A unit is (sequence, head block, query tile): `tokens` new tokens of the sequence
// with the query heads of a block.  Its keys are those its last token sees, K, and its
// cost K + kUnitCost keys.  The units in order make one long row of keys, which the CTAs
// share evenly: a CTA's range begins and ends anywhere inside a unit, so sequences of
// any mix of lengths load the GPU evenly with no choice of a split by the host.  A unit
// that several CTAs share is joined from their partial results; all but its first
// piece are the first of their CTA and its first one the last of its CTA, so a CTA has
// at most two of them.  Range borders are a function of the CTA's number alone, which
// both neighbours evaluate.
#pragma once

#include "paged.h"

namespace attn {
namespace paged {

struct Range {
    // Unit: sequence n, head block x, query tile t; key: where in it.
    int n0, x0, t0, k0;
    int n1, x1, t1, k1;  // n1 == b: up to the last unit
    bool any;
};

// A sequence's units: nt query tiles for each of the head blocks.
struct SeqUnits {
    int first, m, len, nt;
};

// a / b (less than 2^20) and the remainder: an estimate in fp32, which is off by one at most, put right.  (The code of a
// 64-bit division is long, and a CTA runs it once: fetching it took longer than the rest of the range's arithmetic.)
__host__ __device__ __forceinline__ int quotient(int64_t a, int64_t b, int64_t *rest)
{
#ifdef __CUDA_ARCH__
    int q = int(__fdividef(float(a), float(b)));
#else
    int q = int(float(a) / float(b));
#endif
    int64_t r = a - q * b;
    if (r < 0) {
        --q;
        r += b;
    } else if (r >= b) {
        ++q;
        r -= b;
    }
    *rest = r;
    return q;
}

// Cost of the tiles before t of one head block.  (Not inlined: it is called from several places that a CTA passes once.)
template <int kUnitCost>
__host__ __device__ __noinline__ int64_t cost_before(int causal, int tokens, int m, int len, int nt, int t)
{
    int64_t c = int64_t(t) * kUnitCost;
    if (!causal) return c + int64_t(t) * len;
    const int full = t < nt ? t : nt - 1;  // tiles of `tokens` tokens each
    const int past = len - m;
    const int from = past < 0 ? (-past / tokens < full ? -past / tokens : full) : 0;  // the first that sees keys
    c += int64_t(full - from) * past + int64_t(tokens) * (int64_t(full) * (full + 1) - int64_t(from) * (from + 1)) / 2;
    return t < nt ? c : c + len;
}

template <int kUnitCost> struct Sched {
    PagedSeqs s;
    int tokens;   // new tokens of a query tile
    int heads;    // head blocks: kv heads x row blocks
    int causal;

    __host__ __device__ __forceinline__ SeqUnits units(int n, bool *bad) const
    {
        SeqUnits u;
        s.rows(n, &u.first, &u.m, bad);
        u.len = s.len(n, bad);
        u.nt = (u.m + tokens - 1) / tokens;
        return u;
    }
    // keys that tile t sees
    __host__ __device__ __forceinline__ int keys(const SeqUnits &u, int t) const
    {
        if (!causal) return u.len;
        const int last = (t + 1) * tokens < u.m ? (t + 1) * tokens : u.m;
        const int k = u.len - u.m + last;
        return k > 0 ? k : 0;
    }
    // cost of the tiles before t of one head block
    __host__ __device__ __forceinline__ int64_t before(const SeqUnits &u, int t) const
    {
        return cost_before<kUnitCost>(causal, tokens, u.m, u.len, u.nt, t);
    }
    __host__ __device__ __forceinline__ int64_t cost(const SeqUnits &u) const { return u.nt ? heads * before(u, u.nt) : 0; }

    // Where `at` of sequence n's cost lies; keys cut to multiples of kStep, pieces of less than kLeast keys avoided.
    template <int kStep, int kLeast>
    __host__ __device__ __forceinline__ void locate(const SeqUnits &u, int64_t at, int *x, int *t, int *k) const
    {
        *x = quotient(at, before(u, u.nt), &at);
        int lo = 0, hi = u.nt - 1;  // the last tile that begins at or before
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (before(u, mid) <= at) lo = mid;
            else hi = mid - 1;
        }
        *t = lo;
        const int all = keys(u, lo);
        int key = int(at - before(u, lo)) - kUnitCost;
        key = key > 0 ? key / kStep * kStep : 0;
        if (key < kLeast) key = 0;
        if (key > 0 && all - key < kLeast) key = all;
        *k = key;
    }

    // CTAs that have a share worth a start, and where the range of CTA c begins, of a total cost.
    template <int kShare> static __host__ __device__ __forceinline__ int shares(int64_t total, int ctas)
    {
        static_assert((kShare & (kShare - 1)) == 0, "a shift");
        const int64_t n = (total + kShare - 1) / kShare;
        return n > ctas ? ctas : n < 1 ? 1 : int(n);
    }
    // (total c / n, in fractions of 2^-32)
    static __host__ __device__ __forceinline__ int64_t border(int64_t total, int n, int c)
    {
        if (c >= n) return total;
        const uint64_t part = uint64_t(0xffffffffu / uint32_t(n)) * uint32_t(c);
        return int64_t((uint64_t(total) >> 32) * part + ((uint64_t(total) & 0xffffffffu) * part >> 32));
    }

    // The range of CTA c.  All threads of the block; `scratch`: kThreads / 32 + 12 64-bit words of shared memory.  *bad: counts or lengths
    // out of range (known to CTA 0's threads only).
    template <int kThreads, int kStep, int kLeast, int kShare>
    __device__ Range range(int c, int ctas, int64_t *scratch, bool *bad) const
    {
        const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
        const int each = (s.b + kThreads - 1) / kThreads;  // sequences of a thread, in order
        const int lo = tid * each < s.b ? tid * each : s.b, hi = lo + each < s.b ? lo + each : s.b;
        int64_t mine = 0;
        SeqUnits u = {0, 0, 0, 0};
        for (int n = lo; n < hi; ++n) {
            u = units(n, bad);
            mine += cost(u);
        }
        int64_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        // scratch: the warps' sums; where the two borders lie (sequences, cost from the first's start on, the last one's
        // units); the range
        struct Found {
            int64_t off;
            int lo, hi;
            SeqUnits u;
        };
        Found *found = reinterpret_cast<Found *>(scratch + kThreads / 32);
        int *out = reinterpret_cast<int *>(found + 2);
        if (lane == 31) scratch[warp] = sum;
        if (tid < 2) found[tid].lo = s.b;
        __syncthreads();
        int64_t base = sum - mine, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) base += scratch[w];
            total += scratch[w];
        }
        const int n_cta = shares<kShare>(total, ctas);
        if (c < n_cta && mine > 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t at = border(total, n_cta, c + e);
                if (at >= base && at < base + mine) found[e] = {at - base, lo, hi, u};  // (else another thread's, or the end)
            }
        }
        __syncthreads();
        if (lane == 0 && warp < 2) {  // a warp each: one after the other took 1500 cycles more
            const Found f = found[warp];
            int n = f.lo, x = 0, t = 0, k = 0;
            if (n < s.b) {
                bool none = false;
                u = f.u;
                int64_t off = f.off;
                if (f.hi - f.lo > 1) {
                    u = units(n, &none);
                    for (int64_t w = cost(u); off >= w; w = cost(u)) {
                        off -= w;
                        u = units(++n, &none);
                    }
                }
                locate<kStep, kLeast>(u, off, &x, &t, &k);
            }
            out[4 * warp] = n;
            out[4 * warp + 1] = x;
            out[4 * warp + 2] = t;
            out[4 * warp + 3] = k;
        }
        __syncthreads();
        Range r;
        r.any = c < n_cta && total > 0;
        r.n0 = out[0]; r.x0 = out[1]; r.t0 = out[2]; r.k0 = out[3];
        r.n1 = out[4]; r.x1 = out[5]; r.t1 = out[6]; r.k1 = out[7];
        return r;
    }
};

// Where the pages' rows are short (a head's 128 bytes), reading one head's alone uses little of what DRAM opens for it.
// So up to 16 neighbouring head blocks, which cost the same, are shared out alike, a lane each, and CTAs that start together
// read the same keys of neighbouring heads (32 e4m3 sequences of 8192 keys, 8 heads of 128: 122 us, so 105; not for the
// tensor-core kernel, which its arithmetic binds: mixed chunks 330 us, so 345).  A lane's units hold the head blocks lane,
// lane + lanes ..; the CTAs' numbers are in the lanes' order, so that a unit's pieces lie one behind the other.
struct Lanes {
    int lanes, lane;  // this CTA's lane
    int per, share;   // shares of a lane, and this CTA's (per: it has none)
    int me;           // its number
    __host__ __device__ __forceinline__ Lanes(int heads, int ctas, int c)
    {
        lanes = heads < 16 ? heads : 16;
        while (heads % lanes) --lanes;
        per = ctas / lanes;
        lane = c % lanes;
        share = c < per * lanes ? c / lanes : per;
        me = c < per * lanes ? lane * per + share : c;
    }
};

// One CTA's walk over its pieces.
template <int kUnitCost> struct Walk {
    const Sched<kUnitCost> &sc;
    const Range &r;
    int n, x, t;     // the unit at hand
    SeqUnits u;
    int k0, k1, all; // keys of it that are this CTA's, and all
    bool first;

    __host__ __device__ __forceinline__ Walk(const Sched<kUnitCost> &s, const Range &range) : sc(s), r(range), first(true) {}

    // To the next piece; false behind the last.  A unit without keys is a piece of its own (its output is zeros).
    __host__ __device__ __forceinline__ bool next()
    {
        bool bad = false;
        if (first) {
            if (!r.any) return false;
            n = r.n0; x = r.x0; t = r.t0;
            u = sc.units(n, &bad);
        }
        for (;;) {
            int from = 0;
            if (first) {
                from = r.k0;
                first = false;
            } else {
                if (n == r.n1 && x == r.x1 && t == r.t1) return false;
                if (++t == u.nt) {
                    t = 0;
                    if (++x == sc.heads) {
                        x = 0;
                        do {
                            if (++n >= sc.s.b) return false;
                            u = sc.units(n, &bad);
                        } while (u.nt == 0);
                    }
                }
            }
            const bool last = n == r.n1 && x == r.x1 && t == r.t1;
            all = sc.keys(u, t);
            k0 = from;
            k1 = last && r.k1 < all ? r.k1 : all;
            if (k0 < k1 || (all == 0 && from == 0 && !last)) return true;
        }
    }
    __host__ __device__ __forceinline__ bool begins() const { return k0 == 0; }
    __host__ __device__ __forceinline__ bool ends() const { return k1 == all; }
};

// A value's scale is 2^E f, |f| in [1, 2): E + 127 as an exponent's bits, E, and 2^-E.  (E is held between -80 and 126, so that sums of
// 2^-E stay in range; |f| is below 1 for smaller scales and up to 4 for larger ones.)
__device__ __forceinline__ uint32_t exponent_bits(float scale)
{
    return min(max(__float_as_uint(scale) & 0x7f800000u, (127u - 80u) << 23), (127u + 126u) << 23);
}
__device__ __forceinline__ float exponent_of(uint32_t u) { return __uint_as_float(0x4b000000u | u >> 23) - (8388608.f + 127.f); }
__device__ __forceinline__ float exponent_inv(uint32_t u) { return __uint_as_float((254u << 23) - u); }

// Natural log of l 2^m (+inf where no key was seen).  The exponent of l joins m before the logarithm of its fraction
// is added: m and it may be far apart and cancel.
__device__ __forceinline__ float lse_of(float m, float l)
{
    if (l == 0.f) return INFINITY;
    const uint32_t u = __float_as_uint(l);
    if ((u >> 23) - 1u >= 254u) return (m + __log2f(l)) / kLog2e;  // (no normal number: as it comes)
    return ((m + float(int(u >> 23) - 127)) + __log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u))) / kLog2e;
}

// The unit's name in a share's record, for the join.
__host__ __device__ __forceinline__ int4 unit_name(int n, int x, int t, int state) { return make_int4(n, x, t, state); }
enum { kNone = 0, kGoesOn = 1, kEnds = 2 };  // state: no partial result, one that others follow, a unit's last

}  // namespace paged
}  // namespace attn
