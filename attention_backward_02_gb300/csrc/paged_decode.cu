// paged_decode.cu -- attention of a few new tokens per sequence over a paged key /
// value cache, 16-bit or e4m3, and the join of the partial results of both paged
// attention kernels.
//
// A unit (paged_sched.cuh) is up to ROWS rows: as many tokens as fit with the query
// heads that share a kv head, or one token with ROWS of them.  Row (token i, head x):
//   s_j = scale q.k_j over the keys j <= its position,  O = sum_j exp(s_j) v_j / sum_j exp(s_j).
//
// Bound by HBM: every cached key and value is read once a row block against 4 d ROWS
// operations.  A CTA takes its range of keys in stages of 64 or 128, which a producing warp
// brings into a ring in shared memory by TMA (a lane looks up a page, a stage ahead, and
// issues its boxes), so that loads run under the arithmetic and over the ends of pieces;
// four warps take 16 or 32 keys of a stage each.  Both products are mma.sync m16n8k16,
// which keeps the operations off the critical path; what a warp's step takes is their
// latency and the softmax's (650 + 500 + 400 cycles for 16 keys, whether numbers are
// converted or not), so where a key has at most 128 bytes it takes 32.  S = Q K^T has the
// rows as its rows; its accumulator is, as it stands, the second operand of O^T = V^T P^T,
// whose rows are head dims and whose eight columns are rows of S.  The operands are 16-byte
// reads of shared memory as they stand: the order of the contraction over d is free, so a
// lane's 16 bytes of a key serve several steps, and V's key pairs are joined by byte
// permutes.  Keys lie in blocks of 64 bytes a row, in which the eight lanes of a read take
// two whole rows; values in rows of 128 bytes with the 128-byte swizzle, in which they take
// pieces of four rows: neither has bank conflicts (values of 64 e4m3 numbers have two-way
// ones).  CTAs that start together take the same keys of neighbouring heads (Lanes): a head's
// 128 bytes of e4m3 numbers alone came at 0.66 of the measured copy rate even with the
// arithmetic left out, side by side at 0.81 with it.  32 sequences of 1 to 8192 keys, 32 / 8
// heads of 128: 95 us for 537 MB, 0.83 of that rate (all of 8192: 166, 0.95), e4m3 62 us for
// 277 MB, 0.66 (101, 0.81): beside the reading stand the start (a share's range, first loads),
// units that end early and the join.
//
// e4m3: a number is a half-precision number exactly, one conversion a pair, so both products
// are of that type whatever the queries' is.  bf16 queries are scaled by a power of two per row that
// brings their largest element to 2^14 .. 2^15 (exact but for elements 2^-38 below it);
// a key's scale and that power multiply its score.  A value's scale is 2^E f, |f| in [1, 2), and its key's
// weight e^s 2^E f: E joins the score s (log2 units), so that the row's running maximum R is that of s + E over the keys
// that it sees, and P = 2^(s + E - R) says what a key counts for in O.  (Relative to the largest value scale the
// weights lost bits to keys of no weight and to keys that the row does not see.)  l takes P 2^-E, O the products of
// P f and the numbers; both are in units of 2^R.  E is held between -80 and 126, so that l stays in range.
//
// The weights P are rounded to the 16-bit type of the product with V, after their sum is taken: its
// operands are 16-bit, and a weight is off by half a step of that type.
#include <type_traits>

#include "paged.h"
#include "paged_sched.cuh"
#include "sm103.cuh"
#include "tc_util.cuh"
#include "tmap.h"

namespace attn {

using namespace paged;
using namespace sm103;

namespace {

constexpr int kKeyWarps = 4;     // warps that share a stage's keys
constexpr int kUnitCost = 384;   // what a unit's start and end take, in keys (32 e4m3 sequences of 1 to 8192 keys: 128 85 us, 256 73, 384 69)
constexpr int kShare = 256;      // a share worth a start
constexpr int kJoin = 256;       // threads of the join

// CTAs an SM holds: as many as leave each a ring of two stages or more.  (16 bits, d = 128: three with two stages 100 us for
// 32 sequences of 1 to 8192 keys, two with three 97.)
constexpr int decode_blocks(int d, int esize)
{
    return d * esize == 64 ? 3 : 2;
}

template <int D, bool kEight, int ROWS> struct DecodeCfg {
    static constexpr int NR = ROWS / 8;                    // rows of a lane
    static constexpr int CONSUMERS = 32 * kKeyWarps, THREADS = CONSUMERS + 32;
    static constexpr int ESIZE = kEight ? 1 : 2;
    static constexpr int SUB = D * ESIZE <= 128 ? 2 : 1;   // blocks of 16 keys that a warp takes at once
    static constexpr int KEYS = 16 * SUB, STAGE_KEYS = kKeyWarps * KEYS;
    static constexpr int SIDE = STAGE_KEYS * D * ESIZE;    // keys, or values, of a stage
    static constexpr int OS = D + 2;                       // a row of sums: two rows of a lane lie in other banks
    static constexpr int O_BYTES = 2 * ROWS * OS * 4;      // [2][ROWS][OS] floats
    static constexpr int BLOCKS = decode_blocks(D, ESIZE);
    static constexpr int OTHER = O_BYTES + 2 * kKeyWarps * ROWS * 4 + 512 + 1024;
    static constexpr int STAGE = 2 * SIDE + (kEight ? 2 * STAGE_KEYS * 4 : 0) + 16;
    static constexpr int FIT = ((227 * 1024 / BLOCKS - 1024) - OTHER) / STAGE;
    static constexpr int NST = FIT > 12 ? 12 : FIT;
    static_assert(NST >= 2, "a ring of two stages");
    static constexpr int OFF_V = NST * SIDE;               // after the ring of keys
    static constexpr int OFF_SCALE = OFF_V + NST * SIDE;   // [NST][keys, values][STAGE_KEYS]
    static constexpr int OFF_O = OFF_SCALE + (kEight ? NST * 2 * STAGE_KEYS * 4 : 0);
    static constexpr int OFF_M = OFF_O + O_BYTES;          // [key warp][ROWS] maxima, then sums
    static constexpr int OFF_BAR = OFF_M + 2 * kKeyWarps * ROWS * 4;
    static constexpr int OFF_MISC = OFF_BAR + 2 * NST * 8;
    static constexpr int OFF_RANGE = OFF_MISC + 16;        // scratch of the range
    static constexpr int SMEM = OFF_RANGE + (THREADS / 32 + 12) * 8 + 1024;
    static_assert(SMEM <= 227 * 1024 / BLOCKS - 1024, "shared memory budget");
};

struct DecodeParams {
    CUtensorMap tm_k, tm_v;
    PagedAttnArgs a;
};

__device__ __forceinline__ float ex2f(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 lds8(uint32_t addr)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

__device__ __forceinline__ float2 lds_pair(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}

// two e4m3 numbers as half-precision ones
__device__ __forceinline__ uint32_t to_half2(uint32_t e4m3x2)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(e4m3x2)));
    return h;
}

// 4 bytes, global to shared, asynchronous (zeros where `on` is false; the address is then not read)
__device__ __forceinline__ void copy4(uint32_t dst, const float *src, bool on)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
// One arrival on the barrier once this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
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

// A power of two that brings |x| <= most to 2^14 .. 2^15.
__device__ __forceinline__ float half_range(float most)
{
    const uint32_t e = __float_as_uint(fminf(fmaxf(most, 0x1p-100f), 0x1p+127f)) >> 23;
    return __uint_as_float((127u + 14u + 127u - e) << 23);
}

// ROWS: rows of a unit, 8 (the second half of S's rows is zero and never looked at) or 16.  (32, two warps to the same
// keys: drafted tokens of 28 rows 67 us, as two units of 16 that read the keys twice 52.)
template <class T, bool kEight, int D, int ROWS>
__global__ void __launch_bounds__(DecodeCfg<D, kEight, ROWS>::THREADS, DecodeCfg<D, kEight, ROWS>::BLOCKS)
    paged_decode_kernel(const __grid_constant__ DecodeParams p)
{
    using Cfg = DecodeCfg<D, kEight, ROWS>;
    using M = typename std::conditional<kEight, __half, T>::type;  // the products' type
    constexpr int NQ = D / 8;                // 32-bit words of a query row in a lane
    constexpr int NE = D / 16;               // products of O^T
    constexpr int NR = Cfg::NR, NST = Cfg::NST;
    constexpr int KL = D * Cfg::ESIZE / 64;  // reads of a key
    constexpr int SUB = Cfg::SUB, kKeys = Cfg::KEYS, kStage = Cfg::STAGE_KEYS;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_BAR), *empty = full + NST;
    volatile int *abort = reinterpret_cast<volatile int *>(smem + Cfg::OFF_MISC);
    volatile int *bad_page = abort + 1;
    const PagedAttnArgs &a = p.a;
    const PagedCache &cache = a.cache;

    pdl_trigger();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        *abort = 0;
        *bad_page = 0;
        for (int s = 0; s < NST; ++s) {
            mbar_init(&full[s], kEight ? 1 + 32 : 1);  // the boxes, and the scales of each lane
            mbar_init(&empty[s], kKeyWarps);
        }
        fence_mbar_init();
    }
    const int G = a.h / a.h_kv, hb = G < ROWS ? G : ROWS, nrb = (G + ROWS - 1) / ROWS;
    const Lanes side(a.h_kv * nrb, gridDim.x, blockIdx.x);
    const Sched<kUnitCost> sched = {a.seqs, ROWS / hb, a.h_kv * nrb / side.lanes, a.causal};
    bool bad = false;
    const Range range = sched.range<Cfg::THREADS, kStage, kStage, kShare>(
        side.share, side.per, reinterpret_cast<int64_t *>(smem + Cfg::OFF_RANGE), &bad);  // (two barriers inside)
    if (bad && blockIdx.x == 0) *bad_page = 1;  // (one CTA reports the lengths)
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {  // the whole warp
        if (ok && !(ok = mbar_wait(bar, parity, abort))) tc::flag_abort(abort, nullptr);
        ok = __all_sync(0xffffffffu, ok);
    };
    uint32_t s = 0, par = 0;  // ring position and phase

    if (warp == kKeyWarps) {
        // ================================================= producer
        const int in_page = (1 << cache.shift) - 1, pr = 1 << cache.shift < kStage ? 1 << cache.shift : kStage;  // keys of a box
        const int boxes = kStage / pr;
        if (lane == 0) {
            prefetch_tmap(&p.tm_k);
            prefetch_tmap(&p.tm_v);
        }
        uint32_t n_stage = 0;
        Walk<kUnitCost> w(sched, range);
        while (ok && w.next()) {
            const int kvh = (w.x * side.lanes + side.lane) / nrb;
            const int32_t *table = a.seqs.table + w.n * a.seqs.table_stride;
            auto page_of = [&](int k) -> int {
                const int key = k + lane * pr;
                return lane < boxes && key < w.k1 ? table[key >> cache.shift] : -1;
            };
            int id = page_of(w.k0);
            for (int k0 = w.k0; k0 < w.k1; k0 += kStage) {
                const int next = page_of(k0 + kStage);
                if (n_stage >= uint32_t(NST)) wait(&empty[s], par ^ 1);
                if (!ok) break;
                ++n_stage;
                const int key = k0 + lane * pr;
                const bool good = id >= 0 && id < cache.n_pages;
                if (!good && lane < boxes && key < w.k1) *bad_page = 1;
                if (lane == 0) mbar_arrive_expect_tx(&full[s], 2 * Cfg::SIDE);
                __syncwarp();
                if (lane < boxes) {
                    const int page = good ? id : cache.none;  // (out of range: zeros)
                    uint8_t *kd = smem + s * Cfg::SIDE + lane * pr * 64, *vd = smem + Cfg::OFF_V + s * Cfg::SIDE;
                    for (int c = 0; c < KL; ++c)
                        tma_load_4d(kd + c * kStage * 64, &p.tm_k, &full[s], c * 64 / Cfg::ESIZE, key & in_page, kvh, page);
                    if (D * Cfg::ESIZE == 64)
                        tma_load_4d(vd + lane * pr * 64, &p.tm_v, &full[s], 0, key & in_page, kvh, page);
                    else
                        for (int c = 0; c < KL / 2; ++c)
                            tma_load_4d(vd + c * kStage * 128 + lane * pr * 128, &p.tm_v, &full[s], c * 128 / Cfg::ESIZE, key & in_page,
                                        kvh, page);
                }
                if (kEight) {  // scales of keys lane, lane + 32 ..; 0 behind the piece's end
                    constexpr int PER = kStage / 32;
#pragma unroll
                    for (int e = 0; e < 2 * PER; ++e) {
                        const float *scale = e < PER ? cache.k_scale : cache.v_scale;
                        const int x = lane + 32 * (e % PER), pg = __shfl_sync(0xffffffffu, good ? id : -1, x / pr);
                        const bool on = pg >= 0 && k0 + x < w.k1;
                        copy4(smem_u32(smem + Cfg::OFF_SCALE) + ((2 * s + e / PER) * kStage + x) * 4,
                              on ? scale + pg * cache.sc_sp + (kvh * cache.sc_sh + ((k0 + x) & in_page) * cache.sc_ss) : scale, on);
                    }
                    copies_arrive(&full[s]);
                }
                id = next;
                if (++s == NST) {
                    s = 0;
                    par ^= 1;
                }
            }
        }
        if (lane == 0) {  // a CTA does not end before its copies, whoever may have given up
            volatile int never = 0;
            for (uint32_t j = n_stage > uint32_t(NST) ? n_stage - NST : 0; j < n_stage; ++j)
                mbar_wait(&full[j % NST], (j / NST) & 1, &never, 100000000ull);
        }
        __syncwarp();
    } else {
        // ================================================= consumers
        const int g = lane / 4, q = lane % 4, kw = warp;
        const float sc = a.scale * kLog2e;
        float *sm_m = reinterpret_cast<float *>(smem + Cfg::OFF_M), *sm_l = sm_m + kKeyWarps * ROWS;
        float *sm_o = reinterpret_cast<float *>(smem + Cfg::OFF_O);
        int4 named0 = unit_name(0, 0, 0, kNone), named1 = named0;
        auto sync = []() { named_bar_sync(1, Cfg::CONSUMERS); };
        Walk<kUnitCost> w(sched, range);
        while (w.next()) {
            const int x = w.x * side.lanes + side.lane, kvh = x / nrb, rb = x - kvh * nrb;
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
                const T *src = static_cast<const T *>(a.q.ptr) + row + head * a.q.sh;
                // 16-bit caches: 8 elements from 32 n + 8 q on; e4m3: 16 from 64 n + 16 q on
#pragma unroll
                for (int n = 0; n < NQ / 4; ++n) {
                    const int at = kEight ? 64 * (n / 2) + 16 * q + 8 * (n % 2) : 32 * n + 8 * q;
                    const uint4 v = on ? *reinterpret_cast<const uint4 *>(src + at) : make_uint4(0, 0, 0, 0);
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

            float m[NR], l[NR];  // (m: R above, of the scores alone over a 16-bit cache)
            float acc[NR][NE][4];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
#pragma unroll
                for (int e = 0; e < NE; ++e) acc[i][e][0] = acc[i][e][1] = acc[i][e][2] = acc[i][e][3] = 0.f;
            }

            for (int k0 = w.k0; k0 < w.k1; k0 += kStage) {
                const int kb = k0 + kw * kKeys;  // this warp's keys
                const int left = w.k1 - kb < kKeys ? w.k1 - kb : kKeys;
                wait(&full[s], par);
                const uint32_t ks = smem_u32(smem) + s * Cfg::SIDE + kw * kKeys * 64;
                const uint32_t vs = smem_u32(smem) + Cfg::OFF_V + s * Cfg::SIDE;
                if (ok && left > 0) {
                    // scores: lane (g, q) gets rows g, g + 8 and keys 2q, 2q + 1 of every tile of eight
                    float sa[2 * SUB][4];
                    uint4 kr[2 * SUB][KL];
#pragma unroll
                    for (int t = 0; t < 2 * SUB; ++t) {
#pragma unroll
                        for (int n = 0; n < KL; ++n) kr[t][n] = lds16(ks + n * kStage * 64 + (8 * t + g) * 64 + 16 * q);
                        sa[t][0] = sa[t][1] = sa[t][2] = sa[t][3] = 0.f;
                    }
#pragma unroll
                    for (int n = 0; n < NQ / 2; ++n)
#pragma unroll
                        for (int t = 0; t < 2 * SUB; ++t) {
                            uint32_t b0, b1;
                            if (kEight) {
                                const uint32_t x = part(kr[t][n / 4 % KL], n % 4);
                                b0 = to_half2(x);
                                b1 = to_half2(x >> 16);
                            } else {
                                b0 = part(kr[t][n / 2 % KL], 2 * (n % 2));
                                b1 = part(kr[t][n / 2 % KL], 2 * (n % 2) + 1);
                            }
                            mma16816<M>(sa[t], qa[0][2 * n], NR > 1 ? qa[NR - 1][2 * n] : 0u, qa[0][2 * n + 1],
                                        NR > 1 ? qa[NR - 1][2 * n + 1] : 0u, b0, b1);
                        }
                    float fk[4 * SUB], ve[4 * SUB];  // scales of the lane's keys, and E of the values'
                    const uint32_t size = smem_u32(smem) + Cfg::OFF_SCALE + (2 * s * kStage + kw * kKeys + 2 * q) * 4;
                    if (kEight) {
#pragma unroll
                        for (int t = 0; t < 2 * SUB; ++t) {
                            const float2 x = lds_pair(size + 32 * t), y = lds_pair(size + 4 * kStage + 32 * t);
                            fk[2 * t] = x.x; fk[2 * t + 1] = x.y;
                            ve[2 * t] = exponent_of(exponent_bits(y.x)); ve[2 * t + 1] = exponent_of(exponent_bits(y.y));
                        }
                    }
                    float x[NR][4 * SUB], mx[NR];
                    bool raise = false;
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        mx[i] = -INFINITY;
                        // (behind k1 the keys are another CTA's, or hidden from all rows)
                        const int last = (lim[i] < w.k1 - 1 ? lim[i] : w.k1 - 1) - kb - 2 * q;
#pragma unroll
                        for (int e = 0; e < 4 * SUB; ++e) {
                            const float y = sa[e >> 1][2 * i + (e & 1)];
                            x[i][e] = 8 * (e >> 1) + (e & 1) <= last ? (kEight ? fmaf(y, fs[i] * fk[e], ve[e]) : y * fs[i]) : -INFINITY;
                            mx[i] = fmaxf(mx[i], x[i][e]);
                        }
                        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
                        raise |= mx[i] > m[i];
                    }
                    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                        for (int i = 0; i < NR; ++i) {
                            const float nm = fmaxf(m[i], mx[i]);
                            const float f = nm == -INFINITY ? 1.f : ex2f(m[i] - nm);
                            m[i] = nm;
                            l[i] *= f;
                            // (the accumulator holds rows 2 q and 2 q + 1 of the eight)
                            const float f0 = __shfl_sync(0xffffffffu, f, 8 * q), f1 = __shfl_sync(0xffffffffu, f, 8 * q + 4);
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
                    uint32_t pa[2 * SUB][2];  // [key tile][row]
                    float fv[4 * SUB], vinv[4 * SUB];  // f and 2^-E (the scales read again: registers are what is short)
                    if (kEight) {
#pragma unroll
                        for (int t = 0; t < 2 * SUB; ++t) {
                            const float2 y = lds_pair(size + 4 * kStage + 32 * t);
                            vinv[2 * t] = exponent_inv(exponent_bits(y.x)); vinv[2 * t + 1] = exponent_inv(exponent_bits(y.y));
                            fv[2 * t] = y.x * vinv[2 * t]; fv[2 * t + 1] = y.y * vinv[2 * t + 1];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        const float ref = m[i] == -INFINITY ? 0.f : m[i];
                        float sum[SUB];
#pragma unroll
                        for (int t = 0; t < 2 * SUB; ++t) {
                            float e0 = ex2f(x[i][2 * t] - ref), e1 = ex2f(x[i][2 * t + 1] - ref);
                            const float both = kEight ? fmaf(e0, vinv[2 * t], e1 * vinv[2 * t + 1]) : e0 + e1;
                            sum[t / 2] = t % 2 ? sum[t / 2] + both : both;
                            if (kEight) {
                                e0 *= fv[2 * t];
                                e1 *= fv[2 * t + 1];
                            }
                            pa[t][i] = pack2<M>(e0, e1);
                        }
                        l[i] += SUB > 1 ? sum[0] + sum[SUB - 1] : sum[0];
                    }
                    // values of keys 2 q, 2 q + 1 (and + 8) of 16, head dims by g
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int j = 0; j < (KL > 2 ? 2 : 1); ++j) {  // blocks of 128 bytes
                            uint4 vr[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int key = 16 * u + 2 * q + (i & 1) + 8 * (i >> 1), row = kw * kKeys + key;
                                if (D * Cfg::ESIZE == 64) vr[i] = lds8(vs + row * 64 + (((g >> 1) ^ (row >> 1 & 3)) << 4) + (g & 1) * 8);
                                else vr[i] = lds16(vs + j * kStage * 128 + row * 128 + ((g ^ (row & 7)) << 4));
                                if (left < kKeys && key >= left) vr[i] = make_uint4(0, 0, 0, 0);  // (may be anything there)
                            }
                            constexpr int PER = kEight ? NE : 4;
#pragma unroll
                            for (int e = 0; e < PER; ++e) {
                                uint32_t a0, a1, a2, a3;
                                if (kEight) {
                                    const uint32_t sel = e % 2 ? 0x7362 : 0x5140;
                                    const uint32_t x0 = __byte_perm(part(vr[0], e / 2), part(vr[1], e / 2), sel);
                                    const uint32_t x1 = __byte_perm(part(vr[2], e / 2), part(vr[3], e / 2), sel);
                                    a0 = to_half2(x0);
                                    a1 = to_half2(x0 >> 16);
                                    a2 = to_half2(x1);
                                    a3 = to_half2(x1 >> 16);
                                } else {
                                    const uint32_t u0 = part(vr[0], e), u1 = part(vr[1], e), u2 = part(vr[2], e), u3 = part(vr[3], e);
                                    a0 = __byte_perm(u0, u1, 0x5410);
                                    a1 = __byte_perm(u0, u1, 0x7632);
                                    a2 = __byte_perm(u2, u3, 0x5410);
                                    a3 = __byte_perm(u2, u3, 0x7632);
                                }
#pragma unroll
                                for (int i = 0; i < NR; ++i) mma16816<M>(acc[i][PER * j + e], a0, a1, a2, a3, pa[2 * u][i], pa[2 * u + 1][i]);
                            }
                        }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
                if (++s == NST) {
                    s = 0;
                    par ^= 1;
                }
            }

            // ---- join the key warps: maxima and sums of all rows first, then the outputs, brought to the joint maximum,
            // of the upper two warps into the lower ones and of the second into the first.  Lane (g, q) holds the sums of row
            // g (+ 8 i), and dims of rows 2 q and 2 q + 1.
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
                if (q == 0) {
                    sm_m[kw * ROWS + g + 8 * i] = m[i];
                    sm_l[kw * ROWS + g + 8 * i] = l[i];
                }
            }
            sync();
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = 2 * q + c + 8 * i;
                    float mm = sm_m[r];
#pragma unroll
                    for (int k = 1; k < kKeyWarps; ++k) mm = fmaxf(mm, sm_m[k * ROWS + r]);
                    const float f = mm == -INFINITY ? 0.f : ex2f(sm_m[kw * ROWS + r] - mm);
#pragma unroll
                    for (int e = 0; e < NE; ++e) {
                        acc[i][e][c] *= f;
                        acc[i][e][2 + c] *= f;
                    }
                }
            auto slot_of = [&](int slot, int i, int c, int e) -> float2 * {
                const int dim = kEight ? D / 8 * g + 2 * e : 64 * (e / 4) + 8 * g + 2 * (e % 4);
                return reinterpret_cast<float2 *>(sm_o + (slot * ROWS + 2 * q + c + 8 * i) * Cfg::OS + dim);
            };
            auto put = [&](int slot) {
#pragma unroll
                for (int i = 0; i < NR; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < NE; ++e) *slot_of(slot, i, c, e) = make_float2(acc[i][e][c], acc[i][e][2 + c]);
            };
            auto add = [&](int slot) {
#pragma unroll
                for (int i = 0; i < NR; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < NE; ++e) {
                            const float2 y = *slot_of(slot, i, c, e);
                            acc[i][e][c] += y.x;
                            acc[i][e][2 + c] += y.y;
                        }
            };
            if (kw >= 2) put(kw - 2);
            sync();
            if (kw < 2) {
                add(kw);
                put(kw);
            }
            sync();
            const bool whole = w.begins() && w.ends();
            const int slot = w.begins() ? 1 : 0;
            if (!whole) {
                const int4 name = unit_name(w.n, x, w.t, w.ends() ? kEnds : kGoesOn);
                if (slot) named1 = name;
                else named0 = name;
            }
            for (int t = threadIdx.x; t < ROWS * (D / 8); t += Cfg::CONSUMERS) {
                const int r = t / (D / 8), c = t % (D / 8) * 8;
                const int tok = r / hb, ti = w.t * sched.tokens + tok, head = kvh * G + rb * ROWS + r - tok * hb;
                if (tok >= sched.tokens || ti >= w.u.m || rb * ROWS + r - tok * hb >= G) continue;
                float mm = sm_m[r], ll = 0.f, o[8];
#pragma unroll
                for (int k = 1; k < kKeyWarps; ++k) mm = fmaxf(mm, sm_m[k * ROWS + r]);
                const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
                for (int k = 0; k < kKeyWarps; ++k) ll = fmaf(ex2f(sm_m[k * ROWS + r] - ref), sm_l[k * ROWS + r], ll);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 y = *reinterpret_cast<const float2 *>(sm_o + r * Cfg::OS + c + e);
                    const float2 z = *reinterpret_cast<const float2 *>(sm_o + (ROWS + r) * Cfg::OS + c + e);
                    o[e] = y.x + z.x;
                    o[e + 1] = y.y + z.y;
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
                            lse_of(mm, ll);
                } else {
                    const int64_t row = (int64_t(side.me) * 2 + slot) * ROWS + r;
                    if (c == 0) a.part_ml[row] = make_float2(mm, ll);
                    float4 *dst = reinterpret_cast<float4 *>(a.part_o + row * D + c);
                    dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                    dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                }
            }
            sync();
        }
        if (threadIdx.x == 0) {
            a.rec[2 * side.me] = named0;
            a.rec[2 * side.me + 1] = named1;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) a.flags[side.me] = (*bad_page ? ATTN_DEV_INDEX_RANGE : 0u) | (*abort ? ATTN_DEV_TIMEOUT : 0u);
}

// Outputs of the units that several shares hold: a block for every share that may hold a unit's first piece, some of its
// rows (RPT a thread) and COLS columns, COLS / 4 lanes a row.  kGroups groups of lanes take every kGroups-th piece; a row's
// group sums are added in order.  Three round trips to L2: the records of the next shares side by side, the pieces'
// maxima and sums side by side, their outputs several at a time.  The first block gathers the call's status.
// (Rows of the tensor-core kernel: 32 or 64 a block, one wave of blocks; 8 a block, four waves, took 25 us behind 2048
// tokens on 32768 where this takes 19.)
template <class T, int D, int COLS, int RPT>
__global__ void __launch_bounds__(kJoin) paged_join_kernel(const __grid_constant__ PagedAttnArgs a, const PagedShape shape)
{
    constexpr int LPR = COLS / 4, kGroups = RPT > 1 ? 1 : kJoin / (8 * LPR), SLOTS = kJoin / LPR / kGroups, ROWS = SLOTS * RPT;
    constexpr int kBatch = kJoin / ROWS;  // pieces whose maxima and sums are fetched at once
    __shared__ float2 sm_ml[kBatch][ROWS];
    __shared__ float sm_l[kGroups][SLOTS];
    __shared__ float4 sm_o[kGroups][SLOTS][LPR];
    const int c0 = blockIdx.x, shares = shape.shares, rows = shape.rows, t = threadIdx.x, lane = t % 32;
    pdl_wait();
    if (c0 == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
        uint32_t flags = 0;
        for (int k = t; k < shares; k += kJoin) flags |= a.flags[k];
        const int range = __syncthreads_or(flags & ATTN_DEV_INDEX_RANGE), timeout = __syncthreads_or(flags & ATTN_DEV_TIMEOUT);
        if (t == 0) *a.status = (range ? ATTN_DEV_INDEX_RANGE : 0u) | (timeout ? ATTN_DEV_TIMEOUT : 0u);
    }
    // the shares that hold the rest: up to the one whose first piece ends the unit (every warp finds it for itself)
    const int4 name = a.rec[2 * c0 + 1];
    int next = c0 + 1 + lane < shares ? a.rec[2 * (c0 + 1 + lane)].w : kEnds;
    if (name.w == kNone) return;
    int end = c0 + 1;
    while (__ballot_sync(0xffffffffu, next == kEnds) == 0) {
        end += 32;
        next = end + lane < shares ? a.rec[2 * (end + lane)].w : kEnds;
    }
    end += __ffs(__ballot_sync(0xffffffffu, next == kEnds)) - 1;
    const int n = (end < shares ? end : shares - 1) - c0 + 1;  // pieces (a share in between may hold none)

    const int slot = t / LPR % SLOTS, grp = t / (SLOTS * LPR), col = blockIdx.z * COLS + t % LPR * 4, r0 = blockIdx.y * ROWS;
    const int64_t step = 2 * int64_t(rows);  // rows from a share's results to the next one's
    auto row_of = [&](int k, int r) { return (int64_t(c0) * 2 + (k == 0)) * rows + k * step + r0 + r; };
    auto fetch = [&](int k0, int here) {  // maxima and sums of pieces k0 ..
        const int k = t / ROWS, r = t % ROWS;
        if (k < here)
            sm_ml[k][r] = k0 + k > 0 && a.rec[2 * (c0 + k0 + k)].w == kNone ? make_float2(-INFINITY, 0.f) : a.part_ml[row_of(k0 + k, r)];
        __syncthreads();
    };
    float mm[RPT], ll[RPT];
    float4 o[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        mm[i] = -INFINITY;
        ll[i] = 0.f;
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int k0 = 0; k0 < n; k0 += kBatch) {
        const int here = n - k0 < kBatch ? n - k0 : kBatch;
        if (k0 > 0) __syncthreads();
        fetch(k0, here);
        for (int k = 0; k < here; ++k)
#pragma unroll
            for (int i = 0; i < RPT; ++i) mm[i] = fmaxf(mm[i], sm_ml[k][slot + i * SLOTS].x);
    }
    for (int k0 = 0; k0 < n; k0 += kBatch) {
        const int here = n - k0 < kBatch ? n - k0 : kBatch;
        if (n > kBatch) {
            __syncthreads();
            fetch(k0, here);
        }
#pragma unroll 4
        for (int k = grp; k < here; k += kGroups)
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = slot + i * SLOTS;
                const float2 x = sm_ml[k][r];
                const float f = x.y != x.y ? x.y : x.x == -INFINITY ? 0.f : ex2f(x.x - mm[i]);  // (NaN stays NaN)
                const float4 u = f == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                          : *reinterpret_cast<const float4 *>(a.part_o + row_of(k0 + k, r) * D + col);
                o[i].x = fmaf(f, u.x, o[i].x); o[i].y = fmaf(f, u.y, o[i].y);
                o[i].z = fmaf(f, u.z, o[i].z); o[i].w = fmaf(f, u.w, o[i].w);
                ll[i] = fmaf(f, x.y, ll[i]);
            }
    }
    if (kGroups > 1) {
        if (t % LPR == 0) sm_l[grp][slot] = ll[0];
        sm_o[grp][slot][t % LPR] = o[0];
        __syncthreads();
        if (grp > 0) return;
#pragma unroll
        for (int k = 1; k < kGroups; ++k) {
            const float4 u = sm_o[k][slot][t % LPR];
            o[0].x += u.x; o[0].y += u.y; o[0].z += u.z; o[0].w += u.w;
        }
        ll[0] = sm_l[0][slot];
#pragma unroll
        for (int k = 1; k < kGroups; ++k) ll[0] += sm_l[k][slot];
    }
    const int G = a.h / a.h_kv, kvh = name.y / shape.row_blocks, block = name.y - kvh * shape.row_blocks, group_rows = rows / shape.groups;
    bool none = false;
    int first, m;
    a.seqs.rows(name.x, &first, &m, &none);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = r0 + slot + i * SLOTS, g = r / group_rows, in = r - g * group_rows, tok = in / shape.heads;
        const int x = block * shape.heads + in - tok * shape.heads, head = kvh * G + x;
        const int ti = (name.z * shape.groups + g) * shape.tokens + tok;
        if (tok >= shape.tokens || ti >= m || x >= G) continue;
        const float inv = ll[i] == 0.f ? 0.f : 1.f / ll[i];
        T *dst = static_cast<T *>(a.o.ptr) + (a.seqs.cu ? int64_t(first + ti) * a.o.ss : name.x * a.o.sb + ti * a.o.ss) + head * a.o.sh;
        *reinterpret_cast<uint2 *>(dst + col) = make_uint2(pack2<T>(o[i].x * inv, o[i].y * inv), pack2<T>(o[i].z * inv, o[i].w * inv));
        if (a.lse && col == 0)
            a.lse[a.seqs.cu ? int64_t(head) * a.seqs.tokens + first + ti : (int64_t(name.x) * a.h + head) * a.seqs.s_q + ti] =
                lse_of(mm[i], ll[i]);
    }
}

// Pages [n_pages][h_kv][page][d] in boxes of up to `keys` tokens x `bytes` bytes, swizzled over that width or not.
bool tmap_boxes(CUtensorMap *m, void *ptr, const PagedCache &c, int d, int h_kv, int keys, int bytes, bool swizzle)
{
    auto enc = tmap_encoder();
    if (!enc) return false;
    const int page = 1 << c.shift, size = c.type == ATTN_E4M3 ? 1 : 2;
    cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(page), cuuint64_t(h_kv), cuuint64_t(c.none)};
    cuuint64_t strides[3] = {cuuint64_t(c.ss) * size, cuuint64_t(c.sh) * size, cuuint64_t(c.sp) * size};
    cuuint32_t box[4] = {cuuint32_t(bytes / size), cuuint32_t(page < keys ? page : keys), 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    return enc(m, type, 4, ptr, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               tmap_promotion(d * size), CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, bool kEight, int D, int ROWS> cudaError_t run(const PagedAttnArgs &a, const PagedShape &p, cudaStream_t s)
{
    using Cfg = DecodeCfg<D, kEight, ROWS>;
    DecodeParams prm;
    prm.a = a;
    if (!tmap_boxes(&prm.tm_k, a.cache.k, a.cache, D, a.h_kv, Cfg::STAGE_KEYS, 64, false) ||
        !tmap_boxes(&prm.tm_v, a.cache.v, a.cache, D, a.h_kv, Cfg::STAGE_KEYS, D * Cfg::ESIZE < 128 ? 64 : 128, true))
        return cudaErrorInvalidValue;
    auto k = paged_decode_kernel<T, kEight, D, ROWS>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    return launch_kernel(k, dim3(unsigned(p.shares)), dim3(Cfg::THREADS), Cfg::SMEM, s, false, prm);
}

template <class T, bool kEight, int D> cudaError_t pick_rows(const PagedAttnArgs &a, const PagedShape &p, cudaStream_t s)
{
    return p.rows == 16 ? run<T, kEight, D, 16>(a, p, s) : run<T, kEight, D, 8>(a, p, s);
}

template <class T, bool kEight> cudaError_t pick(const PagedAttnArgs &a, const PagedShape &p, cudaStream_t s)
{
    return a.d == 64 ? pick_rows<T, kEight, 64>(a, p, s) : pick_rows<T, kEight, 128>(a, p, s);
}

}  // namespace

PagedShape paged_decode_shape(int64_t h, int64_t h_kv, int64_t d, int64_t s_q, bool eight)
{
    const int group = int(h / h_kv);
    const int64_t rows = group * (s_q < 16 ? s_q : 16);
    PagedShape p;
    p.chunk = false;
    p.rows = rows > 8 ? 16 : 8;
    p.shares = kPagedCtas * decode_blocks(int(d), eight ? 1 : 2);
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

namespace {
template <class T, int D> cudaError_t join(const PagedAttnArgs &a, const PagedShape &p, cudaStream_t s)
{
    if (p.chunk) {
        constexpr int RPT = 4, ROWS = kJoin / (D / 4) * RPT;
        return launch_kernel(paged_join_kernel<T, D, D, RPT>, dim3(unsigned(p.shares), unsigned(p.rows / ROWS)), dim3(kJoin), 0, s, true,
                             a, p);
    }
    // (many blocks for the few rows of the small kernel, whose units may have hundreds of pieces)
    return launch_kernel(paged_join_kernel<T, D, 32, 1>, dim3(unsigned(p.shares), unsigned(p.rows / 8), unsigned(D / 32)), dim3(kJoin), 0,
                         s, true, a, p);
}
}  // namespace

cudaError_t launch_paged_join(const PagedAttnArgs &a, const PagedShape &p, cudaStream_t s)
{
    if (a.d == 64) return a.dtype == ATTN_F16 ? join<__half, 64>(a, p, s) : join<__nv_bfloat16, 64>(a, p, s);
    return a.dtype == ATTN_F16 ? join<__half, 128>(a, p, s) : join<__nv_bfloat16, 128>(a, p, s);
}

}  // namespace attn
