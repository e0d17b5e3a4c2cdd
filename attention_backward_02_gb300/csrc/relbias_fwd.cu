// relbias_fwd.cu -- tensor-core forward of attention with a learned relative
// position bias, in training mode (O and the fp32 log-sum-exp stats), for
// sm_103a: tcgen05 MMAs with TMEM accumulators, TMA tile loads.
//
//   s_ij = scale q_i.k_j + table[bucket(j - i - shift)][head],  O = softmax(s) V
//
// One CTA per (sequence, query head, 256 queries), longest first.  Query rows are
// the MMA M dimension and the TMEM lanes:
//   S = Q K^T      M=128 (queries) N=64 (keys) K=D   A=Q (smem, K-major) B=K (smem, K-major)
//   O += P V       M=128           N=D         K=64  A=P (TMEM, 16-bit)  B=V (smem, MN-major)
//
// Two softmax warpgroups work beside each other, each on 128 query rows of its own
// and 64 keys a step, with its own S, running maximum, sum and O accumulator; the
// MMAs of one run under the softmax of the other.  A thread owns a row: no exchange
// of row maxima between warps.  Each group has two S buffers of 64 columns, so S of
// the next step is ready when the softmax of this one ends (S with 64 columns an MMA
// runs at two thirds of the tensor rate, which costs less than the wait it removes).
// P overwrites the S it came from (each thread its own row, after it has read it);
// TMEM holds S 4 x 64 + O 2 x D columns.  The tensor pipe runs the MMAs in the order
// they were issued, so S of step j + 2 follows O += P V of step j into the same
// columns without a wait.
//
// Bound: the chain S -> softmax -> P -> O of a group.  256 rows a CTA because with
// 128 the K / V tiles' reads from L2 bound it (8 TB/s; taking away the exponentials,
// the MMAs or the maxima changed nothing): b2 h32 s4096 d128 causal bf16 279 us with
// 128 rows, FWD_LONG with 256.  Where 128-row tiles do not fill the SMs once (kSplit),
// a CTA has 128 rows and the groups take the first and last 64 keys of every key
// tile; they meet at the end, when the two O are added, scaled to one maximum
// (SPLIT_NOTE).
//
// The bias of a group's tile is a window of the head's expanded table (log2
// units), element (row r, column c) entry c - r + 127.  A warpgroup loads its next
// tile's window while it works on the current one and reads it without bank
// conflicts, consecutive rows consecutive entries; a tile that lies in one end
// bucket whole takes its bias from a register, folded into the scaling.  The row
// arithmetic is done on pairs (fma.rn.f32x2 and the like).
//
// A row's reference maximum m is raised only when a tile's maximum exceeds it by
// more than 8 (log2 units), and then l and the row of O in TMEM are scaled by
// exp2(m_old - m_new): P = exp2(x - m) <= 2^8 fits both 16-bit types.  P is
// rounded to the 16-bit type for the second product, after its sum l is taken.  A
// row that sees no key has O = 0 and LSE = +inf.
//
// Packed sequences: the last key tile may run into the next sequence, whose values
// meet P = 0; they are set to zero in shared memory first, so that an infinity or
// NaN there does not get into this sequence's O.
//
// Roles (12 warps): warp 0 issues the TMA loads of Q and K, warp 2 those of V,
// warp 1 the MMAs, warps 4..7 and 8..11 are the two softmax warpgroups (warp 3 is
// idle: a warp reads the TMEM lanes of its place in its warpgroup).  Every
// barrier wait is bounded; a wait that runs out sets ATTN_DEV_TIMEOUT and the CTA
// skips the rest of its work, drains its copies and MMAs, and frees its TMEM.
#include <climits>
#include <type_traits>

#include "relbias.h"
#include "sm103.cuh"
#include "tc_util.cuh"
#include "tmap.h"

namespace attn {
using namespace sm103;
using namespace tc;

template <int D> struct RelFwdCfg {
    static constexpr int BM = 128, BN = 128;
    static constexpr int NSK = D == 64 ? 4 : 2;      // K ring stages
    static constexpr int NSV = D == 64 ? 4 : 2;      // V ring stages
    static constexpr int THREADS = 384;
    static constexpr int TILE_BYTES = BN * D * 2;    // a K or V tile, and 128 query rows
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * TILE_BYTES;
    static constexpr int OFF_V = OFF_K + NSK * TILE_BYTES;
    static constexpr int OFF_BAR = OFF_V + NSV * TILE_BYTES;
    static constexpr int OFF_MISC = OFF_BAR + 32 * 8;
    static constexpr int OFF_ML = OFF_MISC + 64;              // [2 groups][m, l][128 rows] floats
    static constexpr int HN = BN / 2;                         // key columns of a step
    static constexpr int OFF_WIN = OFF_ML + 2 * 2 * 128 * 4;  // [2 groups][2 tiles][256] floats
    static constexpr int SMEM = OFF_WIN + 2 * 2 * 256 * 4;
    // at least half the SM's shared memory: one CTA, which holds all of the TMEM, runs per SM
    static constexpr int SMEM_ALLOC = SMEM + 1024 > 116 * 1024 ? SMEM + 1024 : 116 * 1024;
    static constexpr int T_S = 0, T_O = 256;  // S (and P) of group g, step parity b at T_S + 128 g + 64 b, O at T_O + D g
    static constexpr int T_COLS = 512;
    static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");
    static_assert(2 + 2 * NSK + 2 * NSV + 10 <= 32, "barrier slots");
};

struct RelFwdParams {
    CUtensorMap tm_q, tm_k, tm_v;
    DenseArgs a;
    RelArgs rel;
};

namespace {

template <class Geo> struct IsPackedGeo : std::false_type {};
template <> struct IsPackedGeo<PackedGeo> : std::true_type {};

}  // namespace

template <class T, int D, class Geo, bool kSplit>
__global__ void __launch_bounds__(RelFwdCfg<D>::THREADS, 1)
    relbias_fwd_kernel(const __grid_constant__ RelFwdParams p, const Geo geo)
{
    using Cfg = RelFwdCfg<D>;
    constexpr int BM = Cfg::BM, BN = Cfg::BN, HN = Cfg::HN, NSK = Cfg::NSK, NSV = Cfg::NSV;
    constexpr bool kPacked = IsPackedGeo<Geo>::value;
    constexpr int kType = std::is_same<T, __half>::value ? 0 : 1;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_BAR);
    uint64_t *q_full = bars + 0, *drain = bars + 1;
    uint64_t *k_full = bars + 2, *k_empty = k_full + NSK, *v_full = k_empty + NSK, *v_empty = v_full + NSV;
    uint64_t *s_full = v_empty + NSV;      // [2 groups][2 buffers] S is written
    uint64_t *p_full = s_full + 4;         // [2 groups][2 buffers] P is written (and O rescaled if needed)
    uint64_t *o_done = s_full + 8;         // [2 groups] O += P V has completed
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + Cfg::OFF_MISC + 8);
    const DenseArgs &a = p.a;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    // ---- the unit: (sequence b, query head hq, query tile qt, or the two tiles qt and qt + 1), longest first
    constexpr int ROWS = kSplit ? BM : 2 * BM;
    int64_t b, hq, qt;
    {
        const int64_t u = blockIdx.x;
        if (!kPacked) {
            const int64_t nu = (geo.q_len(0) + ROWS - 1) / ROWS, per = a.h * geo.nseq;
            qt = (nu - 1 - u / per) * (ROWS / BM);
            const int64_t rest = u - (u / per) * per;
            b = rest / a.h;
            hq = rest - b * a.h;
        } else {  // 128-row tiles of the packed workspace rows, each sequence's last tile first
            const int64_t tile = u / a.h;
            hq = u - tile * a.h;
            int64_t i0w = 0;
            geo.ws_locate(tile * BM, &b, &i0w);
            const int64_t nqt = (geo.q_len(b) + BM - 1) / BM;
            qt = nqt - 1 - i0w / BM;
            if (!kSplit && (qt & 1)) return;  // the CTA of tile qt - 1 has it
        }
    }
    const int64_t G = a.h / a.h_kv, g = hq / G;
    const int64_t lq = geo.q_len(b), lkv = geo.kv_len(b);
    const int64_t q_row0 = kPacked ? geo.q_start(b) : 0, kv_row0 = kPacked ? geo.kv_start(b) : 0;
    const int q_b = kPacked ? 0 : int(b);
    const int64_t i0 = qt * BM;
    // keys that any of the query rows first .. first + BM - 1 sees
    auto keys_seen = [&](int64_t first) -> int64_t {
        if (first >= lq || lkv <= 0) return 0;
        const int64_t last = first + BM - 1 < lq - 1 ? first + BM - 1 : lq - 1;
        return last_visible_key(a.mask, last, lq, lkv) + 1;
    };
    // steps of the two groups, and the key tiles they span (the second group's rows see at least the first's keys)
    const int64_t seen0 = keys_seen(i0), seen1 = kSplit || i0 + BM >= lq ? seen0 : keys_seen(i0 + BM);
    const int n_kt = seen1 <= 0 ? 0 : int((seen1 + BN - 1) / BN);
    const int steps0 = kSplit ? n_kt : (seen0 <= 0 ? 0 : int((seen0 + HN - 1) / HN));
    const int steps1 = kSplit ? n_kt : (i0 + BM >= lq || seen1 <= 0 ? 0 : int((seen1 + HN - 1) / HN));
    const int n_steps = steps1 > steps0 ? steps1 : steps0;
    auto tile_of = [](int j) { return kSplit ? j : j >> 1; };               // key tile of a step
    auto half_of = [](int j, int grp) { return kSplit ? grp : j & 1; };     // and which half of it

    if (threadIdx.x == 0) {
        *abort = 0;
        mbar_init(q_full, 1);
        mbar_init(drain, 1);
        for (int s = 0; s < NSK; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < NSV; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int k = 0; k < 4; ++k) {
            mbar_init(&s_full[k], 1);
            mbar_init(&p_full[k], 4);
        }
        mbar_init(&o_done[0], 1);
        mbar_init(&o_done[1], 1);
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, Cfg::T_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint8_t *sQ = smem + Cfg::OFF_Q;
    auto sK = [&](int s) { return smem + Cfg::OFF_K + s * Cfg::TILE_BYTES; };
    auto sV = [&](int s) { return smem + Cfg::OFF_V + s * Cfg::TILE_BYTES; };

    if (warp < 4) {
        if ((warp == 0 || warp == 2) && elect_one() && n_kt > 0) {
            // ============================================= TMA producers: Q and K (warp 0), V (warp 2)
            const bool isk = warp == 0;
            const int nst = isk ? NSK : NSV;
            uint64_t *full = isk ? k_full : v_full, *empty = isk ? k_empty : v_empty;
            const CUtensorMap *tm = isk ? &p.tm_k : &p.tm_v;
            prefetch_tmap(tm);
            bool ok = true;
            int armed = 0;
            if (isk) {
                prefetch_tmap(&p.tm_q);
                mbar_arrive_expect_tx(q_full, (steps1 && !kSplit ? 2 : 1) * Cfg::TILE_BYTES);
                for (int k = 0; k < (steps1 && !kSplit ? 2 : 1); ++k)
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_4d(sQ + k * Cfg::TILE_BYTES + c * BM * 128, &p.tm_q, q_full, c * 64,
                                    int(q_row0 + i0 + k * BM), int(hq), q_b);
            }
            for (int j = 0; j < n_kt; ++j) {
                const int s = j % nst, use = j / nst;
                if (use > 0 && ok && !(ok = mbar_wait(&empty[s], uint32_t(use - 1) & 1, abort)))
                    flag_abort(abort, a.status);
                if (!ok) break;
                armed = j + 1;
                mbar_arrive_expect_tx(&full[s], Cfg::TILE_BYTES);
                uint8_t *dst = isk ? sK(s) : sV(s);
                for (int c = 0; c < D / 64; ++c)
                    tma_load_4d(dst + c * BN * 128, tm, &full[s], c * 64, int(kv_row0 + j * BN), int(g), q_b);
            }
            // let every copy this thread started land before the CTA exits
            volatile int never = 0;
            if (isk) mbar_wait(q_full, 0, &never, 100000000ull);
            for (int j = armed - nst; j < armed; ++j)
                if (j >= 0) mbar_wait(&full[j % nst], uint32_t(j / nst) & 1, &never, 100000000ull);
        } else if (warp == 1 && elect_one() && n_kt > 0) {
            // ============================================= MMA issuer
            constexpr uint32_t idS = idesc_f16(128, HN, kType, 0, 0);
            constexpr uint32_t idO = idesc_f16(128, D, kType, 0, 1);
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (ok && !(ok = mbar_wait(bar, parity, abort))) flag_abort(abort, a.status);
                tc_fence_after();
            };
            wait(q_full, 0);
            // S of step j, then O += P V of step j - 1.  S of step j goes where P of step j - 2 was, whose
            // product was issued a round ago
            for (int j = 0; j <= n_steps; ++j) {
                if (j < n_steps) {
                    const int tl = tile_of(j), s = tl % NSK;
                    if (kSplit || (j & 1) == 0) wait(&k_full[s], uint32_t(tl / NSK) & 1);
                    if (ok) {
                        const uint64_t kK = desc_kmaj(smem_u32(sK(s)), BN, 0);
#pragma unroll
                        for (int grp = 0; grp < 2; ++grp) {
                            if (j >= (grp ? steps1 : steps0)) continue;
                            const uint64_t kQ = desc_kmaj(smem_u32(sQ + (kSplit ? 0 : grp * Cfg::TILE_BYTES)), BM, 0);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                mma_f16_ss(tmem + Cfg::T_S + grp * 128 + (j & 1) * 64, kmaj_step(kQ, BM, kk),
                                           kmaj_step(kK + uint64_t(half_of(j, grp) * HN * 128 / 16), BN, kk), idS, kk > 0);
                            mma_commit(&s_full[grp * 2 + (j & 1)]);
                        }
                        // the last S that reads this K stage
                        if (kSplit || (j & 1) || j == n_steps - 1) mma_commit(&k_empty[s]);
                    }
                }
                if (j > 0) {
                    const int x = j - 1, tl = tile_of(x), s = tl % NSV, sb = x & 1;
                    if (kSplit || (x & 1) == 0) wait(&v_full[s], uint32_t(tl / NSV) & 1);
                    const uint64_t mV = desc_mn(smem_u32(sV(s)), BN, 0);
#pragma unroll
                    for (int grp = 0; grp < 2; ++grp) {
                        if (x >= (grp ? steps1 : steps0)) continue;
                        wait(&p_full[grp * 2 + sb], uint32_t(x >> 1) & 1);
                        if (ok) {
#pragma unroll
                            for (int kk = 0; kk < HN / 16; ++kk)
                                mma_f16_ts(tmem + Cfg::T_O + grp * D, tmem + Cfg::T_S + grp * 128 + sb * 64 + kk * 8,
                                           mn_step(mV, half_of(x, grp) * (HN / 16) + kk), idO, x > 0 || kk > 0);
                            mma_commit(&o_done[grp]);
                        }
                    }
                    if (ok && (kSplit || (x & 1) || x == n_steps - 1)) mma_commit(&v_empty[s]);
                }
            }
            volatile int never = 0;
            mma_commit(drain);
            mbar_wait(drain, 0, &never, 100000000ull);
        }
    } else {
        // ================================================= softmax and epilogue (warps 4..11)
        const int grp = (warp >> 2) - 1, qd = warp & 3;  // the group; TMEM lane quadrant
        const uint32_t lane_addr = uint32_t(qd * 32) << 16;
        const int r = qd * 32 + lane, wt = threadIdx.x & 127;
        const int steps = grp ? steps1 : steps0;
        const int64_t first_row = i0 + (kSplit ? 0 : grp * BM);
        const int64_t i = first_row + r;  // query position in the sequence
        const float c = a.scale * kLog2e;
        const int64_t kmax = lkv > 0 && i < lq ? last_visible_key(a.mask, i, lq, lkv) : -1;  // last key it sees
        const uint32_t tO = tmem + lane_addr + Cfg::T_O + grp * D;
        float m_ref = -INFINITY;
        float2 l2 = make_float2(0.f, 0.f);
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok && !(ok = mbar_wait(bar, parity, abort))) flag_abort(abort, a.status);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        };
        // the window of step j, whose first key is key0(j), starts at delta key0(j) - row0; this thread's two
        // entries of it
        float *win = reinterpret_cast<float *>(smem + Cfg::OFF_WIN) + grp * 512;
        auto key0 = [&](int j) { return int64_t(tile_of(j)) * BN + half_of(j, grp) * HN; };
        const int64_t row0 = first_row + (a.mask == ATTN_CAUSAL_BOTTOM_RIGHT ? lkv - lq : 0) + 127;
        auto kind_of = [&](int j) { return rel_tile(p.rel.b, key0(j) - row0, HN + 127); };
        const float *rel = p.rel.rel + hq * p.rel.stride;
        auto window = [&](int j) -> float2 {
            if (kind_of(j) != kRelNear) return make_float2(0.f, 0.f);
            const float *w = rel + (key0(j) - row0 - (p.rel.b.lo - kRelPad)) + wt;
            return make_float2(__ldcg(w), __ldcg(w + 128));
        };
        pdl_wait();  // the bias has been expanded
        const float past = __ldcg(rel), future = __ldcg(rel + p.rel.stride - 1);
        if (steps > 0) {
            const float2 w = window(0);
            win[wt] = w.x;
            win[wt + 128] = w.y;
        }
        named_bar_sync(1 + grp, 128);

        for (int j = 0; j < steps; ++j) {
            const int sb = j & 1;
            const uint32_t tS = tmem + lane_addr + Cfg::T_S + grp * 128 + sb * 64;
            const RelTile kind = kind_of(j);
            const bool next_near = j + 1 < steps && kind_of(j + 1) == kRelNear;
            const float2 next_win = next_near ? window(j + 1) : make_float2(0.f, 0.f);
            const int64_t lim64 = kmax - key0(j);  // columns <= lim are visible
            const int lim = int(lim64 < -1 ? -1 : (lim64 > HN ? HN : lim64));
            const bool whole = __all_sync(0xffffffffu, lim >= HN - 1);
            wait(&s_full[grp * 2 + sb], uint32_t(j >> 1) & 1);
            // the row of S in log2 units, with its bias and masked, and its maximum
            float x[HN];
            float mx = -INFINITY;
            if (ok) {
                uint32_t v[2][32];
                tmem_ld32(tS, v[0]);
                tmem_ld32(tS + 32, v[1]);
                tmem_ld_wait_regs(v[0]);
                tmem_ld_wait_regs(v[1]);
                const float2 c2 = make_float2(c, c);
                if (kind == kRelNear) {
                    const float *w = win + sb * 256 - r + 127;
#pragma unroll
                    for (int e = 0; e < HN; e += 2) {
                        const float2 y = fma2(make_float2(__uint_as_float(v[e / 32][e % 32]), __uint_as_float(v[e / 32][e % 32 + 1])),
                                              c2, make_float2(w[e], w[e + 1]));
                        x[e] = y.x;
                        x[e + 1] = y.y;
                    }
                } else {
                    const float b1 = kind == kRelPast ? past : future;
                    const float2 b2 = make_float2(b1, b1);
#pragma unroll
                    for (int e = 0; e < HN; e += 2) {
                        const float2 y = fma2(make_float2(__uint_as_float(v[e / 32][e % 32]), __uint_as_float(v[e / 32][e % 32 + 1])),
                                              c2, b2);
                        x[e] = y.x;
                        x[e + 1] = y.y;
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int e = 0; e < HN; ++e) x[e] = e <= lim ? x[e] : -INFINITY;
                }
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < HN; e += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) mq[k] = fmaxf(mq[k], fmaxf(x[e + 2 * k], x[e + 2 * k + 1]));
                mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
            }
            if (next_near) {  // the other buffer was last read a tile ago, before that tile's barrier
                win[(sb ^ 1) * 256 + wt] = next_win.x;
                win[(sb ^ 1) * 256 + wt + 128] = next_win.y;
                named_bar_sync(1 + grp, 128);
            }
            const float m_new = fmaxf(m_ref, mx);
            const bool need = m_new > m_ref + 8.f;  // also the first finite max
            if (__any_sync(0xffffffffu, need)) {
                const float f = need ? ex2(m_ref - m_new) : 1.f;  // exp2(-inf) = 0 on the first raise
                if (j > 0) {  // O holds earlier tiles: scale this row once their GEMMs have completed
                    wait(&o_done[grp], uint32_t(j - 1) & 1);
                    if (ok) {
#pragma unroll 1
                        for (int o0 = 0; o0 < D; o0 += 32) {
                            uint32_t v[32];
                            tmem_ld32(tO + o0, v);
                            tmem_ld_wait_regs(v);
#pragma unroll
                            for (int e0 = 0; e0 < 32; e0 += 8) {
                                uint32_t w[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(__uint_as_float(v[e0 + e]) * f);
                                tmem_st8(tO + o0 + e0, w);
                            }
                        }
                        tmem_st_wait();
                    }
                }
                if (need) {
                    l2.x *= f;
                    l2.y *= f;
                    m_ref = m_new;
                }
            }
            // P = exp2(x - m) over the columns S was read from
            if (ok) {
                const float neg = m_ref == -INFINITY ? 0.f : -m_ref;  // no visible key yet: every P is 0
                const float2 neg2 = make_float2(neg, neg);
#pragma unroll
                for (int e0 = 0; e0 < HN; e0 += 16) {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 y = add2(make_float2(x[e0 + e], x[e0 + e + 1]), neg2);
                        const float2 q = make_float2(ex2(y.x), ex2(y.y));
                        l2 = add2(l2, q);
                        w[e / 2] = pack2<T>(q.x, q.y);
                    }
                    tmem_st8(tS + e0 / 2, w);
                }
                tmem_st_wait();
                if (kPacked && key0(j) + HN > lkv) {  // values of the next sequence
                    const int tl = tile_of(j), s = tl % NSV;
                    wait(&v_full[s], uint32_t(tl / NSV) & 1);
                    const int row = half_of(j, grp) * HN + r;  // of the tile
                    if (r < HN && key0(j) + r >= lkv)
                        for (int q = 0; q < D / 64; ++q)
                            for (int e = 0; e < 8; ++e)
                                st_shared_v4(smem_u32(sV(s)) + q * BN * 128 + row * 128 + e * 16, 0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[grp * 2 + sb]);
        }
        // ---- epilogue: O / l (16 bit, row per thread) and LSE; kSplit: the groups' maxima and sums first, and each
        // group writes half of the columns of both
        float m = m_ref, l = l2.x + l2.y, fa = 1.f, fb = 0.f;
        if (kSplit) {
            float *ml = reinterpret_cast<float *>(smem + Cfg::OFF_ML);
            ml[grp * 256 + r] = m_ref;
            ml[grp * 256 + 128 + r] = l;
            named_bar_sync(3, 256);
            const float ma = ml[r], mb = ml[256 + r];
            m = fmaxf(ma, mb);
            fa = ma == -INFINITY ? 0.f : ex2(ma - m);
            fb = mb == -INFINITY ? 0.f : ex2(mb - m);
            l = fa * ml[128 + r] + fb * ml[256 + 128 + r];
        }
        if (n_kt > 0 && (kSplit || steps > 0)) {
            wait(&o_done[grp], uint32_t(steps - 1) & 1);
            if (kSplit) wait(&o_done[grp ^ 1], uint32_t(steps - 1) & 1);
        }
        const bool row_ok = i < lq;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        T *O = static_cast<T *>(a.o.ptr) + (kPacked ? 0 : int64_t(q_b) * a.o.sb) + hq * a.o.sh + (q_row0 + i) * a.o.ss;
        const uint32_t tOa = tmem + lane_addr + Cfg::T_O + (kSplit ? 0 : grp * D);
#pragma unroll 1
        for (int o0 = kSplit ? grp * (D / 2) : 0; o0 < (kSplit ? (grp + 1) * (D / 2) : D); o0 += 32) {
            uint32_t va[32], vb[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) va[e] = vb[e] = 0u;
            if (ok && steps > 0) {
                tmem_ld32(tOa + o0, va);
                if (kSplit) tmem_ld32(tOa + D + o0, vb);
                tmem_ld_wait_regs(va);
                if (kSplit) tmem_ld_wait_regs(vb);
            }
            if (row_ok) {
                const float ga = fa * inv, gb = fb * inv;
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    float y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        y[k] = __uint_as_float(va[e + k]) * ga;
                        if (kSplit) y[k] = fmaf(__uint_as_float(vb[e + k]), gb, y[k]);
                    }
                    *reinterpret_cast<uint4 *>(O + o0 + e) =
                        make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
                }
            }
        }
        if (row_ok && (!kSplit || grp == 0)) {
            const float lse = l > 0.f ? (m + __log2f(l)) / kLog2e : INFINITY;
            const int64_t idx = kPacked ? hq * a.t_q + q_row0 + i : (int64_t(q_b) * a.h + hq) * lq + i;
            a.lse_out[idx] = lse;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::T_COLS);
    }
}

// ===================================================================== host

namespace {

int64_t sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 1;
    return n > 0 ? n : 1;
}

template <class T, int D, class Geo> cudaError_t run(const DenseArgs &a, const RelArgs &rel, const Geo &g, cudaStream_t s)
{
    using Cfg = RelFwdCfg<D>;
    constexpr bool packed = IsPackedGeo<Geo>::value;
    const int64_t tiles = packed ? (g.ws_rows() / Cfg::BM) * a.h : (g.q_len(0) + Cfg::BM - 1) / Cfg::BM * a.h * a.nseq;
    const bool split = tiles <= sm_count();
    // packed: a CTA for every 128-row tile, of which every other one ends at once
    const int64_t units = split || packed ? tiles : (g.q_len(0) + 2 * Cfg::BM - 1) / (2 * Cfg::BM) * a.h * a.nseq;
    if (units == 0) return cudaSuccess;
    if (units > INT32_MAX) return cudaErrorInvalidValue;
    RelFwdParams prm;
    prm.a = a;
    prm.rel = rel;
    const int64_t nb = packed ? 1 : a.nseq;
    const int64_t sq = packed ? a.t_q : g.q_len(0), skv = packed ? a.t_kv : g.kv_len(0);
    if (!tmap_view16(&prm.tm_q, a.q, a.dtype, D, sq, a.h, nb, Cfg::BM)) return cudaErrorInvalidValue;
    if (skv > 0) {
        if (!tmap_view16(&prm.tm_k, a.k, a.dtype, D, skv, a.h_kv, nb, Cfg::BN) ||
            !tmap_view16(&prm.tm_v, a.v, a.dtype, D, skv, a.h_kv, nb, Cfg::BN))
            return cudaErrorInvalidValue;
    } else {
        prm.tm_k = prm.tm_v = prm.tm_q;  // never read: no key tiles
    }
    auto k = split ? relbias_fwd_kernel<T, D, Geo, true> : relbias_fwd_kernel<T, D, Geo, false>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    // starts beside the kernel that expands the table (and clears the status word); the softmax warps wait for it
    return launch_kernel(k, dim3(unsigned(units)), dim3(Cfg::THREADS), Cfg::SMEM_ALLOC, s, true, prm, g);
}

template <class Geo> cudaError_t pick(const DenseArgs &a, const RelArgs &rel, const Geo &g, cudaStream_t s)
{
    if (a.d == 64)
        return a.dtype == ATTN_F16 ? run<__half, 64>(a, rel, g, s) : run<__nv_bfloat16, 64>(a, rel, g, s);
    return a.dtype == ATTN_F16 ? run<__half, 128>(a, rel, g, s) : run<__nv_bfloat16, 128>(a, rel, g, s);
}

}  // namespace

cudaError_t launch_relbias_fwd(const DenseArgs &a, const RelArgs &rel, const FixedGeo &g, cudaStream_t s) { return pick(a, rel, g, s); }
cudaError_t launch_relbias_fwd(const DenseArgs &a, const RelArgs &rel, const PackedGeo &g, cudaStream_t s) { return pick(a, rel, g, s); }

}  // namespace attn
