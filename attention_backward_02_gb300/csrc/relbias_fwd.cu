// relbias_fwd.cu -- tensor-core forward of attention with a learned relative
// position bias, in training mode (O and the fp32 log-sum-exp stats), for
// sm_103a: tcgen05 MMAs with TMEM accumulators, TMA tile loads.
//
//   s_ij = scale q_i.k_j + table[bucket(j - i - shift)][head],  O = softmax(s) V
//
// Persistent, one CTA an SM; a unit is (sequence, query head, 256 queries), dealt
// longest first, in alternating direction.  Query rows are the MMA M dimension and
// the TMEM lanes:
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
// Bound: the chain S -> softmax -> P -> O of a group, about 1700 cycles for 64 keys
// and 256 rows against 1280 of MMAs.  Persistent because a CTA's start, first loads,
// last products and the gap to the next one took 15 000 cycles (of 75 000 a unit at
// b2 h32 s4096 d128 causal): the loads and first S of the next unit now run under the
// end of this one (251 -> 239 us, with the MMA thread's and the rows' integer work
// cut down; 0.60 of the measured tensor peak).  256 rows a unit
// because K / V tiles read for 128 rows came near what L2 delivers (279 us).  Where
// that leaves SMs idle (kSplit; split_rule below), a unit is 128 queries and the
// groups take the first and last 64 keys of every key tile; they meet at its end,
// when the two O are added, scaled to one maximum.
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
// rounded to the 16-bit type for the second product, whose operands are of that type,
// after its sum l is taken.  A row that sees no key has O = 0 and LSE = +inf.
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
#include <algorithm>
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
    static_assert(3 + 2 * NSK + 2 * NSV + 12 <= 32, "barrier slots");
};

struct RelFwdParams {
    CUtensorMap tm_q, tm_k, tm_v;
    DenseArgs a;
    RelArgs rel;
    int64_t units;
};

namespace {

template <class Geo> struct IsPackedGeo : std::false_type {};
template <> struct IsPackedGeo<PackedGeo> : std::true_type {};

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// mbar_wait out of line, for the MMA thread: its waits are nearly always over when it comes.
__device__ __noinline__ bool mbar_wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return mbar_wait(bar, parity, abort);
}

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
    uint64_t *q_full = bars + 0, *q_empty = bars + 1, *drain = bars + 2;
    uint64_t *k_full = bars + 3, *k_empty = k_full + NSK, *v_full = k_empty + NSK, *v_empty = v_full + NSV;
    uint64_t *s_full = v_empty + NSV;      // [2 groups][2 buffers] S is written
    uint64_t *p_full = s_full + 4;         // [2 groups][2 buffers] P is written (and O rescaled if needed)
    uint64_t *o_prev = s_full + 8;         // [2 groups] O += P V of a unit's last step but one has completed ...
    uint64_t *o_last = s_full + 10;        // [2 groups] ... and of its last step
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + Cfg::OFF_MISC + 8);
    const DenseArgs &a = p.a;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    // ---- a unit: (sequence b, query head hq, queries i0 .. i0 + ROWS - 1)
    constexpr int ROWS = kSplit ? BM : 2 * BM;
    const int64_t G = a.h / a.h_kv;
    struct Unit {
        int64_t b, hq, g, lq, lkv, q_row0, kv_row0, i0;
        int q_b;
        int steps0, steps1;  // steps of the groups
        int n_steps, n_kt;   // the longer of the two, and the key tiles they span
    };
    // this CTA's unit of round r into u; false behind the last one
    auto next_unit = [&](int64_t &r, Unit &u) -> bool {
        for (;; ++r) {
            const int64_t k = r * gridDim.x + ((r & 1) ? int64_t(gridDim.x) - 1 - blockIdx.x : int64_t(blockIdx.x));
            if (r * gridDim.x >= p.units) return false;
            if (k >= p.units) continue;
            int64_t qt;
            if (!kPacked) {
                const int64_t nu = (geo.q_len(0) + ROWS - 1) / ROWS, per = a.h * geo.nseq;
                qt = (nu - 1 - k / per) * (ROWS / BM);
                const int64_t rest = k - (k / per) * per;
                u.b = rest / a.h;
                u.hq = rest - u.b * a.h;
            } else {  // 128-row tiles of the packed workspace rows, each sequence's last tile first
                const int64_t tile = k / a.h;
                u.hq = k - tile * a.h;
                int64_t i0w = 0;
                geo.ws_locate(tile * BM, &u.b, &i0w);
                const int64_t nqt = (geo.q_len(u.b) + BM - 1) / BM;
                qt = nqt - 1 - i0w / BM;
                if (!kSplit && (qt & 1)) continue;  // goes with tile qt - 1
            }
            u.g = u.hq / G;
            u.lq = geo.q_len(u.b);
            u.lkv = geo.kv_len(u.b);
            u.q_row0 = kPacked ? geo.q_start(u.b) : 0;
            u.kv_row0 = kPacked ? geo.kv_start(u.b) : 0;
            u.q_b = kPacked ? 0 : int(u.b);
            u.i0 = qt * BM;
            // keys that any of the query rows first .. first + BM - 1 sees
            auto keys_seen = [&](int64_t first) -> int64_t {
                if (first >= u.lq || u.lkv <= 0) return 0;
                const int64_t last = first + BM - 1 < u.lq - 1 ? first + BM - 1 : u.lq - 1;
                const int64_t n = last_visible_key(a.mask, last, u.lq, u.lkv) + 1;
                return n > 0 ? n : 0;
            };
            const int64_t seen0 = keys_seen(u.i0), seen1 = kSplit ? seen0 : keys_seen(u.i0 + BM);
            u.steps0 = int((seen0 + (kSplit ? BN : HN) - 1) / (kSplit ? BN : HN));
            u.steps1 = int((seen1 + (kSplit ? BN : HN) - 1) / (kSplit ? BN : HN));
            u.n_steps = u.steps1 > u.steps0 ? u.steps1 : u.steps0;
            u.n_kt = kSplit ? u.n_steps : (u.n_steps + 1) / 2;
            return true;
        }
    };
    auto tile_of = [](int j) { return kSplit ? j : j >> 1; };               // key tile of a step
    auto half_of = [](int j, int grp) { return kSplit ? grp : j & 1; };     // and which half of it

    if (threadIdx.x == 0) {
        *abort = 0;
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
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
        for (int k = 0; k < 2; ++k) {
            mbar_init(&o_prev[k], 1);
            mbar_init(&o_last[k], 1);
        }
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
        if ((warp == 0 || warp == 2) && elect_one()) {
            // ============================================= TMA producers: Q and K (warp 0), V (warp 2)
            const bool isk = warp == 0;
            const int nst = isk ? NSK : NSV;
            uint64_t *full = isk ? k_full : v_full, *empty = isk ? k_empty : v_empty;
            const CUtensorMap *tm = isk ? &p.tm_k : &p.tm_v;
            prefetch_tmap(tm);
            if (isk) prefetch_tmap(&p.tm_q);
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (ok && !(ok = mbar_wait(bar, parity, abort))) flag_abort(abort, a.status);
            };
            uint32_t n_tile = 0, n_unit = 0;  // key tiles and units with keys so far
            Unit u;
            for (int64_t r = 0; ok && next_unit(r, u); ++r) {
                if (u.n_steps == 0) continue;
                if (isk) {
                    if (n_unit > 0) wait(q_empty, (n_unit - 1) & 1);
                    if (!ok) break;
                    const int n = !kSplit && u.steps1 ? 2 : 1;
                    ++n_unit;
                    mbar_arrive_expect_tx(q_full, n * Cfg::TILE_BYTES);
                    for (int k = 0; k < n; ++k)
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_4d(sQ + k * Cfg::TILE_BYTES + c * BM * 128, &p.tm_q, q_full, c * 64,
                                        int(u.q_row0 + u.i0 + k * BM), int(u.hq), u.q_b);
                }
                for (int j = 0; j < u.n_kt; ++j) {
                    const uint32_t s = n_tile % nst, use = n_tile / nst;
                    if (use > 0) wait(&empty[s], (use - 1) & 1);
                    if (!ok) break;
                    ++n_tile;
                    mbar_arrive_expect_tx(&full[s], Cfg::TILE_BYTES);
                    uint8_t *dst = isk ? sK(s) : sV(s);
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_4d(dst + c * BN * 128, tm, &full[s], c * 64, int(u.kv_row0 + j * BN), int(u.g), u.q_b);
                }
            }
            if (!ok) {  // let every copy this thread started land before the CTA exits
                volatile int never = 0;
                if (isk && n_unit > 0) mbar_wait(q_full, (n_unit - 1) & 1, &never, 100000000ull);
                for (uint32_t j = n_tile > uint32_t(nst) ? n_tile - nst : 0; j < n_tile; ++j)
                    mbar_wait(&full[j % nst], (j / nst) & 1, &never, 100000000ull);
            }
        } else if (warp == 1 && elect_one()) {
            // ============================================= MMA issuer
            // One thread, and the time it takes between two MMAs is the tensor pipe's to lose: descriptors are
            // one add from values kept in registers, a unit starts at buffer 0 so that buffers and halves are
            // constants of the (two-step) loop body, and phases are bits that flip with each wait.
            constexpr uint32_t idS = idesc_f16(128, HN, kType, 0, 0);
            constexpr uint32_t idO = idesc_f16(128, D, kType, 0, 1);
            constexpr uint32_t STAGE = Cfg::TILE_BYTES / 16;  // a ring stage, in descriptor units
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (ok && !mbar_test_wait(bar, parity) && !(ok = mbar_wait_slow(bar, parity, abort))) flag_abort(abort, a.status);
                tc_fence_after();
            };
            const uint64_t kQ = desc_kmaj(smem_u32(sQ), BM, 0), kK = desc_kmaj(smem_u32(sK(0)), BN, 0);
            const uint64_t mV = desc_mn(smem_u32(sV(0)), BN, 0);
            uint32_t ks = 0, vs = 0, k_par = 0, v_par = 0, q_par = 0, p_par = 0;  // p_par: bit 2 group + buffer
            Unit u;
            for (int64_t r = 0; next_unit(r, u); ++r) {
                if (u.n_steps == 0) continue;
                wait(q_full, q_par);
                q_par ^= 1;
                const int n_steps = u.n_steps, steps0 = u.steps0, steps1 = u.steps1;
                // S of step j, then O += P V of step j - 1 (buffer sb ^ 1).  S of step j goes where P of step
                // j - 2 was, whose product was issued a round ago
                auto round = [&](int j, auto sb_tag) {
                    constexpr int sb = decltype(sb_tag)::value, xb = sb ^ 1;
                    if (j < n_steps) {
                        if (kSplit || sb == 0) wait(&k_full[ks], k_par);
                        if (ok) {
#pragma unroll
                            for (int grp = 0; grp < 2; ++grp) {
                                if (j >= (grp ? steps1 : steps0)) continue;
                                const uint64_t dk = kK + ks * STAGE + (kSplit ? grp : sb) * (HN * 128 / 16);
                                const uint64_t dq = kQ + (kSplit ? 0 : grp * STAGE);
#pragma unroll
                                for (int kk = 0; kk < D / 16; ++kk)
                                    mma_f16_ss(tmem + Cfg::T_S + grp * 128 + sb * 64, kmaj_step(dq, BM, kk), kmaj_step(dk, BN, kk), idS,
                                               kk > 0);
                                mma_commit(&s_full[grp * 2 + sb]);
                            }
                        }
                        if (kSplit || sb || j == n_steps - 1) {  // the last S that reads this K stage
                            if (ok) mma_commit(&k_empty[ks]);
                            if (++ks == NSK) {
                                ks = 0;
                                k_par ^= 1;
                            }
                            if (ok && j == n_steps - 1) mma_commit(q_empty);
                        }
                    }
                    if (j > 0) {
                        const int x = j - 1;
                        if (kSplit || xb == 0) wait(&v_full[vs], v_par);
#pragma unroll
                        for (int grp = 0; grp < 2; ++grp) {
                            const int steps = grp ? steps1 : steps0;
                            if (x >= steps) continue;
                            wait(&p_full[grp * 2 + xb], p_par >> (grp * 2 + xb) & 1);
                            p_par ^= 1u << (grp * 2 + xb);
                            if (ok) {
                                const uint64_t dv = mV + vs * STAGE + (kSplit ? grp : xb) * (HN / 16) * 128;
#pragma unroll
                                for (int kk = 0; kk < HN / 16; ++kk)
                                    mma_f16_ts(tmem + Cfg::T_O + grp * D, tmem + Cfg::T_S + grp * 128 + xb * 64 + kk * 8,
                                               mn_step(dv, kk), idO, x > 0 || kk > 0);
                                // (earlier ones are behind S of step x + 2)
                                if (x >= steps - 2) mma_commit(x == steps - 1 ? &o_last[grp] : &o_prev[grp]);
                            }
                        }
                        if (kSplit || xb || x == n_steps - 1) {
                            if (ok) mma_commit(&v_empty[vs]);
                            if (++vs == NSV) {
                                vs = 0;
                                v_par ^= 1;
                            }
                        }
                    }
                };
                for (int j = 0; j <= n_steps; j += 2) {
                    round(j, std::integral_constant<int, 0>{});
                    if (j < n_steps) round(j + 1, std::integral_constant<int, 1>{});
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
        const float c = a.scale * kLog2e;
        const uint32_t tO = tmem + lane_addr + Cfg::T_O + grp * D;
        float *win = reinterpret_cast<float *>(smem + Cfg::OFF_WIN) + grp * 512;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok && !(ok = mbar_wait(bar, parity, abort))) flag_abort(abort, a.status);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        };
        // key tiles, and phases of o_prev and o_last before this unit; phase parity of the S buffers
        uint32_t k_base = 0, n_prev = 0, n_last = 0, s_par = 0;
        pdl_wait();  // the bias has been expanded

        Unit u;
        for (int64_t round = 0; next_unit(round, u); ++round) {
        const int steps = grp ? u.steps1 : u.steps0;
        const int64_t first_row = u.i0 + (kSplit ? 0 : grp * BM);
        const int64_t i = first_row + r;  // query position in the sequence
        // Positions in 32 bits, relative to the unit (sequence lengths fit): step j's first key is kfirst + j kstep, of
        // which this row sees those up to kmax; its window starts at delta dfirst + j kstep.
        constexpr int kstep = kSplit ? BN : HN;
        const int kfirst = kSplit ? grp * HN : 0;
        const int kmax = u.lkv > 0 && i < u.lq ? int(last_visible_key(a.mask, i, u.lq, u.lkv)) : -1;
        const int dfirst = kfirst - int(first_row + (a.mask == ATTN_CAUSAL_BOTTOM_RIGHT ? u.lkv - u.lq : 0)) - 127;
        const int dlo = p.rel.b.lo - (HN + 126), dhi = p.rel.b.hi;  // near: dlo < first delta < dhi
        float m_ref = -INFINITY;
        float2 l2 = make_float2(0.f, 0.f);
        const float *rel = p.rel.rel + u.hq * p.rel.stride;
        const float *rel_wt = rel + (kRelPad - p.rel.b.lo) + wt;  // this thread's entry of the window at delta 0
        auto window = [&](int d) -> float2 {  // its two entries of the window at delta d
            return d > dlo && d < dhi ? make_float2(__ldcg(rel_wt + d), __ldcg(rel_wt + d + 128)) : make_float2(0.f, 0.f);
        };
        const float past = __ldcg(rel), future = __ldcg(rel + p.rel.stride - 1);
        named_bar_sync(1 + grp, 128);  // the last unit's windows have been read
        if (steps > 0) {
            const float2 w = window(dfirst);
            win[wt] = w.x;
            win[wt + 128] = w.y;
        }
        named_bar_sync(1 + grp, 128);

        for (int j = 0; j < steps; ++j) {
            const int sb = j & 1;
            const uint32_t tS = tmem + lane_addr + Cfg::T_S + grp * 128 + sb * 64;
            const int d = dfirst + j * kstep;
            const bool near = d > dlo && d < dhi;
            const bool next_near = j + 1 < steps && d + kstep > dlo && d + kstep < dhi;
            const float2 next_win = next_near ? window(d + kstep) : make_float2(0.f, 0.f);
            const int lim = kmax - kfirst - j * kstep;  // columns <= lim are visible
            const bool whole = __all_sync(0xffffffffu, lim >= HN - 1);
            wait(&s_full[grp * 2 + sb], s_par >> sb & 1);
            s_par ^= 1u << sb;
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
                if (near) {
                    const float *w = win + sb * 256 - r + 127;
#pragma unroll
                    for (int e = 0; e < HN; e += 2) {
                        const float2 y = fma2(make_float2(__uint_as_float(v[e / 32][e % 32]), __uint_as_float(v[e / 32][e % 32 + 1])),
                                              c2, make_float2(w[e], w[e + 1]));
                        x[e] = y.x;
                        x[e + 1] = y.y;
                    }
                } else {
                    const float b1 = d <= dlo ? past : future;
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
                    for (int k = 0; k < 4; ++k) mq[k] = max3(mq[k], x[e + 2 * k], x[e + 2 * k + 1]);
                mx = fmaxf(max3(mq[0], mq[1], mq[2]), mq[3]);
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
                if (j > 0) {  // O holds earlier tiles: scale this row once their GEMMs have completed, which S of
                              // the next step, issued behind the last of them, shows
                    if (j + 1 < steps) wait(&s_full[grp * 2 + (sb ^ 1)], s_par >> (sb ^ 1) & 1);
                    else wait(&o_prev[grp], n_prev & 1);
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
                if (kPacked && kfirst + j * kstep + HN > int(u.lkv)) {  // values of the next sequence
                    const uint32_t tl = k_base + tile_of(j), s = tl % NSV;
                    wait(&v_full[s], (tl / NSV) & 1);
                    const int row = half_of(j, grp) * HN + r;  // of the tile
                    if (r < HN && kfirst + j * kstep + r >= int(u.lkv))
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
        // (neither barrier gets to its next phase before every warp that waits here is through: the next unit's
        // products wait for their P)
        if (steps > 0) {
            wait(&o_last[grp], n_last & 1);
            if (kSplit) wait(&o_last[grp ^ 1], n_last & 1);
            ++n_last;
        }
        if (steps > 1) ++n_prev;
        const bool row_ok = i < u.lq;
        const float inv = l == 0.f ? 0.f : 1.f / l;  // (NaN stays NaN)
        T *O = static_cast<T *>(a.o.ptr) + (kPacked ? 0 : int64_t(u.q_b) * a.o.sb) + u.hq * a.o.sh +
               (u.q_row0 + i) * a.o.ss;
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
            const float lse = l == 0.f ? INFINITY : (m + __log2f(l)) / kLog2e;
            const int64_t idx = kPacked ? u.hq * a.t_q + u.q_row0 + i : (int64_t(u.q_b) * a.h + u.hq) * u.lq + i;
            a.lse_out[idx] = lse;
        }
        k_base += u.n_kt;
        // the next unit's first product overwrites O once this group's P of it is there, which is behind these
        // reads; with kSplit the other group's reads too
        if (kSplit) named_bar_sync(3, 256);
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

// Units of 128 queries, the keys of a tile split between the groups, or of 256?  A step of either takes about the
// same time (split a little more), and what lies around a unit that of 3 to 5 steps, so the estimate of each is the
// longest sum of a CTA's units as they are dealt.  Measured (us, split / whole, causal: c): d = 64, h12: b1 s1024 14.0
// / 20.7; b2 s1024 25.5 / 20.9, c 15.4 / 20.9; b4 s1024 35.4 / 39.3; b8 s1024 c 45.6 / 38.2; b1 h5 s4096 c 34.7 / 59.9.
// d = 128: b1 h16 s1024 c 16.3 / 22.9; b4 h12 s1024 c 32.1 / 27.0; b8 h32 s333 50.8 / 42.5; b2 h32 s4096 c 297 / 239.
// Packed batches, and batches of more units than are worth adding up: whole where there are tiles for every SM four
// times over.
template <int D, int BM, int BN, class Geo> bool split_rule(const DenseArgs &a, const Geo &g, int64_t tiles, int64_t sms)
{
    constexpr int64_t kMaxCtas = 512;
    if (IsPackedGeo<Geo>::value || tiles > 4096 || sms > kMaxCtas) return tiles < 4 * sms;
    const int64_t lq = g.q_len(0), lkv = g.kv_len(0), per = a.h * a.nseq;
    float est[2];
    for (int whole = 0; whole < 2; ++whole) {
        const int64_t rows = whole ? 2 * BM : BM, keys = whole ? BN / 2 : BN, n = (lq + rows - 1) / rows;
        const int64_t ctas = n * per < sms ? n * per : sms;
        float load[kMaxCtas] = {};
        int64_t u = 0;
        for (int64_t k = n - 1; k >= 0; --k) {
            const int64_t last = (k + 1) * rows - 1 < lq - 1 ? (k + 1) * rows - 1 : lq - 1;
            const int64_t seen = lkv > 0 ? last_visible_key(a.mask, last, lq, lkv) + 1 : 0;
            const float steps = seen > 0 ? float((seen + keys - 1) / keys) : 0.f;
            const float cost = whole ? steps + (D == 64 ? 3.f : 4.f) : 1.05f * steps + (D == 64 ? 3.5f : 5.f);
            for (int64_t x = 0; x < per; ++x, ++u) load[(u / ctas) & 1 ? ctas - 1 - u % ctas : u % ctas] += cost;
        }
        est[whole] = *std::max_element(load, load + ctas);
    }
    return est[0] < est[1];
}

template <class T, int D, class Geo> cudaError_t run(const DenseArgs &a, const RelArgs &rel, const Geo &g, cudaStream_t s)
{
    using Cfg = RelFwdCfg<D>;
    constexpr bool packed = IsPackedGeo<Geo>::value;
    const int64_t tiles = packed ? (g.ws_rows() / Cfg::BM) * a.h : (g.q_len(0) + Cfg::BM - 1) / Cfg::BM * a.h * a.nseq;
    const int64_t sms = sm_count();
    const bool split = split_rule<D, Cfg::BM, Cfg::BN>(a, g, tiles, sms);
    // packed: a unit for every 128-row tile, of which every other one is passed over
    const int64_t units = split || packed ? tiles : (g.q_len(0) + 2 * Cfg::BM - 1) / (2 * Cfg::BM) * a.h * a.nseq;
    if (units == 0) return cudaSuccess;
    if (units > INT32_MAX) return cudaErrorInvalidValue;
    RelFwdParams prm;
    prm.a = a;
    prm.rel = rel;
    prm.units = units;
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
    const int64_t ctas = units < sms ? units : sms;
    return launch_kernel(k, dim3(unsigned(ctas)), dim3(Cfg::THREADS), Cfg::SMEM_ALLOC, s, true, prm, g);
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
