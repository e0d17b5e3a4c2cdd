// bwd_tc.cu -- tensor-core SDPA backward for sm_103a (tcgen05 + TMA + TMEM).
//
// FlashAttention-2 backward (cuDNN-frontend sample
// "51_scaled_dot_product_attention_backward": backward from the saved
// (B,H,S,1) stats, no stored P), with the gradient formulas of the Ascend page
// "aclnnNsaSelectedAttentionGrad", Function / Formula (dV = P^T dY,
// dQ = dS K scale, dK = dS^T Q scale).
//
// One CTA owns a tile of BN = 128 key/value rows of one (sequence, kv head)
// and walks every (query head of the group, query tile of BM rows) that sees
// it.  Everything is computed transposed, so the 128 key rows are the MMA M
// dimension and the TMEM lanes:
//   S^T  = K Q^T           M=128 (keys) N=BM  K=D    A=K  (smem, K-major) B=Q  (K-major)
//   dP^T = V dO^T          M=128        N=BM  K=D    A=V  (smem, K-major) B=dO (K-major)
//   P^T  = exp2(S^T scale log2 e - LSE log2 e),  dS^T = P^T (dP^T - D)   (CUDA cores)
//   dV  += P^T dO          M=128        N=D   K=BM   A=P^T (TMEM, 16-bit)   B=dO (MN-major)
//   dK  += dS^T Q          M=128        N=D   K=BM   A=dS^T (smem, K-major) B=Q  (MN-major)
//   dQ   = dS K     (D=64) M=BM=128     N=64  K=128  A=dS (MN-major)       B=K  (MN-major)
//   dQ^T = K^T dS^T (D=128) M=D=128     N=BM=64 K=128 A=K^T (MN-major)     B=dS^T (MN-major)
// dV, dK stay in TMEM for the whole key tile and are written once; each dQ
// tile is read out of TMEM, staged in shared memory half a tile at a time and
// added into the fp32 accumulator with a TMA reduce-add; a kernel chained
// behind this one converts the accumulator into dQ.  Bitwise reproducible dQ
// either way: split (n_part partial buffers, each with one chain of key tiles
// adding in a fixed order) or ordered (one buffer; the adds into a query tile
// go in decreasing key-tile order, each waiting on a per-tile counter in the
// workspace).  TMEM: S^T BM + dP^T BM + P^T BM/2 + dV D + dK D + dQ 64 columns
// (512 at D = 64, 480 at D = 128).
//
// Pipeline.  The MMA warp issues S/dP of query tile i and then dV/dK/dQ of
// tile i-1, so the tensor cores run tile i-1's three GEMMs while the softmax
// warps turn tile i's S/dP into P/dS.  Two 32 KB shared buffers alternate
// per query tile: tile i writes its dS into one while tile i-1's GEMMs read
// their dS from the other.  P (16-bit, packed) waits in registers until tile
// i-1's dV GEMM has released the P columns of TMEM.  At d = 128 the softmax
// warps copy S^T / dP^T into registers and release them before computing, so
// tile i+1's S/dP GEMMs run during tile i's element-wise work.  Q, dO and the
// LSE / D vectors stream through a 3-stage ring.  Fixed-length batches take
// their work units in a longest-first order planned on the host.
//
// Roles (14 warps): warp 0 issues TMA loads, warp 1 the MMAs, warps 2..9 do
// the element-wise work (warp w reads TMEM lanes 32 (w % 4) .. + 31; the two
// warps on the same lanes split the columns), warps 10..13 the dQ staging and
// the dK / dV epilogue.  The ordered dQ mode adds warp 14, which publishes the
// per-tile add counts.
//
// Causal masking: query tiles entirely before the first query that sees the
// key tile are skipped; the rest are masked per element when needed.  Key
// rows past the sequence end are masked by row; query rows past it have
// LSE = +inf in the workspace and so P = 0.
//
// Relative position bias (kBias): the bias of a tile is a window of the head's
// expanded bias (log2 units), element (key row r, query column c) entry r - c +
// const; the window rides in the Q / dO ring stage, and beside it a window of
// bucket codes.  The gradient of the bias table is the sum of dS over each bucket,
// taken from the fp32 dS before it is rounded (P and dS are computed in fp32 for
// both types here, two columns an instruction).  A warp works on blocks of 32 key
// rows x 32 query columns, whose 63 deltas are consecutive.  A block in one bucket
// takes its bias from a register and adds its dS to one running sum a thread.
// Otherwise the block is summed along its diagonals, the sums of even and of odd
// columns each passed two lanes up per pair of columns (one packed add for both;
// one lane up per column took 797 us where this takes 790 at b2 h32 s4096 d128
// causal); then runs of diagonals of one bucket are added up and the runs
// added to the warp's row of buckets in shared memory, both behind the arrival that
// lets the tile's GEMMs go.  The causal mask is in the expanded bias (-inf), so a
// tile on the diagonal runs the same code as its neighbours: the P / dS loop's copies
// compete for the instruction cache (790 -> 758 us; a third copy for blocks of two
// buckets, without shuffles, cost 50).  Element masks remain where a tile passes the
// end of a sequence.  At those sizes 767 us against 751 without a bias; 75 / 53 at b4
// h12 s1024 d64 without a mask.  Each warp stores its row once per (key tile, head); a
// kernel behind this one adds them up in a fixed order, so the table's gradient is
// bitwise reproducible in every dQ mode.  Packed sequences: rows of a tile that
// belong to the next sequence are set to zero in shared memory before the GEMMs
// that would multiply them by P = dS = 0, so that no infinity or NaN crosses over.
//
// With few kv heads and many queries each the units are too large to spread evenly:
// the query heads of a group are then shared out among several units (kBias, shares;
// to the kernel, shares x h_kv kv heads), whose dK and dV go as fp32 into the
// workspace and are added in order by the kernel behind this one.
//
// Every barrier wait is bounded (about a second).  On a timeout the thread
// sets ATTN_DEV_TIMEOUT in the status word and an abort flag in shared
// memory; from then on every wait of the CTA fails fast and all work is
// skipped while the control flow (and so every named barrier) stays the same;
// the CTA drains its in-flight copies and MMAs, frees its TMEM and exits.
#include <algorithm>
#include <climits>
#include <queue>
#include <type_traits>
#include <utility>
#include <vector>

#include "plan.h"
#include "relbias.h"
#include "sm103.cuh"
#include "tc_util.cuh"
#include "tmap.h"

namespace attn {
using namespace sm103;

template <int D>
struct TcCfg {
    static constexpr int BN = 128;                  // key rows per CTA tile
    static constexpr int BM = D == 64 ? 128 : 64;   // query rows per iteration
    static constexpr int NG = D == 64 ? 2 : 1;      // column groups of 32 per softmax thread
#ifndef ATTN_SDP_RELEASE_GROUPS
    static constexpr int NH = NG;                   // groups of S^T / dP^T columns released one by one
#else
    static constexpr int NH = ATTN_SDP_RELEASE_GROUPS;
#endif
    static constexpr int NST = 3;                   // Q / dO ring stages
#ifndef ATTN_SOFTMAX_WARPS
    static constexpr int NSW = 8;                   // P / dS warps (two or four per TMEM lane quadrant)
#else
    static constexpr int NSW = ATTN_SOFTMAX_WARPS;
#endif
    static constexpr int THREADS = 32 * (2 + NSW + 4);  // TMA, MMA, P / dS, dQ + dK / dV
    static constexpr int KV_BYTES = BN * D * 2;
    static constexpr int Q_BYTES = BM * D * 2;
    static constexpr int DS_BYTES = BN * BM * 2;
    static constexpr int X_BYTES = DS_BYTES;
    static constexpr int DQS_BYTES = BM * D * 2;             // fp32 dQ, half of the columns
    static constexpr int DQ_BOX_ROWS = D == 64 ? BM : 32;    // rows of one dQ reduce box (32 fp32 wide)
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = OFF_K + KV_BYTES;
    static constexpr int OFF_Q = OFF_V + KV_BYTES;            // NST stages
    static constexpr int OFF_DO = OFF_Q + NST * Q_BYTES;      // NST stages
    static constexpr int OFF_X = OFF_DO + NST * Q_BYTES;      // 2 dS buffers
    static constexpr int OFF_DQS = OFF_X + 2 * X_BYTES;       // dQ staging, half a tile
    static constexpr int OFF_LSE = OFF_DQS + DQS_BYTES;       // NST x BM floats
    static constexpr int OFF_DVEC = OFF_LSE + NST * BM * 4;   // NST x BM floats
    static constexpr int OFF_BAR = OFF_DVEC + NST * BM * 4;
    static constexpr int OFF_MISC = OFF_BAR + 32 * 8;
    static constexpr int SMEM = OFF_MISC + 64;
    static constexpr int SMEM_ALLOC = SMEM + 1024;            // room to align the base to 1024
    // kBias, behind the rest: the ring stages' windows of bias and bucket codes (the window's start is rounded
    // down to 16 bytes), each P / dS warp's bucket sums, and its finished diagonals
    static constexpr int WIN_BYTES = (BN + BM + 4) * 4;
    static constexpr int OFF_WIN = SMEM;                      // NST x (bias, codes)
    static constexpr int OFF_HIST = OFF_WIN + NST * 2 * WIN_BYTES;
    static constexpr int OFF_DIAG = OFF_HIST + NSW * kRelCodes * 4;
    static constexpr int SMEM_ALLOC_BIAS = OFF_DIAG + NSW * 32 * 8 + 1024;
    static_assert(WIN_BYTES % 16 == 0 && SMEM % 16 == 0 && SMEM_ALLOC_BIAS <= 227 * 1024, "shared memory budget");
    static_assert(kRelPad >= BN + BM + 4, "a near tile's window lies within the expanded bias");
    static constexpr int T_S = 0, T_DP = BM, T_P = 2 * BM, T_DV = 2 * BM + BM / 2, T_DK = T_DV + D,
                         T_DQ = T_DK + D;
    static constexpr int T_COLS = 512;
    static_assert(T_DQ + 64 <= T_COLS, "TMEM budget");
    static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");
    static constexpr int GW = BM / NG / (NSW / 4);  // query columns per P / dS thread and column group
    static_assert(GW % 16 == 0 && (NSW == 8 || NSW == 16), "P / dS work split");
    static_assert(NH == 1 || NH == NG, "release groups");
};

// Work units of each CTA, chosen on the host (see plan_units).  on = 0: the CTAs
// take the units in snake order instead.
constexpr int kSchedCtas = 160;
constexpr int kMailbox = 4;  // ordered dQ mode: counters in flight from the dQ leader to the publishing warp
constexpr int kSchedUnits = 4096;
struct TcSched {
    int32_t on;
    uint16_t off[kSchedCtas + 1];  // CTA c takes unit[off[c]] .. unit[off[c + 1] - 1], in this order
    uint16_t unit[kSchedUnits];
};

struct TcParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_do, tm_dq, tm_dk, tm_dv;
    DenseArgs a;
    TcSched sched;
    RelArgs rel;  // kBias
};

using namespace tc;

namespace {

// Query tiles that see the key tile starting at j0: [qt0, qt0 + nq).
template <int BM>
__device__ __forceinline__ void query_tiles(int mask, int64_t j0, int64_t lq, int64_t lkv, int *qt0, int *nq)
{
    const int64_t i_lo = first_query_seeing(mask, j0, lq, lkv);
    if (lq <= 0 || lkv <= 0 || i_lo >= lq) {
        *qt0 = 0;
        *nq = 0;
        return;
    }
    *qt0 = int(i_lo / BM);
    *nq = int((lq + BM - 1) / BM) - *qt0;
}

// Unit this CTA takes in its round r, or -1 once it has none left.
__device__ __forceinline__ int64_t cta_unit(const TcParams &p, int64_t r)
{
    if (p.sched.on) {
        const int k = int(p.sched.off[blockIdx.x]) + int(r);
        return k < int(p.sched.off[blockIdx.x + 1]) ? int64_t(p.sched.unit[k]) : -1;
    }
    const int64_t u = r * gridDim.x + ((r & 1) ? int64_t(gridDim.x) - 1 - blockIdx.x : int64_t(blockIdx.x));
    return u < p.a.tc_units ? u : -1;
}

template <class Geo> struct IsPacked : std::false_type {};
template <> struct IsPacked<PackedGeo> : std::true_type {};

}  // namespace

// kOrdered: ordered dQ mode (one accumulator, each query tile's adds in a fixed order; needs the planned
// unit order and a cooperative launch).  kBias: a relative position bias in the scores, and its gradient.
// Template parameters, so the other modes carry none of their code.
template <class T, int D, class Geo, bool kOrdered, bool kBias>
__global__ void __launch_bounds__(TcCfg<D>::THREADS + (kOrdered ? 32 : 0), 1)
    dense_bwd_tc_kernel(const __grid_constant__ TcParams p, const Geo geo)
{
    using Cfg = TcCfg<D>;
    constexpr int BM = Cfg::BM, BN = Cfg::BN, NST = Cfg::NST, NH = Cfg::NH, NG = Cfg::NG;
    constexpr int GW = Cfg::GW;      // query columns per softmax thread and column group
    constexpr bool kPacked = IsPacked<Geo>::value;
    constexpr int kType = std::is_same<T, __half>::value ? 0 : 1;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_BAR);
    uint64_t *kv_full = bars + 0, *kv_empty = bars + 1, *q_full = bars + 2, *q_empty = bars + 2 + NST;
    uint64_t *s_full = bars + 2 + 2 * NST;   // [NH] S^T / dP^T column group written
    uint64_t *s_free = s_full + 2;           // [NH] column group read out by the softmax warps
    uint64_t *p_ready = s_full + 4;          // P^T in TMEM and dS^T in shared memory
    uint64_t *p_free = s_full + 5;           // the dV GEMM has read P^T
    uint64_t *mma_done = s_full + 6;         // all GEMMs of a query tile have completed
    uint64_t *dq_free = s_full + 7;          // the dQ accumulator has been read out
    uint64_t *ds_free = s_full + 8;          // [2] dS buffer: the GEMMs that read it have completed
    uint64_t *acc_free = s_full + 10;        // the dK / dV accumulators have been read out
    uint64_t *drain = s_full + 11;
    // ordered dQ mode: counters handed from the dQ leader to the warp that publishes them
    uint64_t *mb_full = s_full + 12, *mb_empty = s_full + 12 + kMailbox;  // [kMailbox]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + Cfg::OFF_MISC + 8);
    uint32_t **mailbox = reinterpret_cast<uint32_t **>(smem + Cfg::OFF_MISC + 16);  // [kMailbox]
    const DenseArgs &a = p.a;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        *abort = 0;
        mbar_init(kv_full, 1);
        mbar_init(kv_empty, 1);
        for (int s = 0; s < NST; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
        }
        for (int q = 0; q < NH; ++q) {
            mbar_init(&s_full[q], 1);
            mbar_init(&s_free[q], Cfg::NSW);
        }
        mbar_init(p_ready, Cfg::NSW);
        mbar_init(p_free, 1);
        mbar_init(mma_done, 1);
        mbar_init(dq_free, 4);
        mbar_init(&ds_free[0], 1);
        mbar_init(&ds_free[1], 1);
        mbar_init(acc_free, 4);
        mbar_init(drain, 1);
        if (kOrdered)
            for (int k = 0; k < kMailbox; ++k) {
                mbar_init(&mb_full[k], 1);
                mbar_init(&mb_empty[k], 1);
            }
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, Cfg::T_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The preprocess (LSE, D, zeroed dQ accumulator) may still be running: only the loads of
    // LSE / D and the dQ reduce-adds wait for it (pdl_wait below), the Q / K / V / dO loads do not.

    // ---- work units: (sequence b, kv head g) and its key tiles; unit
    // index = first tile * (nseq * h_kv) + (b * h_kv + g).  Each CTA takes
    // the units the host planned for it (cta_unit).
    const int64_t nheads = a.nseq * a.h_kv;
    const int64_t tile_step = a.deterministic ? a.n_part : INT64_MAX / 2;
    const int G = int(a.h / a.h_kv);
    const int shares = kBias ? p.rel.shares : 1;  // units of a (key tile, kv head); a.h_kv counts them
#define ATTN_FOR_EACH_UNIT                                                                                    \
    for (int64_t round_ = 0;; ++round_) {                                                                     \
        const int64_t unit = cta_unit(p, round_);                                                             \
        if (unit < 0) break;                                                                                  \
        /* 32-bit divisions: the unit count fits (checked at launch) */                                       \
        const uint32_t ft_ = uint32_t(unit) / uint32_t(nheads), bg_ = uint32_t(unit) - ft_ * uint32_t(nheads);  \
        const uint32_t b_ = bg_ / uint32_t(a.h_kv);                                                           \
        const int64_t bg = bg_, first_tile = ft_;                                                             \
        const int64_t b = b_, g = int64_t(bg_ - b_ * uint32_t(a.h_kv));                                       \
        const int64_t part = a.deterministic ? first_tile : 0;                                                \
        const int64_t lq = geo.q_len(b), lkv = geo.kv_len(b);                                                 \
        const int64_t ntiles = (lkv + BN - 1) / BN;                                                           \
        const int q_b = kPacked ? 0 : int(b), kv_b = q_b;                                                     \
        const int64_t q_row0 = kPacked ? geo.q_start(b) : 0, kv_row0 = kPacked ? geo.kv_start(b) : 0;         \
        (void)part;                                                                                           \
        (void)bg;                                                                                             \
        (void)g;                                                                                              \
        (void)kv_b;                                                                                           \
        (void)q_row0;                                                                                         \
        (void)kv_row0;
#define ATTN_END_UNITS }

    uint8_t *sK = smem + Cfg::OFF_K, *sV = smem + Cfg::OFF_V, *sX = smem + Cfg::OFF_X;
    // kBias: entry of the expanded bias at which the window of a tile whose first delta is dmin starts; of a tile
    // in one end bucket whole, a place in the pad where every entry is that bucket's
    // (32 bits: sequence lengths fit)
    auto window_start = [&](int dmin) -> int {
        const int lo = p.rel.b.lo;
        return dmin <= lo - (BN + BM - 2) ? 0 : dmin >= p.rel.b.hi ? int(p.rel.stride) - Cfg::WIN_BYTES / 4 : dmin - lo + kRelPad;
    };

    if (warp == 0) {
        // ================================================= TMA producer
        if (elect_one()) {
            prefetch_tmap(&p.tm_q); prefetch_tmap(&p.tm_k); prefetch_tmap(&p.tm_v); prefetch_tmap(&p.tm_do);
            bool ok = true, pre_done = false;
            int64_t kt = 0, qi = 0, q_armed = 0, kv_armed = 0;  // loads started (for the drain below)
            ATTN_FOR_EACH_UNIT
            for (int64_t jt = first_tile; jt < ntiles; jt += tile_step) {
                const int64_t j0 = jt * BN;
                int qt0, nq;
                query_tiles<BM>(a.mask, j0, lq, lkv, &qt0, &nq);
                const int n_iter = G * nq;
                if (n_iter == 0) continue;
                // Q / dO of query tile `it` (global iteration index x) into its ring stage
                auto load_q = [&](int it, int64_t x) {
                    const int st = int(x % NST);
                    const int64_t use = x / NST;
                    if (use > 0 && ok && !(ok = mbar_wait(&q_empty[st], uint32_t(use - 1) & 1, abort)))
                        flag_abort(abort, a.status);
                    // the CTA's first tile gets its inputs before the rest of the ring is filled: every
                    // CTA starts by loading at once, and the later stages would compete for the memory
                    if (x == 1 && ok && !(ok = mbar_wait(&q_full[0], 0, abort))) flag_abort(abort, a.status);
                    if (!ok) return;
                    const int64_t hq = g * G + it / nq, i0 = int64_t(qt0 + it % nq) * BM;
                    const uint32_t win_bytes = kBias ? 2u * Cfg::WIN_BYTES : 0u;
                    uint8_t *sQ = smem + Cfg::OFF_Q + st * Cfg::Q_BYTES, *sdO = smem + Cfg::OFF_DO + st * Cfg::Q_BYTES;
                    q_armed = x + 1;
                    mbar_arrive_expect_tx(&q_full[st], 2 * Cfg::Q_BYTES + 2 * BM * 4 + win_bytes);
                    for (int c = 0; c < D / 64; ++c) {
                        tma_load_4d(sQ + c * BM * 128, &p.tm_q, &q_full[st], c * 64, int(q_row0 + i0), int(hq), q_b);
                        tma_load_4d(sdO + c * BM * 128, &p.tm_do, &q_full[st], c * 64, int(q_row0 + i0), int(hq), q_b);
                    }
                    const int64_t wrow = hq * a.t_pad + geo.ws_start(b) + i0;
                    if (!pre_done) {  // LSE / D come from the preprocess
                        pdl_wait();
                        pre_done = true;
                    }
                    bulk_load(smem + Cfg::OFF_LSE + st * BM * 4, a.lse2 + wrow, BM * 4, &q_full[st]);
                    bulk_load(smem + Cfg::OFF_DVEC + st * BM * 4, a.dvec + wrow, BM * 4, &q_full[st]);
                    if (kBias) {  // the windows from the tile's first delta on, 16-byte aligned
                        uint8_t *win = smem + Cfg::OFF_WIN + st * 2 * Cfg::WIN_BYTES;
                        const int w0 = window_start(int(j0 - i0 - (BM - 1) - (a.mask == ATTN_CAUSAL_BOTTOM_RIGHT ? lkv - lq : 0))) & ~3;
                        bulk_load(win, p.rel.rel + hq * p.rel.stride + w0, Cfg::WIN_BYTES, &q_full[st]);
                        bulk_load(win + Cfg::WIN_BYTES, p.rel.code + w0, Cfg::WIN_BYTES, &q_full[st]);
                    }
                };
                // the first query tile does not need the key tile: load it before waiting for K / V
                // (except on the very first tile, whose K / V load should start first)
                auto load_kv = [&]() {
                    if (kt > 0 && ok && !(ok = mbar_wait(kv_empty, uint32_t(kt - 1) & 1, abort)))
                        flag_abort(abort, a.status);
                    if (ok) {
                        kv_armed = kt + 1;
                        mbar_arrive_expect_tx(kv_full, 2 * Cfg::KV_BYTES);
                        for (int c = 0; c < D / 64; ++c) {
                            tma_load_4d(sK + c * BN * 128, &p.tm_k, kv_full, c * 64, int(kv_row0 + j0), int(g) / shares, kv_b);
                            tma_load_4d(sV + c * BN * 128, &p.tm_v, kv_full, c * 64, int(kv_row0 + j0), int(g) / shares, kv_b);
                        }
                    }
                };
                if (kt == 0) load_kv();
                load_q(0, qi);
                // warm L2 with the K / V tile this CTA takes next, so its load does not stall the next unit
                // (on the CTA's first tile only after its second query tile: the first tile's own loads
                // go first)
                auto prefetch_next = [&]() {
                    int64_t nb = b, ng = g, njt = jt + tile_step, nrow0 = kv_row0;
                    int nkv_b = kv_b;
                    bool has = njt < ntiles;
                    if (!has) {
                        const int64_t u2 = cta_unit(p, round_ + 1);
                        if (u2 >= 0) {
                            const uint32_t njt_ = uint32_t(u2) / uint32_t(nheads);
                            const uint32_t bg2 = uint32_t(u2) - njt_ * uint32_t(nheads);
                            nb = bg2 / uint32_t(a.h_kv);
                            ng = int64_t(bg2) - nb * a.h_kv;
                            njt = njt_;
                            nrow0 = kPacked ? geo.kv_start(nb) : 0;
                            nkv_b = kPacked ? 0 : int(nb);
                            has = njt * BN < geo.kv_len(nb);
                        }
                    }
                    if (has)
                        for (int c = 0; c < D / 64; ++c) {
                            tma_prefetch_4d(&p.tm_k, c * 64, int(nrow0 + njt * BN), int(ng) / shares, nkv_b);
                            tma_prefetch_4d(&p.tm_v, c * 64, int(nrow0 + njt * BN), int(ng) / shares, nkv_b);
                        }
                };
                if (kt > 0 || n_iter == 1) prefetch_next();
                if (kt > 0) load_kv();
                ++qi;
                for (int it = 1; it < n_iter; ++it, ++qi) {
                    load_q(it, qi);
                    if (kt == 0 && it == 1) prefetch_next();
                }
                ++kt;
            }
            ATTN_END_UNITS
            if (!ok) {
                // let every copy this thread started land before the CTA exits
                volatile int never = 0;
                for (int64_t x = q_armed - NST; x < q_armed; ++x)
                    if (x >= 0) mbar_wait(&q_full[x % NST], uint32_t(x / NST) & 1, &never, 100000000ull);
                if (kv_armed > 0) mbar_wait(kv_full, uint32_t(kv_armed - 1) & 1, &never, 100000000ull);
            }
        }
    } else if (warp == 1) {
        // ================================================= MMA issuer
        if (elect_one()) {
            constexpr uint32_t idS = idesc_f16(128, BM / NH, kType, 0, 0);
            constexpr uint32_t idDV = idesc_f16(128, D, kType, 0, 1);
            constexpr uint32_t idDQ = idesc_f16(128, 64, kType, 1, 1);
            const uint32_t aK = smem_u32(sK), aV = smem_u32(sV);
            bool ok = true;
            int64_t kt = 0;
            uint32_t qi = 0, st_par = 0;
            int st = 0;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (ok && !(ok = mbar_wait(bar, parity, abort))) flag_abort(abort, a.status);
                tc_fence_after();
            };
            // step-0 descriptors of the K / V tile (K-major for S / dP, MN-major for dQ)
            const uint64_t kK = desc_kmaj(aK, BN, 0), kV = desc_kmaj(aV, BN, 0), mK = desc_mn(aK, BN, 0);
            // dV, dK, dQ of query tile x (global index) whose P / dS are ready
            // x: global index of the query tile, xs: its ring stage
            // last: the key tile's last query tile; its dQ GEMM, the only one of the three that reads K,
            // goes first, so the K / V reload for the next key tile can start as early as possible
            auto grads = [&](uint32_t x, int xs, bool first, bool last) {
                const int st = xs;
                const uint32_t adS = smem_u32(sX + (x & 1) * Cfg::X_BYTES);
                const uint64_t mdO = desc_mn(smem_u32(smem + Cfg::OFF_DO + st * Cfg::Q_BYTES), BM, 0);
                const uint64_t mQ = desc_mn(smem_u32(smem + Cfg::OFF_Q + st * Cfg::Q_BYTES), BM, 0);
                const uint64_t kdS = desc_kmaj(adS, BN, 0), mdS = desc_mn(adS, BN, 0);
                auto dq_gemm = [&]() {
                    if (x > 0) wait(dq_free, (x - 1) & 1);
                    if (ok) {
#pragma unroll
                        for (int kk = 0; kk < BN / 16; ++kk) {
                            if (D == 64)
                                mma_f16_ss(tmem + Cfg::T_DQ, mn_step(mdS, kk), mn_step(mK, kk), idDQ, kk > 0);
                            else
                                mma_f16_ss(tmem + Cfg::T_DQ, mn_step(mK, kk), mn_step(mdS, kk), idDQ, kk > 0);
                        }
                        if (last) mma_commit(kv_empty);  // K / V are no longer read once these GEMMs finish
                    }
                };
                if (last) dq_gemm();
                // a new key tile overwrites dV / dK: the previous tile's epilogue has read them
                if (first && kt > 0) wait(acc_free, uint32_t(kt - 1) & 1);
                if (ok) {
#pragma unroll
                    for (int kk = 0; kk < BM / 16; ++kk)
                        mma_f16_ts(tmem + Cfg::T_DV, tmem + Cfg::T_P + kk * 8, mn_step(mdO, kk), idDV, !first || kk > 0);
                    mma_commit(p_free);
#pragma unroll
                    for (int kk = 0; kk < BM / 16; ++kk)
                        mma_f16_ss(tmem + Cfg::T_DK, kmaj_step(kdS, BN, kk), mn_step(mQ, kk), idDV, !first || kk > 0);
                    mma_commit(&q_empty[st]);  // the Q / dO stage may be refilled once dV / dK have read it
                }
                if (!last) dq_gemm();
                if (ok) {
                    mma_commit(mma_done);
                    mma_commit(&ds_free[x & 1]);
                }
            };
            ATTN_FOR_EACH_UNIT
            for (int64_t jt = first_tile; jt < ntiles; jt += tile_step) {
                const int64_t j0 = jt * BN;
                int qt0, nq;
                query_tiles<BM>(a.mask, j0, lq, lkv, &qt0, &nq);
                const int n_iter = G * nq;
                if (n_iter == 0) continue;
                wait(kv_full, uint32_t(kt) & 1);
                int prev_st = 0;
                for (int it = 0; it < n_iter; ++it, ++qi) {
                    const uint64_t kQ = desc_kmaj(smem_u32(smem + Cfg::OFF_Q + st * Cfg::Q_BYTES), BM, 0);
                    const uint64_t kdO = desc_kmaj(smem_u32(smem + Cfg::OFF_DO + st * Cfg::Q_BYTES), BM, 0);
                    wait(&q_full[st], st_par);
#pragma unroll
                    for (int q = 0; q < NH; ++q) {
                        // this column group of the previous tile has been read out of TMEM
                        if (qi > 0) wait(&s_free[q], (qi - 1) & 1);
                        if (ok) {
                            const uint32_t qoff = uint32_t(q * (BM / NH) * 128 / 16);  // query rows, in 16 B
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                mma_f16_ss(tmem + Cfg::T_S + q * (BM / NH), kmaj_step(kK, BN, kk),
                                           kmaj_step(kQ + qoff, BM, kk), idS, kk > 0);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                mma_f16_ss(tmem + Cfg::T_DP + q * (BM / NH), kmaj_step(kV, BN, kk),
                                           kmaj_step(kdO + qoff, BM, kk), idS, kk > 0);
                            mma_commit(&s_full[q]);
                        }
                    }
                    if (it > 0) {
                        wait(p_ready, (qi - 1) & 1);
                        grads(qi - 1, prev_st, it == 1, false);
                    }
                    prev_st = st;
                    if (++st == NST) {
                        st = 0;
                        st_par ^= 1;
                    }
                }
                wait(p_ready, (qi - 1) & 1);
                grads(qi - 1, prev_st, n_iter == 1, true);
                ++kt;
            }
            ATTN_END_UNITS
            // wait for every MMA this thread issued before TMEM is freed
            volatile int never = 0;
            mma_commit(drain);
            mbar_wait(drain, 0, &never, 100000000ull);
        }
    } else if (warp < 2 + Cfg::NSW) {
        // ================================================= P^T / dS^T (warps 2 .. 1 + NSW)
        const int lg = warp & 3, half = (warp - 2) >> 2;  // lane quadrant, column slice
        const uint32_t lane_addr = uint32_t(lg * 32) << 16;
        const int r = lg * 32 + lane;  // TMEM lane of this thread = key row of the tile
        const float sc = a.scale * kLog2e;
        const uint32_t aX = smem_u32(sX);
        bool ok = true;
        uint32_t qi = 0;            // query tiles done by this CTA
        int st = 0;                 // their Q / dO ring stage ...
        uint32_t st_par = 0;        // ... and its phase parity
        // tc: the wait orders later TMEM accesses (else it only guards shared memory)
        auto wait = [&](uint64_t *bar, uint32_t parity, bool tc) {
            if (ok && !(ok = mbar_wait(bar, parity, abort))) flag_abort(abort, a.status);
            ok = __all_sync(0xffffffffu, ok);
            if (tc) tc_fence_after();
        };

        // relative bias: this warp's bucket sums and finished diagonals; the bucket of the last block that lay in
        // one, and each thread's sum since
        float *hist = reinterpret_cast<float *>(smem + Cfg::OFF_HIST) + (warp - 2) * kRelCodes;
        float2 *diag = reinterpret_cast<float2 *>(smem + Cfg::OFF_DIAG) + (warp - 2) * 32;
        float one_sum = 0.f;
        uint32_t one_bucket = 0;
        if (kBias) {
            for (int n = lane; n < kRelCodes; n += 32) hist[n] = 0.f;
            __syncwarp();
        }
        // adds v, the sum of one diagonal a lane (consecutive deltas), to the bucket sums: runs of one bucket are
        // added up towards their first lane, whose bucket no other run has
        auto add_runs = [&](float v, uint32_t code) {
            const int rem = min(int(code >> 8 & 31u), 31 - lane);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float t = __shfl_down_sync(0xffffffffu, v, o);
                if (o <= rem) v += t;
            }
            if (lane == 0 || (code >> 16)) hist[code & 255u] += v;
            __syncwarp();
        };
        auto add_one = [&]() {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) one_sum += __shfl_xor_sync(0xffffffffu, one_sum, o);
            if (lane == 0) hist[one_bucket] += one_sum;
            __syncwarp();
            one_sum = 0.f;
        };
        // end of a (key tile, head): the sums go to their row of the workspace
        auto flush = [&](int64_t row, int64_t head) {
            add_one();
            float *dst = p.rel.part + ((row * a.h + head) * 8 + (warp - 2)) * p.rel.b.buckets;
            for (int n = lane; n < p.rel.b.buckets; n += 32) {
                dst[n] = hist[n];
                hist[n] = 0.f;
            }
            __syncwarp();
        };

        ATTN_FOR_EACH_UNIT
        const int64_t shift = a.mask == ATTN_CAUSAL_BOTTOM_RIGHT ? lkv - lq : 0;
        for (int64_t jt = first_tile; jt < ntiles; jt += tile_step) {
            const int64_t j0 = jt * BN, j = j0 + r;
            const bool row_ok = j < lkv;
            int qt0, nq;
            query_tiles<BM>(a.mask, j0, lq, lkv, &qt0, &nq);
            const int n_iter = G * nq;
            int iq = 0;  // query tile within the head
            int64_t hq = g * G;                 // kBias: the head
            const int jrel = int(j - shift);    // kBias: the key's position as the queries' are counted
            for (int it = 0; it < n_iter; ++it, ++qi) {
                const int64_t i0 = int64_t(qt0 + iq) * BM;
                // Usually LSE / D of this tile have landed (q_full), the GEMMs of tile qi - 2 that read
                // dS buffer qi & 1 have completed (ds_free) and the first S^T / dP^T group is written
                // (s_full): test all three at once and wait one by one only if one is not.
                const uint32_t t_q = mbar_test_wait(&q_full[st], st_par);
                const uint32_t t_d = qi >= 2 ? mbar_test_wait(&ds_free[qi & 1], ((qi >> 1) - 1) & 1) : 1u;
                const uint32_t t_s = mbar_test_wait(&s_full[0], qi & 1);
                const bool ready0 = __all_sync(0xffffffffu, t_q && t_d && t_s);
                if (!ready0) {
                    wait(&q_full[st], st_par, false);
                    if (qi >= 2) wait(&ds_free[qi & 1], ((qi >> 1) - 1) & 1, false);
                }
                bool ready1 = false;  // the previous tile's dV has read P^T and the second group is written
                const uint32_t adS = aX + uint32_t(qi & 1) * Cfg::X_BYTES;
                const uint32_t a_lse = smem_u32(smem + Cfg::OFF_LSE + st * BM * 4);
                const uint32_t a_dv = smem_u32(smem + Cfg::OFF_DVEC + st * BM * 4);
                // first visible query column of this key row; everything is masked past the sequence (kBias: the
                // causal mask is in the bias)
                int cmin;
                if (kBias) {
                    cmin = !row_ok ? BM : -1;
                } else {
                    const int64_t cmin64 = !row_ok ? INT64_MAX : (a.mask ? j - shift - i0 : INT64_MIN);
                    cmin = int(cmin64 < -1 ? -1 : (cmin64 > BM ? BM : cmin64));
                }
                // kBias: the tile's windows; columns from cmax on lie past the sequence's queries; a block's share of
                // the table's gradient: two diagonal sums a lane and their codes, or (one bucket) the thread's sum
                const float *win = reinterpret_cast<const float *>(smem + Cfg::OFF_WIN + st * 2 * Cfg::WIN_BYTES);
                if (kBias) win += window_start(jrel - r - (BM - 1) - int(i0)) & 3;
                const uint32_t *wcode = reinterpret_cast<const uint32_t *>(win) + Cfg::WIN_BYTES / 4;
                const int cmax = kBias ? min(BM, int(lq) - int(i0)) : BM;
                float left_a = 0.f, left_b = 0.f;
                uint32_t code_a = 0, code_b = 0;
                bool several = false;
                auto add_block = [&]() {
                    if (several) {
                        add_runs(left_a, code_a);
                        add_runs(left_b, code_b);
                    } else {
                        if (code_a != one_bucket) {
                            add_one();
                            one_bucket = code_a;
                        }
                        one_sum += left_a;
                    }
                };
                // (with a bias the column groups share one copy of the code: unrolled, it does not fit the
                // instruction cache)
#pragma unroll (kBias ? 1 : NG)
                for (int q = 0; q < NG; ++q) {
                    const int rel = NH == NG ? q : 0;  // release group of these columns
                    if (q == 0 ? !ready0 : (NH == NG && !ready1)) wait(&s_full[rel], qi & 1, true);
                    else if (q == 0) tc_fence_after();
                    const int c0 = q * (BM / NG) + half * GW;
                    uint32_t pk[GW / 2];  // P^T of this column group, packed
                    // S^T / dP^T of the group in chunks of 16 columns.  With one group a thread (d = 128)
                    // the whole group is loaded at once and its TMEM columns released before P / dS are
                    // computed, so the next tile's S^T / dP^T GEMMs overlap this tile's element-wise work;
                    // with two (d = 64) chunk cc + 1 is loaded while chunk cc is computed and the columns
                    // are released after the group (the early release measured slower there; so it does with a
                    // bias at d = 128, whose arithmetic needs the registers: 816 us against 926 at b2 h32 s4096)
                    constexpr int NCH = GW / 16;
                    constexpr bool kEarlyFree = NG == 1 && NCH == 2 && !kBias;
                    uint32_t sbuf[2][16], dbuf[2][16];
                    auto release = [&]() {
                        if (NH == NG || q == NG - 1) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&s_free[rel]);  // these columns may be overwritten
                        }
                    };
                    if (kEarlyFree) {
                        if (ok) {
#pragma unroll
                            for (int cc = 0; cc < NCH; ++cc) {
                                tmem_ld16(tmem + lane_addr + Cfg::T_S + c0 + 16 * cc, sbuf[cc & 1]);
                                tmem_ld16(tmem + lane_addr + Cfg::T_DP + c0 + 16 * cc, dbuf[cc & 1]);
                            }
                            tmem_ld_wait_regs(sbuf[0], dbuf[0]);
                            tmem_ld_wait_regs(sbuf[1], dbuf[1]);
                        }
                        release();
                    } else if (ok) {
                        tmem_ld16(tmem + lane_addr + Cfg::T_S + c0, sbuf[0]);
                        tmem_ld16(tmem + lane_addr + Cfg::T_DP + c0, dbuf[0]);
                    }
                    if (ok) {
                        const bool any_mask = __any_sync(0xffffffffu, cmin > c0) || (kBias && cmax < c0 + GW);
                        // chunk cc's S^T / dP^T has arrived; the next chunk's loads go out
                        auto fetch = [&](int cc) {
                            if (!kEarlyFree) {
                                tmem_ld_wait_regs(sbuf[cc & 1], dbuf[cc & 1]);
                                if (cc + 1 < NCH) {
                                    tmem_ld16(tmem + lane_addr + Cfg::T_S + c0 + cc * 16 + 16, sbuf[(cc & 1) ^ 1]);
                                    tmem_ld16(tmem + lane_addr + Cfg::T_DP + c0 + cc * 16 + 16, dbuf[(cc & 1) ^ 1]);
                                }
                            }
                        };
                        auto store_ds = [&](int cc, const uint32_t (&dk)[8]) {
#pragma unroll
                            for (int q2 = 0; q2 < 2; ++q2) {
                                const uint32_t off = sw128_offset(uint32_t(r), uint32_t(c0 + cc * 16 + 8 * q2), BN);
                                st_shared_v4(adS + off, dk[4 * q2], dk[4 * q2 + 1], dk[4 * q2 + 2], dk[4 * q2 + 3]);
                            }
                        };
                        if constexpr (kBias) {
                            static_assert(GW == 32, "blocks of 32 x 32");
                            const float *wrow = win + r + BM - 1 - c0;  // entry of column c0 + k: wrow[-k]
                            const uint32_t *code = wcode + lg * 32 + BM - 1 - c0;  // of diagonal (row - column) 0
                            several = (code[-31] & 255u) != (code[31] & 255u) || any_mask;
                            float2 sum2 = make_float2(0.f, 0.f);
                            float2 run = make_float2(0.f, 0.f);
                            const float2 up1 = lane < 2 ? make_float2(0.f, 0.f) : make_float2(1.f, 1.f);
                            // kAny: several buckets, or masked elements (kMask)
                            auto block = [&](auto any_tag, auto mask_tag) {
                                constexpr bool kAny = decltype(any_tag)::value, kMask = decltype(mask_tag)::value;
                                const float wone = wrow[0];
                                const float2 sc2 = make_float2(sc, sc), neg2 = make_float2(-1.f, -1.f);
#pragma unroll
                                for (int cc = 0; cc < NCH; ++cc) {
                                    const int col0 = c0 + cc * 16, cur = cc & 1;
                                    fetch(cc);
                                    uint32_t dk[8];
                                    float2 lse4[2], dv4[2];
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) {
                                        const int k = cc * 16 + e, c = c0 + k;
                                        if (e % 4 == 0) {
                                            const float4 l4 = ld_shared_f4(a_lse + uint32_t(col0 + e) * 4);
                                            const float4 d4 = ld_shared_f4(a_dv + uint32_t(col0 + e) * 4);
                                            lse4[0] = make_float2(l4.x, l4.y);
                                            lse4[1] = make_float2(l4.z, l4.w);
                                            dv4[0] = make_float2(d4.x, d4.y);
                                            dv4[1] = make_float2(d4.z, d4.w);
                                        }
                                        const float2 lse2 = lse4[e / 2 % 2], dv2 = dv4[e / 2 % 2];
                                        const float2 b2 = kAny ? make_float2(wrow[-k], wrow[-k - 1]) : make_float2(wone, wone);
                                        float2 x = fma2(make_float2(__uint_as_float(sbuf[cur][e]), __uint_as_float(sbuf[cur][e + 1])),
                                                        sc2, fma2(lse2, neg2, b2));
                                        float2 g = fma2(dv2, neg2,
                                                        make_float2(__uint_as_float(dbuf[cur][e]), __uint_as_float(dbuf[cur][e + 1])));
                                        if (kMask) {  // a masked element's dP may be anything
                                            const bool v0 = c >= cmin && c < cmax, v1 = c + 1 >= cmin && c + 1 < cmax;
                                            x.x = v0 ? x.x : -INFINITY;
                                            x.y = v1 ? x.y : -INFINITY;
                                            g.x = v0 ? g.x : 0.f;
                                            g.y = v1 ? g.y : 0.f;
                                        }
                                        const float2 pp = make_float2(ex2(x.x), ex2(x.y)), ds = mul2(pp, g);
                                        pk[k / 2] = pack2<T>(pp.x, pp.y);
                                        dk[e / 2] = pack2<T>(ds.x, ds.y);
                                        if (kAny) {
                                            // the sums of diagonals lane - k (even columns) and lane - k - 1 (odd
                                            // ones) go two lanes up a pair; those of lanes 30 and 31 are complete
                                            if (k > 0) {
                                                if (lane >= 30) diag[lane - k + 2] = run;
                                                const float2 up = make_float2(__shfl_up_sync(0xffffffffu, run.x, 2),
                                                                              __shfl_up_sync(0xffffffffu, run.y, 2));
                                                run = fma2(up, up1, ds);
                                            } else {
                                                run = ds;
                                            }
                                        } else {
                                            sum2 = add2(sum2, ds);
                                        }
                                    }
                                    store_ds(cc, dk);
                                }
                            };
                            if (several) {  // diag[d]: diagonal d's even columns and diagonal d - 1's odd ones
                                if (any_mask) block(std::true_type{}, std::true_type{});
                                else block(std::true_type{}, std::false_type{});
                                const float up = __shfl_up_sync(0xffffffffu, run.x, 1);
                                if (lane == 31) diag[1] = run;
                                __syncwarp();
                                left_a = lane == 0 ? run.y : up + run.y;
                                code_a = code[lane - 31];
                                // diagonal lane + 1: its even columns' sum is in that entry, its odd ones' in the next
                                left_b = (lane < 31 ? diag[lane + 1].x : 0.f) + (lane < 30 ? diag[lane + 2].y : 0.f);
                                code_b = code[lane + 1];
                            } else {
                                block(std::false_type{}, std::false_type{});
                                left_a = sum2.x + sum2.y;
                                code_a = code[0] & 255u;
                            }
                            if (q < NG - 1) add_block();  // the last group's waits for the arrival below
                        } else {
#pragma unroll
                            for (int cc = 0; cc < NCH; ++cc) {
                                const int col0 = c0 + cc * 16, cur = cc & 1;
                                fetch(cc);
                                uint32_t dk[8];
#pragma unroll
                                for (int q4 = 0; q4 < 4; ++q4) {
                                    const float4 l4 = ld_shared_f4(a_lse + uint32_t(col0 + 4 * q4) * 4);
                                    const float4 d4 = ld_shared_f4(a_dv + uint32_t(col0 + 4 * q4) * 4);
                                    const float lse4[4] = {l4.x, l4.y, l4.z, l4.w}, dv4[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                                    for (int h2 = 0; h2 < 2; ++h2) {
                                        const int e = 4 * q4 + 2 * h2, c = col0 + e;
                                        float x0 = fmaf(__uint_as_float(sbuf[cur][e]), sc, -lse4[2 * h2]);
                                        float x1 = fmaf(__uint_as_float(sbuf[cur][e + 1]), sc, -lse4[2 * h2 + 1]);
                                        if (any_mask) {
                                            x0 = c >= cmin ? x0 : -INFINITY;
                                            x1 = c + 1 >= cmin ? x1 : -INFINITY;
                                        }
                                        const float g0 = __uint_as_float(dbuf[cur][e]) - dv4[2 * h2];
                                        const float g1 = __uint_as_float(dbuf[cur][e + 1]) - dv4[2 * h2 + 1];
                                        pk[cc * 8 + 2 * q4 + h2] = p_and_ds<T>(x0, x1, g0, g1, &dk[2 * q4 + h2]);
                                    }
                                }
                                store_ds(cc, dk);
                            }
                        }
                    }
                    if (!kEarlyFree) release();
                    // P^T into TMEM once the previous tile's dV GEMM has read it
                    if (q == 0) {
                        const uint32_t t_p = qi > 0 ? mbar_test_wait(p_free, (qi - 1) & 1) : 1u;
                        const uint32_t t_s1 = NH == NG && NG > 1 ? mbar_test_wait(&s_full[NG > 1 ? 1 : 0], qi & 1) : 1u;
                        ready1 = __all_sync(0xffffffffu, t_p && t_s1);
                        if (!ready1 && qi > 0) wait(p_free, (qi - 1) & 1, true);
                        else tc_fence_after();
                    }
                    if (ok) {
#pragma unroll
                        for (int cc = 0; cc < GW / 16; ++cc) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = pk[cc * 8 + e];
                            tmem_st8(tmem + lane_addr + Cfg::T_P + c0 / 2 + cc * 8, w);
                        }
                    }
                }
                if (kBias && kPacked && ok) {  // rows of other sequences: zero before the GEMMs that read them by rows
                    const int t = threadIdx.x - 64;
                    auto zero_rows = [&](uint8_t *tile, int first, int rows) {
                        for (int k = first * (D / 8) + t; k < rows * (D / 8); k += 32 * Cfg::NSW) {
                            const int row = k / (D / 8), piece = k % (D / 8);
                            st_shared_v4(smem_u32(tile) + uint32_t(piece / 8 * rows * 128 + row * 128 + piece % 8 * 16), 0, 0, 0, 0);
                        }
                    };
                    if (cmax < BM) {
                        zero_rows(smem + Cfg::OFF_Q + st * Cfg::Q_BYTES, cmax, BM);
                        zero_rows(smem + Cfg::OFF_DO + st * Cfg::Q_BYTES, cmax, BM);
                    }
                    if (it == 0 && lkv - j0 < BN) zero_rows(sK, int(lkv - j0), BN);
                }
                if (ok) tmem_st_wait();
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready);
                if (kBias && ok) add_block();
                if (++st == NST) {
                    st = 0;
                    st_par ^= 1;
                }
                if (++iq == nq) {
                    iq = 0;
                    if (kBias) flush(geo.kv_start(b) / 128 + b + jt, hq++);
                }
            }
        }
        ATTN_END_UNITS
        pdl_trigger();
    } else if (kOrdered && warp == 2 + Cfg::NSW + 4) {
        // ================================================= ordered dQ mode: add counts (warp 14)
        // A GPU-scope release stalls the warp that issues it for about a microsecond; the dQ leader
        // hands each counter over (after its adds have landed and a proxy fence) and goes on, and
        // this warp publishes it.  A null counter ends the list.
        if (lane == 0) {
            for (uint32_t n = 0;; ++n) {
                const int k = int(n % kMailbox);
                if (!mbar_wait(&mb_full[k], (n / kMailbox) & 1, abort)) {
                    if (!*abort) flag_abort(abort, a.status);
                    break;
                }
                uint32_t *const ctr = mailbox[k];
                mbar_arrive(&mb_empty[k]);
                if (!ctr) break;
                red_release_gpu_add(ctr, 1u);
            }
        }
    } else {
        // ================================================= dQ reduce, dK / dV epilogue (warps 10..13)
        const int lg = warp & 3;
        const uint32_t lane_addr = uint32_t(lg * 32) << 16;
        const int r = lg * 32 + lane;  // TMEM lane of this thread
        const bool leader = warp == 2 + Cfg::NSW && lane == 0;
        uint8_t *sDQS = smem + Cfg::OFF_DQS;
        const uint32_t aDQS = smem_u32(sDQS);
        T *dK = static_cast<T *>(a.dK.ptr), *dV = static_cast<T *>(a.dV.ptr);
        bool ok = true;
        uint32_t qi = 0;
        uint32_t *pend = nullptr;  // ordered dQ mode: counter of the tile whose adds are still to be counted
        uint32_t n_post = 0;       // ... and the counters handed to the publishing warp so far
        auto post = [&](uint32_t *ctr) {
            const int k = int(n_post % kMailbox);
            if (n_post >= kMailbox && ok && !(ok = mbar_wait(&mb_empty[k], ((n_post / kMailbox) - 1) & 1, abort)))
                flag_abort(abort, a.status);
            if (ok) {
                mailbox[k] = ctr;
                mbar_arrive(&mb_full[k]);
            }
            ++n_post;
        };
        pdl_wait();  // the dQ accumulator (and the ordered mode's counters) have been zeroed

        ATTN_FOR_EACH_UNIT
        for (int64_t jt = first_tile; jt < ntiles; jt += tile_step) {
            const int64_t j0 = jt * BN, j = j0 + r;
            const bool row_ok = j < lkv;
            // element offsets of this thread's dK / dV row (recomputed where used: fewer live registers)
            auto offk = [&]() { return kv_b * a.dK.sb + g * a.dK.sh + (kv_row0 + j) * a.dK.ss; };
            auto offv = [&]() { return kv_b * a.dV.sb + g * a.dV.sh + (kv_row0 + j) * a.dV.ss; };
            int qt0, nq;
            query_tiles<BM>(a.mask, j0, lq, lkv, &qt0, &nq);
            const int n_iter = G * nq;
            // shares > 1: this thread's row of its unit's fp32 dK, and how far behind that of dV lies
            const int64_t share_size = (a.h_kv / shares) * a.t_kv * D;
            auto share_row = [&]() {
                return p.rel.kv_part + (g % shares) * share_size +
                       ((g / shares) * a.t_kv + (kPacked ? kv_row0 : int64_t(kv_b) * lkv) + j) * D;
            };
            if (n_iter == 0) {  // no query sees these keys: dK = dV = 0
                if (kBias && shares > 1) {
                    if (row_ok)
                        for (int x = 0; x < D; x += 4) {
                            *reinterpret_cast<float4 *>(share_row() + x) = make_float4(0.f, 0.f, 0.f, 0.f);
                            *reinterpret_cast<float4 *>(share_row() + shares * share_size + x) = make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                } else if (row_ok)
                    for (int x = 0; x < D; x += 8) {
                        *reinterpret_cast<uint4 *>(dK + offk() + x) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(dV + offv() + x) = make_uint4(0, 0, 0, 0);
                    }
                continue;
            }
            // dK (scaled) and dV of this key tile, once its last GEMMs have completed.  When TMA may
            // store the tile whole (fixed-length layout, whose extent clips the last tile; or a packed
            // tile inside its sequence), dV, then dK, is staged as 16-bit rows in the dQ staging buffer
            // and written by a TMA store
            // (d = 64 only: at d = 128 the 64 KB of dK / dV would pass through the 16 KB buffer in four
            // serial rounds, slower than the row stores)
            const bool tma_epi = D == 64 && (!kPacked || j0 + BN <= lkv) && !(kBias && shares > 1);
            auto epilogue_tma = [&]() {
                constexpr int NBOX = D / 64;
#pragma unroll 1
                for (int t = 0; t < 2 * NBOX; ++t) {
                    const bool isk = t >= NBOX;
                    const int cb = t % NBOX;
                    const uint32_t tcol = (isk ? Cfg::T_DK : Cfg::T_DV) + cb * 64;
                    const float mul = isk ? a.scale : 1.f;
                    if (leader) bulk_wait_read0();  // the buffer's previous reader (reduce or store) is done
                    named_bar_sync(2, 128);
                    if (ok) {
#pragma unroll
                        for (int c16 = 0; c16 < 4; ++c16) {  // 16 columns at a time, two 16-byte chunks
                            uint32_t w[16];
                            tmem_ld16(tmem + lane_addr + tcol + c16 * 16, w);
                            tmem_ld_wait_regs(w);
#pragma unroll
                            for (int h2 = 0; h2 < 2; ++h2) {
                                const uint32_t off = sw128_offset(uint32_t(r), uint32_t(c16 * 16 + h2 * 8), BN);
                                st_shared_v4(aDQS + off,
                                             pack2<T>(__uint_as_float(w[8 * h2 + 0]) * mul, __uint_as_float(w[8 * h2 + 1]) * mul),
                                             pack2<T>(__uint_as_float(w[8 * h2 + 2]) * mul, __uint_as_float(w[8 * h2 + 3]) * mul),
                                             pack2<T>(__uint_as_float(w[8 * h2 + 4]) * mul, __uint_as_float(w[8 * h2 + 5]) * mul),
                                             pack2<T>(__uint_as_float(w[8 * h2 + 6]) * mul, __uint_as_float(w[8 * h2 + 7]) * mul));
                            }
                        }
                    }
                    if (t == 2 * NBOX - 1) {  // every accumulator column has been read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(acc_free);
                    }
                    fence_proxy_async_smem();
                    named_bar_sync(2, 128);
                    if (leader && ok) {
                        tma_store_4d(isk ? &p.tm_dk : &p.tm_dv, sDQS, cb * 64, int(kv_row0 + j0), int(g), kv_b);
                        bulk_commit();
                    }
                }
            };
            // otherwise: read out of TMEM first (the accumulators are released right after the last
            // read, so the next key tile's first GEMMs need not wait for the dQ reduce), then stored
            // row by row
            auto epilogue = [&]() {
#pragma unroll 1
                for (int cc = 0; cc < D / 8; ++cc) {
                    uint32_t w[8], u[8];
                    if (ok) {
                        tmem_ld8(tmem + lane_addr + Cfg::T_DV + cc * 8, w);
                        tmem_ld8(tmem + lane_addr + Cfg::T_DK + cc * 8, u);
                        tmem_ld_wait_regs(w, u);
                    }
                    if (cc == D / 8 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(acc_free);
                    }
                    if (kBias && shares > 1) {
                        if (ok && row_ok) {
                            uint4 *pk = reinterpret_cast<uint4 *>(share_row() + cc * 8);
                            uint4 *pv = reinterpret_cast<uint4 *>(share_row() + shares * share_size + cc * 8);
                            pk[0] = make_uint4(u[0], u[1], u[2], u[3]);
                            pk[1] = make_uint4(u[4], u[5], u[6], u[7]);
                            pv[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            pv[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    } else if (ok && row_ok) {
                        uint4 ov, ok4;
                        ov.x = pack2<T>(__uint_as_float(w[0]), __uint_as_float(w[1]));
                        ov.y = pack2<T>(__uint_as_float(w[2]), __uint_as_float(w[3]));
                        ov.z = pack2<T>(__uint_as_float(w[4]), __uint_as_float(w[5]));
                        ov.w = pack2<T>(__uint_as_float(w[6]), __uint_as_float(w[7]));
                        ok4.x = pack2<T>(__uint_as_float(u[0]) * a.scale, __uint_as_float(u[1]) * a.scale);
                        ok4.y = pack2<T>(__uint_as_float(u[2]) * a.scale, __uint_as_float(u[3]) * a.scale);
                        ok4.z = pack2<T>(__uint_as_float(u[4]) * a.scale, __uint_as_float(u[5]) * a.scale);
                        ok4.w = pack2<T>(__uint_as_float(u[6]) * a.scale, __uint_as_float(u[7]) * a.scale);
                        *reinterpret_cast<uint4 *>(dV + offv() + cc * 8) = ov;
                        *reinterpret_cast<uint4 *>(dK + offk() + cc * 8) = ok4;
                    }
                }
            };
            int iq = 0, hg = 0;  // query tile within the head, head within the group
            for (int it = 0; it < n_iter; ++it, ++qi) {
                const int64_t hq = g * G + hg, i0 = int64_t(qt0 + iq) * BM;
                if (++iq == nq) {
                    iq = 0;
                    ++hg;
                }
                if (ok && !(ok = mbar_wait(mma_done, qi & 1, abort))) flag_abort(abort, a.status);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                if (it == n_iter - 1) {
                    if (tma_epi) epilogue_tma();
                    else epilogue();
                }
                // dQ of tile qi, half of its columns at a time, through the staging buffer
                const int64_t row0 = part * a.h * a.t_pad + geo.ws_start(b) + hq * a.t_pad + i0;
                // ordered dQ mode: this query tile's add counter
                auto sem_of = [&]() { return a.sem + hq * a.sem_stride + (geo.ws_start(b) + i0) / 64; };
                // read the whole accumulator first, so the next tile's dQ GEMM is not held up by the
                // reduce (whose rate the L2 sets)
                uint32_t v[2][32];
                if (ok) {
                    tmem_ld32(tmem + lane_addr + Cfg::T_DQ, v[0]);
                    tmem_ld32(tmem + lane_addr + Cfg::T_DQ + 32, v[1]);
                    tmem_ld_wait_regs(v[0]);
                    tmem_ld_wait_regs(v[1]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dq_free);
#pragma unroll
                for (int hb = 0; hb < 2; ++hb) {  // half of the columns at a time through the staging buffer
                    if (leader) bulk_wait_read0();  // the previous reduce has read the staging buffer
                    named_bar_sync(2, 128);
                    if (ok) {
                        if (D == 64) {  // lane = query row r, columns = head dims 32 hb ..
                            const uint32_t base = aDQS + uint32_t(r * 128);
#pragma unroll
                            for (int ch = 0; ch < 8; ++ch)
                                st_shared_v4(base + (uint32_t(ch ^ (r & 7)) << 4), v[hb][4 * ch], v[hb][4 * ch + 1],
                                             v[hb][4 * ch + 2], v[hb][4 * ch + 3]);
                        } else {  // lane = head dim r (box lg), columns = query rows 32 hb ..
                            const uint32_t base = aDQS + uint32_t(lg * 32 * 128) + uint32_t((lane & 3) << 2);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                st_shared_f32(base + uint32_t(e * 128) + (uint32_t((lane >> 2) ^ (e & 7)) << 4), v[hb][e]);
                        }
                    }
                    fence_proxy_async_smem();
                    ok = bar_and(2, 128, ok);
                    if (kOrdered && leader && ok && hb == 0) {
                        // the key tiles with work for this query tile are 0 .. J (whether a key tile has
                        // work for it does not increase with the key tile: J by bisection) and they add
                        // in the order J, J - 1, .., 0, so this add waits until J - jt adds have landed
                        const int qtile = int(i0 / BM);
                        int64_t lo = jt, hi = ntiles - 1;
                        while (lo < hi) {
                            const int64_t mid = (lo + hi + 1) / 2;
                            int q0, n;
                            query_tiles<BM>(a.mask, mid * BN, lq, lkv, &q0, &n);
                            if (n > 0 && q0 <= qtile) lo = mid;
                            else hi = mid - 1;
                        }
                        if (!(ok = wait_count(sem_of(), uint32_t(lo - jt), abort))) flag_abort(abort, a.status);
                        fence_proxy_async_global();
                    }
                    if (leader && ok) {
                        if (D == 64)
                            tma_reduce_add_2d(&p.tm_dq, sDQS, hb * 32, int(row0));
                        else
                            for (int box = 0; box < 4; ++box)
                                tma_reduce_add_2d(&p.tm_dq, sDQS + box * 32 * 128, box * 32, int(row0 + hb * 32));
                        bulk_commit();
                    }
                    if (kOrdered && leader && ok && hb == 1) {
                        // count the previous tile's adds once they have landed (this tile's two groups may
                        // still be in flight); the key tile's last tile is counted at once, so a unit
                        // leaves nothing pending behind it
                        if (pend) {
                            bulk_wait2();
                            fence_proxy_async_global();
                            post(pend);
                            pend = nullptr;
                        }
                        if (it == n_iter - 1) {
                            bulk_wait0();
                            fence_proxy_async_global();
                            post(sem_of());
                        } else {
                            pend = sem_of();
                        }
                    }
                }
            }
            // deterministic mode: this tile's dQ adds land before the next tile's (fixed order)
            if (leader && a.deterministic) bulk_wait0();
        }
        ATTN_END_UNITS
        if (kOrdered && leader) post(nullptr);  // the publishing warp may exit
        if (leader) bulk_wait0();  // the reduce-adds have read the staging buffer (and landed) before the exit
        pdl_trigger();  // the dQ finalize may start launching; it waits for this grid
    }

#undef ATTN_FOR_EACH_UNIT
#undef ATTN_END_UNITS
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::T_COLS);
    }
}

// ===================================================================== host

namespace {

bool map_dqacc(CUtensorMap *m, float *base, int64_t d, int64_t rows, uint32_t box_rows)
{
    auto enc = tmap_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {cuuint64_t(d), cuuint64_t(rows)};
    cuuint64_t strides[1] = {cuuint64_t(d * 4)};
    cuuint32_t box[2] = {32, box_rows};
    cuuint32_t es[2] = {1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

int64_t sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 1;
    return n > 0 ? n : 1;
}

template <class Geo> int64_t max_kv_len(const Geo &g)
{
    int64_t m = 0;
    for (int64_t b = 0; b < g.nseq; ++b) m = g.kv_len(b) > m ? g.kv_len(b) : m;
    return m;
}

// Ordered dQ mode: the adds into each query tile's dQ go in decreasing key-tile order, each one
// waiting until the adds of all higher key tiles have landed.  Units are dealt in decreasing key-tile
// order (longest first among equal ones) to the least loaded CTA, and every CTA takes its units in
// the order dealt, so the key tiles a CTA works on never increase.  A wait then depends only on
// units of higher key tiles, which their CTAs take before any lower one; with every CTA resident
// (cooperative launch) no cycle of waits can form.  Leaves on = 0 when the units do not fit (the API
// refuses such problems).
template <int BM, int BN, class Geo>
void plan_ordered(TcSched &S, const DenseArgs &a, const Geo &g, int64_t units, int64_t ctas)
{
    S.on = 0;
    if (units > kSchedUnits || ctas > kSchedCtas || ctas < 1) return;
    const int64_t nheads = a.nseq * a.h_kv, G = a.h / a.h_kv;
    const int n = int(ctas), nu = int(units);
    static thread_local int32_t cost[kSchedUnits], order[kSchedUnits], cta_of[kSchedUnits];
    for (int u = 0; u < nu; ++u) {
        const int64_t jt = u / nheads, b = (u % nheads) / a.h_kv;
        const int64_t lq = g.q_len(b), lkv = g.kv_len(b);
        int64_t nq = 0;
        if (jt * BN < lkv) {
            const int64_t i_lo = first_query_seeing(a.mask, jt * BN, lq, lkv);
            nq = lq <= 0 || i_lo >= lq ? 0 : (lq + BM - 1) / BM - i_lo / BM;
        }
        cost[u] = jt * BN >= lkv ? 0 : nq > 0 ? int32_t(2 * G * nq + 2) : 1;
        order[u] = u;
    }
    std::stable_sort(order, order + nu, [&](int32_t x, int32_t y) {
        const int64_t jx = x / nheads, jy = y / nheads;
        return jx != jy ? jx > jy : cost[x] > cost[y];
    });
    // least loaded CTA first (lowest index among equals): a min-heap of (load, cta)
    std::priority_queue<std::pair<int64_t, int>, std::vector<std::pair<int64_t, int>>,
                        std::greater<std::pair<int64_t, int>>> heap;
    for (int c = 0; c < n; ++c) heap.push({0, c});
    int cnt[kSchedCtas];
    for (int c = 0; c < n; ++c) cnt[c] = 0;
    for (int k = 0; k < nu; ++k) {
        const int u = order[k];
        cta_of[u] = -1;
        if (cost[u] == 0) continue;  // past the sequence's keys: nothing to do
        const auto top = heap.top();
        heap.pop();
        cta_of[u] = top.second;
        ++cnt[top.second];
        heap.push({top.first + cost[u], top.second});
    }
    S.off[0] = 0;
    for (int c = 0; c < n; ++c) S.off[c + 1] = uint16_t(S.off[c] + cnt[c]);
    for (int c = 0; c < n; ++c) cnt[c] = S.off[c];
    for (int k = 0; k < nu; ++k) {
        const int u = order[k];
        if (cta_of[u] >= 0) S.unit[cnt[cta_of[u]]++] = uint16_t(u);
    }
    S.on = 1;
}

// Assigns the work units of a fixed-length batch to `ctas` CTAs.  A unit's cost is its query tiles
// plus one for its start (loading K / V, the pipeline refill, the dK / dV epilogue), in half tiles;
// units without work cost one (they write zero dK / dV rows).  Two plans: greedy (each unit,
// longest first, to the least loaded CTA) and bin packing, first fit decreasing (with a capacity
// starting at the mean load per CTA, at least the largest unit, units longest first go to the
// first CTA they fit in; the capacity grows until ctas CTAs suffice).  The packing finds the
// balanced groupings of the causal workloads' regular unit sizes that greedy misses by up to a
// tile; it is used when its makespan is at least 3 % shorter.  Each CTA takes its units longest
// first.  The plan of the last shape is kept
// (planning is host work on every call).  Varlen batches take only the head-local plan below, when
// its makespan is within 5 % of the snake order's; otherwise, in the split deterministic mode or
// when the plan does not fit, on = 0 (snake order).
template <int BM, int BN, class Geo>
void plan_units(TcSched &S, const DenseArgs &a, const Geo &g, int64_t units, int64_t ctas)
{
    S.on = 0;
    if (a.ordered) {
        plan_ordered<BM, BN>(S, a, g, units, ctas);
        return;
    }
    constexpr bool packed = IsPacked<Geo>::value;
    if (a.deterministic || units > kSchedUnits || ctas > kSchedCtas || ctas < 1) return;
    struct Key {
        int64_t nseq, h, h_kv, s_q, s_kv, units, ctas;
        int mask;
        uint64_t lens;  // packed batches: a hash of the sequence lengths
        bool operator==(const Key &o) const
        {
            return nseq == o.nseq && h == o.h && h_kv == o.h_kv && s_q == o.s_q && s_kv == o.s_kv && units == o.units &&
                   ctas == o.ctas && mask == o.mask && lens == o.lens;
        }
    };
    uint64_t lens = 1469598103934665603ull;  // FNV-1a over the (query, key) lengths
    if (packed)
        for (int64_t b = 0; b < a.nseq; ++b)
            for (const int64_t l : {g.q_len(b), g.kv_len(b)}) {
                lens ^= uint64_t(l);
                lens *= 1099511628211ull;
            }
    static thread_local Key last_key = {-1, 0, 0, 0, 0, 0, 0, 0, 0};
    static thread_local TcSched last_plan;
    const Key key = {a.nseq, a.h, a.h_kv, g.q_len(0), g.kv_len(0), units, ctas, a.mask, lens};
    if (key == last_key) {
        S = last_plan;
        return;
    }
    const int64_t nheads = a.nseq * a.h_kv, G = a.h / a.h_kv;
    const int n = int(ctas), nu = int(units);
    static thread_local int32_t cost[kSchedUnits], order[kSchedUnits], cta_of[kSchedUnits];
    int64_t load[kSchedCtas];
    int64_t total = 0, biggest = 0;
    for (int u = 0; u < nu; ++u) {
        const int64_t jt = u / nheads, b = (u % nheads) / a.h_kv;
        const int64_t lq = g.q_len(b), lkv = g.kv_len(b);
        int64_t nq = 0;
        if (jt * BN < lkv) {
            const int64_t i_lo = first_query_seeing(a.mask, jt * BN, lq, lkv);
            nq = lq <= 0 || i_lo >= lq ? 0 : (lq + BM - 1) / BM - i_lo / BM;
        }
        cost[u] = jt * BN >= lkv ? 0 : nq > 0 ? int32_t(2 * G * nq + 2) : 1;
        order[u] = u;
        total += cost[u];
        biggest = cost[u] > biggest ? cost[u] : biggest;
    }
    std::stable_sort(order, order + nu, [&](int32_t x, int32_t y) { return cost[x] > cost[y]; });
    // greedy: each unit, longest first, to the least loaded CTA
    static thread_local int32_t greedy_of[kSchedUnits];
    int64_t greedy_max = 0;
    {
        for (int c = 0; c < n; ++c) load[c] = 0;
        for (int k = 0; k < nu; ++k) {
            const int u = order[k];
            greedy_of[u] = -1;
            if (cost[u] == 0) continue;
            int c = 0;
            for (int d = 1; d < n; ++d)
                if (load[d] < load[c]) c = d;
            greedy_of[u] = c;
            load[c] += cost[u];
            greedy_max = load[c] > greedy_max ? load[c] : greedy_max;
        }
    }
    int64_t cap = (total + n - 1) / n;
    cap = cap > biggest ? cap : biggest;
    for (;; ++cap) {
        int used = 0;
        bool fits = true;
        for (int k = 0; k < nu && fits; ++k) {
            const int u = order[k];
            cta_of[u] = -1;
            if (cost[u] == 0) continue;  // past the keys: nothing to do
            int c = 0;
            while (c < used && load[c] + cost[u] > cap) ++c;
            if (c == used) {
                if (used == n) {
                    fits = false;
                    break;
                }
                load[used++] = 0;
            }
            cta_of[u] = c;
            load[c] += cost[u];
        }
        if (fits) break;
    }
    // the packing is kept only where it shortens the planned makespan clearly
    bool use_ffd = 100 * cap <= 97 * greedy_max;
    int64_t best = use_ffd ? cap : greedy_max;
    // head-local plan, for problems whose inputs and dQ accumulator do not fit in L2: the key tiles of
    // one (sequence, kv head) are paired (jt, n - 1 - jt), equal in cost under a causal mask; pairs
    // go out head by head in full rounds of `ctas` (all rounds but the last full one), so the CTAs
    // running together share a few heads' Q / dO rows and dQ accumulator rows; the remaining units
    // go greedily, longest first, to the least loaded CTA
    static thread_local int32_t local_of[kSchedUnits], local_rank[kSchedUnits], tail[kSchedUnits];
    bool use_local = false;
    const int64_t ws_bytes = (a.t_q * a.h * a.d * 2 + a.t_kv * a.h_kv * a.d) * 2 + a.h * a.t_pad * a.d * 4;
    if (ws_bytes > (int64_t(64) << 20)) {
        // the (sequence, kv head) heads, largest first (packed batches: their lengths differ), each with
        // its key tiles in pairs (jt, n_b - 1 - jt)
        static thread_local int32_t heads[kSchedUnits];
        static thread_local int64_t head_cost[kSchedUnits];
        for (int64_t hd = 0; hd < nheads; ++hd) {
            heads[hd] = int32_t(hd);
            head_cost[hd] = 0;
        }
        for (int u = 0; u < nu; ++u) head_cost[u % nheads] += cost[u];
        std::stable_sort(heads, heads + nheads, [&](int32_t x, int32_t y) { return head_cost[x] > head_cost[y]; });
        int64_t njobs = 0;
        for (int64_t hd = 0; hd < nheads; ++hd) {
            const int64_t nt = (g.kv_len(hd / a.h_kv) + BN - 1) / BN;
            njobs += (nt + 1) / 2;
        }
        const int64_t full = njobs / n > 1 ? njobs / n - 1 : 0;
        for (int c = 0; c < n; ++c) load[c] = 0;
        for (int u = 0; u < nu; ++u) local_of[u] = -1;
        int32_t rank = 0;
        int ntail = 0;
        int64_t job = 0;
        for (int64_t k = 0; k < nheads; ++k) {
            const int64_t head = heads[k];
            const int64_t nt = (g.kv_len(head / a.h_kv) + BN - 1) / BN;
            for (int64_t pj = 0; pj < (nt + 1) / 2; ++pj, ++job) {
                const int64_t ua = pj * nheads + head, ub = (nt - 1 - pj) * nheads + head;
                for (int kk = 0; kk < (ua == ub ? 1 : 2); ++kk) {
                    const int64_t u = kk == 0 ? ua : ub;
                    if (cost[u] == 0) continue;
                    if (job < full * n) {
                        const int c = int(job % n);
                        local_of[u] = c;
                        local_rank[u] = rank++;
                        load[c] += cost[u];
                    } else {
                        tail[ntail++] = int32_t(u);
                    }
                }
            }
        }
        std::stable_sort(tail, tail + ntail, [&](int32_t x, int32_t y) { return cost[x] > cost[y]; });
        for (int k = 0; k < ntail; ++k) {
            const int u = tail[k];
            int c = 0;
            for (int d = 1; d < n; ++d)
                if (load[d] < load[c]) c = d;
            local_of[u] = c;
            local_rank[u] = rank++;
            load[c] += cost[u];
        }
        int64_t local_max = 0;
        for (int c = 0; c < n; ++c) local_max = load[c] > local_max ? load[c] : local_max;
        use_local = 100 * local_max <= 105 * best;
        if (packed) {  // against the snake order packed batches take otherwise
            for (int c = 0; c < n; ++c) load[c] = 0;
            for (int u = 0; u < nu; ++u) {
                const int r = u / n, c = u % n;
                load[(r & 1) ? n - 1 - c : c] += cost[u];
            }
            int64_t snake_max = 0;
            for (int c = 0; c < n; ++c) snake_max = load[c] > snake_max ? load[c] : snake_max;
            use_local = 100 * local_max <= 105 * snake_max;
        }
    }
    if (packed && !use_local) {  // snake order (units running together would add into one long sequence's rows)
        last_plan = S;
        last_key = key;
        return;
    }
    if (use_local)
        for (int u = 0; u < nu; ++u) cta_of[u] = local_of[u];
    else if (!use_ffd)
        for (int u = 0; u < nu; ++u) cta_of[u] = greedy_of[u];
    int cnt[kSchedCtas];
    for (int c = 0; c < n; ++c) cnt[c] = 0;
    for (int u = 0; u < nu; ++u)
        if (cta_of[u] >= 0) ++cnt[cta_of[u]];
    S.off[0] = 0;
    for (int c = 0; c < n; ++c) S.off[c + 1] = uint16_t(S.off[c] + cnt[c]);
    for (int c = 0; c < n; ++c) cnt[c] = S.off[c];
    if (use_local) {  // each CTA's units in the order they were dealt
        std::stable_sort(order, order + nu, [&](int32_t x, int32_t y) {
            const int32_t rx = cta_of[x] >= 0 ? local_rank[x] : INT32_MAX, ry = cta_of[y] >= 0 ? local_rank[y] : INT32_MAX;
            return rx < ry;
        });
    }
    for (int k = 0; k < nu; ++k) {  // each CTA's units longest first (head-local plan: as dealt)
        const int u = order[k];
        if (cta_of[u] >= 0) S.unit[cnt[cta_of[u]]++] = uint16_t(u);
    }
    S.on = 1;
    last_plan = S;
    last_key = key;
}

template <class T, int D, class Geo> cudaError_t run_tc(const DenseArgs &a, const RelArgs *rel, const Geo &g, cudaStream_t s)
{
    using Cfg = TcCfg<D>;
    constexpr bool packed = IsPacked<Geo>::value;
    const int64_t ntiles = (max_kv_len(g) + Cfg::BN - 1) / Cfg::BN;
    if (ntiles == 0) return cudaSuccess;
    TcParams prm;
    prm.a = a;
    if (rel) prm.rel = *rel;
    const int64_t nb = packed ? 1 : a.nseq;
    const int64_t sq = packed ? a.t_q : (a.t_q / (a.nseq ? a.nseq : 1));
    const int64_t skv = packed ? a.t_kv : (a.t_kv / (a.nseq ? a.nseq : 1));
    if (sq > 0 && (!tmap_view16(&prm.tm_q, a.q, a.dtype, D, sq, a.h, nb, Cfg::BM) ||
                   !tmap_view16(&prm.tm_do, a.dO, a.dtype, D, sq, a.h, nb, Cfg::BM)))
        return cudaErrorInvalidValue;
    if (!tmap_view16(&prm.tm_k, a.k, a.dtype, D, skv, a.h_kv, nb, Cfg::BN) ||
        !tmap_view16(&prm.tm_v, a.v, a.dtype, D, skv, a.h_kv, nb, Cfg::BN) ||
        !tmap_view16(&prm.tm_dk, a.dK, a.dtype, D, skv, a.h_kv, nb, Cfg::BN) ||
        !tmap_view16(&prm.tm_dv, a.dV, a.dtype, D, skv, a.h_kv, nb, Cfg::BN))
        return cudaErrorInvalidValue;
    if (sq > 0 && !map_dqacc(&prm.tm_dq, a.dqacc, D, int64_t(a.n_part) * a.h * a.t_pad, Cfg::DQ_BOX_ROWS))
        return cudaErrorInvalidValue;
    if (sq == 0) prm.tm_q = prm.tm_do = prm.tm_dq = prm.tm_k;  // never used: no query tiles
    auto k = rel ? (a.ordered ? dense_bwd_tc_kernel<T, D, Geo, true, true> : dense_bwd_tc_kernel<T, D, Geo, false, true>)
                 : (a.ordered ? dense_bwd_tc_kernel<T, D, Geo, true, false> : dense_bwd_tc_kernel<T, D, Geo, false, false>);
    const int smem = rel ? Cfg::SMEM_ALLOC_BIAS : Cfg::SMEM_ALLOC;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (rel) prm.a.h_kv *= rel->shares;  // (the tensor maps have the real ones)
    prm.a.tc_units = (a.deterministic ? a.n_part : ntiles) * a.nseq * prm.a.h_kv;
    if (prm.a.tc_units > INT32_MAX) return cudaErrorInvalidValue;  // the kernel splits units in 32 bits
    const int64_t units = prm.a.tc_units < sm_count() ? prm.a.tc_units : sm_count();
    plan_units<Cfg::BM, Cfg::BN>(prm.sched, prm.a, g, prm.a.tc_units, units);
    if (a.ordered && !prm.sched.on) return cudaErrorNotSupported;  // the waits need the planned order
    // ordered dQ mode waits across CTAs: a cooperative launch puts all of them on the GPU at once
    return launch_kernel_ex(k, dim3(unsigned(units)), dim3(Cfg::THREADS + (a.ordered ? 32 : 0)), smem, s, true,
                            a.ordered != 0, prm, g);
}

template <class Geo> cudaError_t dispatch(const DenseArgs &a, const RelArgs *rel, const Geo &g, cudaStream_t s)
{
    if (a.d == 64)
        return a.dtype == ATTN_F16 ? run_tc<__half, 64>(a, rel, g, s) : run_tc<__nv_bfloat16, 64>(a, rel, g, s);
    return a.dtype == ATTN_F16 ? run_tc<__half, 128>(a, rel, g, s) : run_tc<__nv_bfloat16, 128>(a, rel, g, s);
}

}  // namespace

cudaError_t launch_dense_bwd_main(const DenseArgs &a, const FixedGeo &g, cudaStream_t s, const RelArgs *rel)
{
    return dispatch(a, rel, g, s);
}
cudaError_t launch_dense_bwd_main(const DenseArgs &a, const PackedGeo &g, cudaStream_t s, const RelArgs *rel)
{
    return dispatch(a, rel, g, s);
}

}  // namespace attn
