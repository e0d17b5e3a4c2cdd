// paged_chunk.cu -- tensor-core attention of chunks of new tokens over a paged key /
// value cache, 16-bit or e4m3, for sm_103a: tcgen05 MMAs with TMEM accumulators, pages by
// TMA.
//
//   s_ij = scale q_i.k_j,  O = softmax(s) V  over the keys j <= position of i (or all)
//
// Persistent, one CTA an SM, each with an even share of all keys of all units
// (paged_sched.cuh).  A unit is (sequence, kv head, query tile): the rows are the new
// tokens with all query heads of the kv head, so a group's keys are read once for its
// heads.  Query rows are the MMA M dimension and the TMEM lanes:
//   S = Q K^T      M=128 (rows) N=64 (keys) K=D   A=Q (smem, K-major) B=K (smem, K-major)
//   O += P V       M=128        N=D         K=64  A=P (TMEM, 16-bit)  B=V (smem, MN-major)
// Two softmax warpgroups work beside each other, each on 128 rows and 64 keys a step,
// with its own S (two buffers), running maximum, sum and O accumulator; a thread owns a
// row.  kSplit, for chunks that fit 128 rows: a unit is 128 rows and the groups take
// turns at the stages of 64 keys; their O are added at its end.
// P overwrites the S it came from; the tensor pipe runs the MMAs in the order they were
// issued, so S of step j + 2 follows O += P V of step j into the same columns without a wait.
//
// A stage is one to eight pages (or part of one).  A lane of the producing warp looks up a
// page, a stage ahead, and issues its TMA boxes.  16 bits: stages of 128 keys, 64 elements x page
// rows with the 128-byte swizzle, straight to where the MMA reads them (stages of 64: 930 us for 905,
// each wait of the MMA thread takes it 100 cycles).  e4m3: stages of 64, rows of d bytes to a
// ring of their own, with their scales (4-byte asynchronous copies), from which a warpgroup
// makes 16-bit numbers in the swizzled layout (a lane a row, so that neither side has bank
// conflicts: 1512 -> 1445 us).  Keys unscaled, of the queries' type (e4m3 numbers are
// 16-bit numbers exactly); their scales multiply S's columns.
// Values as half-precision numbers times f, where their scale is 2^E f, |f| in [1, 2): number,
// factor and product in one multiplication a pair, the latter two rounded by at most half a step of that
// type.  2^E goes into the weight of its key: P' = exp2(x + E - m) with m over x + E, so that O and l keep one
// reference, which is what the row's keys weigh with their scales; l takes P' 2^-E.  (One E for a stage, that of its
// largest scale, needs two numbers less a key in the softmax and takes 1220 us for 1360, but lets a key of no weight,
// or one that a row does not see, take the bits of the others.  One E where the scales are near one another, and each its
// own elsewhere: 1410 and more, in one loop or two; the code of both is too much for the instruction cache.)
// A page id out of range reads as zeros.
//
// Bound: 16 bits, the chain S -> softmax -> P -> O of a group, 2000 cycles for 64 keys and 256
// rows against 1260 of MMAs (2048 tokens on 32768, 32 / 8 heads of 128: 905 us, 0.65 of the measured tensor
// rate).  e4m3, 1360 us: the converting warps share the issue slots with the softmax, whose chain has the scales
// of 64 keys to read, and shared memory's bandwidth with the MMAs.  Measured and not taken (16 bits, and e4m3 where that had
// one E a stage and 1225 us): 128 keys a step with one S a group, whose MMAs run at the full rate (M=128 N=64 from shared
// memory reads 128 rows of Q for 64 of K: two thirds), 876 and 1470 us; the same with two threads a row, 865 and 1900; a
// warp that tells the MMA thread its steps, 913 and 1290.
//
// A row's reference maximum m is raised only when a step's maximum exceeds it by more
// than 8 (log2 units), and then l and the row of O in TMEM are scaled by exp2(m_old - m_new):
// P = exp2(x - m) <= 2^8 fits both 16-bit types.  P is rounded to the 16-bit type for
// the second product, whose operands are of that type, after its sum l is taken.  A row
// that sees no key has O = 0 and LSE = +inf.  Values from the sequence's end on meet P = 0 and
// may be anything: they are set to zero in shared memory first.
//
// Roles: warp 0 loads Q and K, warp 2 V, warp 1 issues the MMAs, warps 4..7 and 8..11
// are the softmax warpgroups, warps 12..15 (e4m3) convert K and V.  Every barrier wait is
// bounded; a wait that runs out sets ATTN_DEV_TIMEOUT and the CTA skips the rest of its
// work, drains its copies and MMAs, and frees its TMEM.
#include <type_traits>

#include "paged.h"
#include "paged_sched.cuh"
#include "sm103.cuh"
#include "tc_util.cuh"
#include "tmap.h"

namespace attn {
using namespace sm103;
using namespace tc;
using namespace paged;

template <int D, bool kEight, bool kSplit> struct ChunkCfg {
    static constexpr int BM = 128, HN = 64;          // rows of a group, keys of a stage (and of a step)
    static constexpr int SN = kEight ? 64 : 128;     // keys of a K or V stage
    static constexpr int NS = kEight ? (D == 64 ? 4 : 3) : (D == 64 ? 4 : 2);  // K and V ring stages
    static constexpr int NE = !kEight ? 0 : D == 64 ? 8 : kSplit ? 5 : 3;      // e4m3 ring stages
    static constexpr int NKS = 8;                    // key scales: read until two steps behind S
    static constexpr int THREADS = kEight ? 512 : 384;
    static constexpr int TILE_BYTES = BM * D * 2;    // 128 query rows
    static constexpr int STAGE_BYTES = SN * D * 2;   // a K or V stage
    static constexpr int E_BYTES = HN * D;           // and as e4m3
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + (kSplit ? 1 : 2) * TILE_BYTES;
    static constexpr int OFF_V = OFF_K + NS * STAGE_BYTES;
    static constexpr int OFF_E = OFF_V + NS * STAGE_BYTES;    // [NE][keys, values]
    static constexpr int OFF_ES = OFF_E + NE * 2 * E_BYTES;   // [NE][keys, values][64] scales
    static constexpr int OFF_BAR = OFF_ES + NE * 2 * HN * 4;
    static constexpr int OFF_MISC = OFF_BAR + 80 * 8;
    static constexpr int OFF_ML = OFF_MISC + 64;              // [2 groups][m, l][128 rows] floats
    static constexpr int OFF_KS = OFF_ML + 2 * 2 * 128 * 4;   // [NKS][key scale, E, 2^-E][64] floats
    static constexpr int OFF_RANGE = OFF_KS + (kEight ? NKS * 3 * HN * 4 : 0);  // scratch of the range, then the range
    static constexpr int SMEM = OFF_RANGE + 320;
    // at least half the SM's shared memory: one CTA, which holds all of the TMEM, runs per SM
    static constexpr int SMEM_ALLOC = SMEM + 1024 > 116 * 1024 ? SMEM + 1024 : 116 * 1024;
    static constexpr int T_S = 0, T_O = 256;  // S (and P) of group g, step parity b at T_S + 128 g + 64 b, O at T_O + D g
    static constexpr int T_COLS = 512;
    static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");
    static_assert(3 + 4 * NS + 12 + NKS + 4 * NE <= 80, "barrier slots");
    static_assert(!kEight || NKS >= NS + 4, "key scale slots");
    static_assert((THREADS / 32 + 12) * 8 <= 256 && sizeof(Range) <= 64, "range scratch");
};

// What a unit's start and end take, in keys; pieces of fewer than kLeast keys are avoided; a share worth a start.
constexpr int kChunkCost = 256, kChunkLeast = 512, kChunkShare = 1024;

struct ChunkParams {
    CUtensorMap tm_q, tm_k, tm_v;
    PagedAttnArgs a;
    int tokens;  // new tokens of 128 rows
};

namespace {

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// mbar_wait out of line, for the MMA thread: its waits are nearly always over when it comes.
__device__ __noinline__ bool chunk_wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort)
{
    return mbar_wait(bar, parity, abort);
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

// (volatile: read where it is used, not held in registers)
__device__ __forceinline__ float4 lds4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// two e4m3 numbers as half-precision ones, and as numbers of type T
__device__ __forceinline__ uint32_t half_pair(uint32_t e4m3x2)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(e4m3x2)));
    return h;
}
template <class T> __device__ __forceinline__ uint32_t widen(uint32_t e4m3x2)
{
    const uint32_t h = half_pair(e4m3x2);
    if (std::is_same<T, __half>::value) return h;
    const float2 y = unpack2<__half>(h);
    return pack2<T>(y.x, y.y);
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b)
{
    uint32_t c;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

}  // namespace

template <class T, int D, bool kEight, bool kSplit>
__global__ void __launch_bounds__(ChunkCfg<D, kEight, kSplit>::THREADS, 1) paged_chunk_kernel(const __grid_constant__ ChunkParams p)
{
    using Cfg = ChunkCfg<D, kEight, kSplit>;
    constexpr int BM = Cfg::BM, HN = Cfg::HN, SN = Cfg::SN, NS = Cfg::NS, NE = Cfg::NE, NKS = Cfg::NKS;
    constexpr int kType = std::is_same<T, __half>::value ? 0 : 1;
    using P16 = typename std::conditional<kEight, __half, T>::type;  // type of P and V

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::OFF_BAR);
    uint64_t *q_full = bars + 0, *q_empty = bars + 1, *drain = bars + 2;
    uint64_t *k_full = bars + 3, *k_empty = k_full + NS, *v_full = k_empty + NS, *v_empty = v_full + NS;
    uint64_t *s_full = v_empty + NS;       // [2 groups][2 buffers] S is written
    uint64_t *p_full = s_full + 4;         // [2 groups][2 buffers] P is written (and O rescaled if needed)
    uint64_t *o_prev = s_full + 8;         // [2 groups] O += P V of a unit's last step but one has completed ...
    uint64_t *o_last = s_full + 10;        // [2 groups] ... and of its last step
    uint64_t *ks_full = s_full + 12;       // [NKS] a stage's key scales are written
    uint64_t *e_full = ks_full + NKS, *e_empty = e_full + 2 * NE;  // [keys, values][NE] e4m3 stages
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::OFF_MISC);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + Cfg::OFF_MISC + 8);
    volatile int *bad_page = reinterpret_cast<volatile int *>(smem + Cfg::OFF_MISC + 12);
    const PagedAttnArgs &a = p.a;
    const PagedCache &cache = a.cache;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    pdl_trigger();
    if (threadIdx.x == 0) {
        *abort = 0;
        *bad_page = 0;
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(drain, 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&k_full[s], kEight ? 4 : 1);
            mbar_init(&k_empty[s], 1);
            mbar_init(&v_full[s], kEight ? 4 : 1);
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
        for (int k = 0; k < NKS; ++k) mbar_init(&ks_full[k], 4);
        for (int k = 0; k < 2 * NE; ++k) {
            mbar_init(&e_full[k], 1 + 32);  // the boxes, and the scales of each lane
            mbar_init(&e_empty[k], 4);
        }
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, Cfg::T_COLS);

    // ---- this CTA's share, and a piece of it
    const int G = a.h / a.h_kv;
    const Sched<kChunkCost> sched = {a.seqs, kSplit ? p.tokens : 2 * p.tokens, a.h_kv, a.causal};
    bool bad = false;
    Range *range = reinterpret_cast<Range *>(smem + Cfg::OFF_RANGE + 256);
    {
        const Range r = sched.template range<Cfg::THREADS, 2 * HN, kChunkLeast, kChunkShare>(
            blockIdx.x, gridDim.x, reinterpret_cast<int64_t *>(smem + Cfg::OFF_RANGE), &bad);
        if (threadIdx.x == 0) *range = r;
    }
    if (bad && blockIdx.x == 0) *bad_page = 1;  // (one CTA reports the lengths)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint8_t *sQ = smem + Cfg::OFF_Q;
    auto sK = [&](int s) { return smem + Cfg::OFF_K + s * Cfg::STAGE_BYTES; };
    auto sV = [&](int s) { return smem + Cfg::OFF_V + s * Cfg::STAGE_BYTES; };
    // steps of each group, the longer of them, stages
    struct Steps {
        int s0, s1, n, stages;
    };
    auto steps_of = [&](const Walk<kChunkCost> &w) -> Steps {
        Steps st;
        if (kSplit) {
            st.s0 = st.s1 = st.n = (w.k1 - w.k0 + 2 * HN - 1) / (2 * HN);
            st.stages = kEight ? 2 * st.n : st.n;
            return st;
        }
        auto of = [&](int grp) -> int {
            const int first = w.t * sched.tokens + grp * p.tokens;
            if (first >= w.u.m) return 0;
            int seen = w.u.len;
            if (a.causal) seen += (first + p.tokens < w.u.m ? first + p.tokens : w.u.m) - w.u.m;
            if (seen > w.k1) seen = w.k1;
            return seen > w.k0 ? (seen - w.k0 + HN - 1) / HN : 0;
        };
        st.s0 = of(0);
        st.s1 = of(1);
        st.n = st.s0 > st.s1 ? st.s0 : st.s1;
        st.stages = kEight ? st.n : (st.n + 1) / 2;
        return st;
    };
    // stage of a step's keys, from the piece's first on, and which half of it (e4m3: it has but one)
    auto stage_of = [](int j, int grp) { return kEight ? (kSplit ? 2 * j + grp : j) : kSplit ? j : j >> 1; };
    auto half_of = [](int j, int grp) { return kEight ? 0 : kSplit ? grp : j & 1; };

    // (e4m3: 512 threads are launched with 128 registers each; the warpgroups' shares add up to that.  The MMA thread's
    // count: 2048 tokens on 32768 with 112 registers, and 152 for the softmax, 1390 us, 120: 1381, 128: 1361)
    constexpr uint32_t kRegsIssue = 128, kRegsSoftmax = 144, kRegsConvert = 96;
    static_assert(kRegsIssue + 2 * kRegsSoftmax + kRegsConvert == 4 * 128, "register shares");
    if (warp < 4) {
        if (kEight) regs_decrease<kRegsIssue>();
        if (warp == 0 || warp == 2) {
            // ============================================= producers: Q and K (warp 0), V (warp 2)
            const bool isk = warp == 0;
            constexpr int NR = kEight ? NE : NS;  // ring
            uint64_t *full = kEight ? e_full + (isk ? 0 : NE) : isk ? k_full : v_full;
            uint64_t *empty = kEight ? e_empty + (isk ? 0 : NE) : isk ? k_empty : v_empty;
            const CUtensorMap *tm = isk ? &p.tm_k : &p.tm_v;
            const int in_page = (1 << cache.shift) - 1, pr = 1 << cache.shift < SN ? 1 << cache.shift : SN;  // keys of a box
            const int boxes = SN / pr;
            if (lane == 0) {
                prefetch_tmap(tm);
                if (isk) prefetch_tmap(&p.tm_q);
            }
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {  // the whole warp
                if (lane == 0 && !(ok = mbar_wait(bar, parity, abort))) flag_abort(abort, nullptr);
                ok = __shfl_sync(0xffffffffu, ok, 0);
            };
            uint32_t n_stage = 0, s = 0, par = 1, n_unit = 0;  // stages so far, ring position and phase, pieces with keys
            Walk<kChunkCost> w(sched, *range);
            while (ok && w.next()) {
                const Steps st = steps_of(w);
                if (st.n == 0) continue;
                const int32_t *table = a.seqs.table + w.n * a.seqs.table_stride;
                // page of this lane's box of the stage at key k (-1: none of this piece)
                auto page_of = [&](int k) -> int {
                    const int key = k + lane * pr;
                    return lane < boxes && key < w.k1 ? table[key >> cache.shift] : -1;
                };
                int id = page_of(w.k0);
                if (isk) {
                    if (n_unit > 0) wait(q_empty, (n_unit - 1) & 1);
                    if (!ok) break;
                    ++n_unit;
                    const int n = !kSplit && st.s1 ? 2 : 1;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(q_full, n * p.tokens * G * D * 2);
                        for (int k = 0; k < n; ++k) {
                            const int tok = w.t * sched.tokens + k * p.tokens;
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_4d(sQ + k * Cfg::TILE_BYTES + c * BM * 128, &p.tm_q, q_full, c * 64, w.x * G,
                                            a.seqs.cu ? w.u.first + tok : tok, a.seqs.cu ? 0 : w.n);
                        }
                    }
                }
                for (int j = 0; j < st.stages; ++j) {
                    const int k0 = w.k0 + j * SN, next = page_of(k0 + SN);
                    if (n_stage >= uint32_t(NR)) wait(&empty[s], par);
                    if (!ok) break;
                    ++n_stage;
                    const int key = k0 + lane * pr;
                    const bool good = id >= 0 && id < cache.n_pages;
                    if (!good && lane < boxes && key < w.k1) *bad_page = 1;
                    if (lane == 0) mbar_arrive_expect_tx(&full[s], kEight ? Cfg::E_BYTES : Cfg::STAGE_BYTES);
                    __syncwarp();
                    if (lane < boxes) {
                        const int page = good ? id : cache.none;  // (out of range: zeros)
                        if (kEight) {
                            tma_load_4d(smem + Cfg::OFF_E + (2 * s + !isk) * Cfg::E_BYTES + lane * pr * D, tm, &full[s], 0,
                                        key & in_page, w.x, page);
                        } else {
                            uint8_t *dst = (isk ? sK(s) : sV(s)) + lane * pr * 128;
                            for (int c = 0; c < D / 64; ++c)
                                tma_load_4d(dst + c * SN * 128, tm, &full[s], c * 64, key & in_page, w.x, page);
                        }
                    }
                    if (kEight) {  // scales of keys lane and lane + 32; 0 behind the piece's end
                        const float *scale = isk ? cache.k_scale : cache.v_scale;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int x = lane + 32 * e, pg = __shfl_sync(0xffffffffu, good ? id : -1, x / pr);
                            const bool on = pg >= 0 && k0 + x < w.k1;
                            copy4(smem_u32(smem + Cfg::OFF_ES) + ((2 * s + !isk) * HN + x) * 4,
                                  on ? scale + pg * cache.sc_sp + (w.x * cache.sc_sh + ((k0 + x) & in_page) * cache.sc_ss) : scale, on);
                        }
                        copies_arrive(&full[s]);
                    }
                    id = next;
                    if (++s == NR) {
                        s = 0;
                        par ^= 1;
                    }
                }
            }
            if (lane == 0) {  // a CTA does not end before its copies, whoever may have given up
                volatile int never = 0;
                if (isk && n_unit > 0) mbar_wait(q_full, (n_unit - 1) & 1, &never, 100000000ull);
                for (uint32_t j = n_stage > uint32_t(NR) ? n_stage - NR : 0; j < n_stage; ++j)
                    mbar_wait(&full[j % NR], (j / NR) & 1, &never, 100000000ull);
            }
            __syncwarp();
        } else if (warp == 1 && elect_one()) {
            // ============================================= MMA issuer
            // One thread, and the time it takes between two MMAs is the tensor pipe's to lose: descriptors are
            // one add from values kept in registers, a piece starts at buffer 0 so that buffers are constants of the
            // (two-step) loop body, and phases are bits that flip with each wait.
            constexpr uint32_t idS = idesc_f16(128, HN, kType, 0, 0);
            constexpr uint32_t idO = idesc_f16(128, D, kEight ? 0 : kType, 0, 1);
            constexpr uint32_t STAGE = Cfg::STAGE_BYTES / 16, QROWS = Cfg::TILE_BYTES / 16;  // in descriptor units
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (ok && !mbar_test_wait(bar, parity) && !(ok = chunk_wait_slow(bar, parity, abort))) flag_abort(abort, nullptr);
                tc_fence_after();
            };
            const uint64_t kQ = desc_kmaj(smem_u32(sQ), BM, 0), kK = desc_kmaj(smem_u32(sK(0)), SN, 0);
            const uint64_t mV = desc_mn(smem_u32(sV(0)), SN, 0);
            uint32_t ks = 0, vs = 0, k_par = 0, v_par = 0, q_par = 0, p_par = 0;  // p_par: bit 2 group + buffer
            Walk<kChunkCost> w(sched, *range);
            while (w.next()) {
                const Steps st = steps_of(w);
                if (st.n == 0) continue;
                wait(q_full, q_par);
                q_par ^= 1;
                const int n_steps = st.n, steps0 = st.s0, steps1 = st.s1;
                // S of step j, then O += P V of step j - 1 (buffer sb ^ 1).  S of step j goes where P of step
                // j - 2 was, whose product was issued a round ago
                auto k_next = [&]() {
                    if (ok) mma_commit(&k_empty[ks]);
                    if (++ks == NS) {
                        ks = 0;
                        k_par ^= 1;
                    }
                };
                auto v_next = [&]() {
                    if (ok) mma_commit(&v_empty[vs]);
                    if (++vs == NS) {
                        vs = 0;
                        v_par ^= 1;
                    }
                };
                auto round = [&](int j, auto sb_tag) {
                    constexpr int sb = decltype(sb_tag)::value, xb = sb ^ 1;
                    // a stage is waited for by its first user and released by its last: a group of its own (e4m3, kSplit),
                    // both groups of a step, or both groups of two steps
                    constexpr bool kOwn = kEight && kSplit, kTwo = !kEight && !kSplit;
                    if (j < n_steps) {
                        if (!kOwn && (!kTwo || sb == 0)) wait(&k_full[ks], k_par);
#pragma unroll
                        for (int grp = 0; grp < 2; ++grp) {
                            if (j >= (grp ? steps1 : steps0)) continue;
                            if (kOwn) wait(&k_full[ks], k_par);
                            if (ok) {
                                const uint64_t dk = kK + ks * STAGE + half_of(sb, grp) * (HN * 128 / 16), dq = kQ + (kSplit ? 0 : grp * QROWS);
#pragma unroll
                                for (int kk = 0; kk < D / 16; ++kk)
                                    mma_f16_ss(tmem + Cfg::T_S + grp * 128 + sb * 64, kmaj_step(dq, BM, kk), kmaj_step(dk, SN, kk), idS,
                                               kk > 0);
                                mma_commit(&s_full[grp * 2 + sb]);
                            }
                            if (kOwn) k_next();
                        }
                        if (!kOwn && (!kTwo || sb || j == n_steps - 1)) k_next();
                        if (ok && j == n_steps - 1) mma_commit(q_empty);
                    }
                    if (j > 0) {
                        const int x = j - 1;
                        if (!kOwn && (!kTwo || xb == 0)) wait(&v_full[vs], v_par);
#pragma unroll
                        for (int grp = 0; grp < 2; ++grp) {
                            const int steps = grp ? steps1 : steps0;
                            if (x >= steps) continue;
                            if (kOwn) wait(&v_full[vs], v_par);
                            wait(&p_full[grp * 2 + xb], p_par >> (grp * 2 + xb) & 1);
                            p_par ^= 1u << (grp * 2 + xb);
                            if (ok) {
                                const uint64_t dv = mV + vs * STAGE + half_of(xb, grp) * (HN / 16) * 128;
#pragma unroll
                                for (int kk = 0; kk < HN / 16; ++kk)
                                    mma_f16_ts(tmem + Cfg::T_O + grp * D, tmem + Cfg::T_S + grp * 128 + xb * 64 + kk * 8,
                                               mn_step(dv, kk), idO, x > 0 || kk > 0);
                                // (earlier ones are behind S of step x + 2)
                                if (x >= steps - 2) mma_commit(x == steps - 1 ? &o_last[grp] : &o_prev[grp]);
                            }
                            if (kOwn) v_next();
                        }
                        if (!kOwn && (!kTwo || xb || x == n_steps - 1)) v_next();
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
    } else if (warp < 12) {
        // ================================================= softmax and epilogue (warps 4..11)
        if (kEight) regs_increase<kRegsSoftmax>();
        const int grp = (warp >> 2) - 1, qd = warp & 3;  // the group; TMEM lane quadrant
        const uint32_t lane_addr = uint32_t(qd * 32) << 16;
        const int r = qd * 32 + lane;
        // (scores in log2 units are c times S; a scale below zero turns S's sign; c > 0, so that a masked -inf stays one)
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-100f);
        const uint32_t tO = tmem + lane_addr + Cfg::T_O + grp * D;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok && !(ok = mbar_wait(bar, parity, abort))) flag_abort(abort, nullptr);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        };
        // stages, and phases of o_prev and o_last before this piece; phase parity of the S buffers
        uint32_t k_base = 0, n_prev = 0, n_last = 0, s_par = 0;
        int4 named0 = unit_name(0, 0, 0, kNone), named1 = named0;
        const int row_tok = r / G, row_head = r - row_tok * G;

        Walk<kChunkCost> w(sched, *range);
        while (w.next()) {
            const Steps st = steps_of(w);
            const int steps = grp ? st.s1 : st.s0;
            const int ti = w.t * sched.tokens + (kSplit ? 0 : grp * p.tokens) + row_tok;  // the row's new token
            const bool row_ok = row_tok < p.tokens && ti < w.u.m;
            // step j's first key is kfirst + j kstep, of which this row sees those up to kmax
            constexpr int kstep = kSplit ? 2 * HN : HN;
            const int kfirst = w.k0 + (kSplit ? grp * HN : 0);
            const int kmax = !row_ok ? -1 : a.causal ? w.u.len - w.u.m + ti : w.u.len - 1;
            float m_ref = -INFINITY, l = 0.f, l_lost = 0.f;  // l: sum of P, and what its additions have rounded off

            for (int j = 0; j < steps; ++j) {
                const int sb = j & 1;
                const uint32_t tS = tmem + lane_addr + Cfg::T_S + grp * 128 + sb * 64;
                const int lim = kmax - kfirst - j * kstep;  // columns <= lim are visible
                const bool whole = __all_sync(0xffffffffu, lim >= HN - 1);
                const uint32_t stage = k_base + stage_of(j, grp);
                if (kEight) wait(&ks_full[stage % NKS], (stage / NKS) & 1);
                wait(&s_full[grp * 2 + sb], s_par >> sb & 1);
                s_par ^= 1u << sb;
                // the row of S (e4m3: in log2 units, plus E), masked, and its maximum
                float x[HN];
                float mx = -INFINITY;
                const uint32_t scales = smem_u32(smem) + Cfg::OFF_KS + stage % NKS * (3 * HN * 4);
                if (ok) {
                    uint32_t v[2][32];
                    tmem_ld32(tS, v[0]);
                    tmem_ld32(tS + 32, v[1]);
                    tmem_ld_wait_regs(v[0]);
                    tmem_ld_wait_regs(v[1]);
#pragma unroll
                    for (int e = 0; e < HN; ++e) x[e] = __uint_as_float(v[e / 32][e % 32]);
                    if (kEight) {
#pragma unroll
                        for (int e = 0; e < HN; e += 4) {
                            const float4 q = lds4(scales + e * 4), ve = lds4(scales + (HN + e) * 4);
                            const float2 y0 = fma2(make_float2(x[e], x[e + 1]), make_float2(q.x, q.y), make_float2(ve.x, ve.y));
                            const float2 y1 = fma2(make_float2(x[e + 2], x[e + 3]), make_float2(q.z, q.w), make_float2(ve.z, ve.w));
                            x[e] = y0.x; x[e + 1] = y0.y; x[e + 2] = y1.x; x[e + 3] = y1.y;
                        }
                    } else if (a.scale < 0.f) {
#pragma unroll
                        for (int e = 0; e < HN; ++e) x[e] = -x[e];
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
                    if (!kEight) mx *= c;
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
                                    uint32_t y[8];
#pragma unroll
                                    for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(__uint_as_float(v[e0 + e]) * f);
                                    tmem_st8(tO + o0 + e0, y);
                                }
                            }
                            tmem_st_wait();
                        }
                    }
                    if (need) {
                        l *= f;
                        l_lost *= f;
                        m_ref = m_new;
                    }
                }
                // P = exp2(x - m) over the columns S was read from
                if (ok) {
                    const float neg = m_ref == -INFINITY ? 0.f : -m_ref;  // no visible key yet: every P is 0
                    const float2 neg2 = make_float2(neg, neg), c2 = make_float2(c, c);
                    float2 l2 = make_float2(0.f, 0.f);
                    float4 inv = make_float4(1.f, 1.f, 1.f, 1.f);  // e4m3: 2^-E of four keys
#pragma unroll
                    for (int e0 = 0; e0 < HN; e0 += 16) {
                        uint32_t y[8];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 z = make_float2(x[e0 + e], x[e0 + e + 1]);
                            const float2 t = kEight ? add2(z, neg2) : fma2(z, c2, neg2);
                            const float2 q = make_float2(ex2(t.x), ex2(t.y));
                            if (kEight) {
                                if (e % 4 == 0) inv = lds4(scales + (2 * HN + e0 + e) * 4);
                                l2 = fma2(q, e % 4 ? make_float2(inv.z, inv.w) : make_float2(inv.x, inv.y), l2);
                            } else {
                                l2 = add2(l2, q);
                            }
                            y[e / 2] = pack2<P16>(q.x, q.y);
                        }
                        tmem_st8(tS + e0 / 2, y);
                    }
                    // a step's sum is added with what earlier additions lost: thousands of weights far below the largest
                    // would each be rounded away
                    const float add = l2.x + l2.y - l_lost, sum = l + add;
                    l_lost = sum - l - add;
                    l = sum;
                    tmem_st_wait();
                    if (!kEight && kfirst + j * kstep + HN > w.u.len) {  // values from the sequence's end on
                        const uint32_t s = stage % NS;
                        wait(&v_full[s], (stage / NS) & 1);
                        const int row = half_of(j, grp) * HN + r;  // of the stage
                        if (r < HN && kfirst + j * kstep + r >= w.u.len)
                            for (int q = 0; q < D / 64; ++q)
                                for (int e = 0; e < 8; ++e)
                                    st_shared_v4(smem_u32(sV(s)) + q * SN * 128 + row * 128 + e * 16, 0, 0, 0, 0);
                        fence_proxy_async_smem();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[grp * 2 + sb]);
            }
            // ---- epilogue: O / l (16 bit) and LSE, or O, m and l in fp32 where other CTAs have the rest of the unit; a
            // thread a row; kSplit: the groups' maxima and sums first, and each group writes half of the columns
            float m = m_ref, fa = 1.f, fb = 0.f;
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
            // (neither barrier gets to its next phase before every warp that waits here is through: the next piece's
            // products wait for their P)
            if (steps > 0) {
                wait(&o_last[grp], n_last & 1);
                if (kSplit) wait(&o_last[grp ^ 1], n_last & 1);
                ++n_last;
            }
            if (steps > 1) ++n_prev;
            const bool done = w.begins() && w.ends();
            const int slot = w.begins() ? 1 : 0;
            if (!done) {
                const int4 name = unit_name(w.n, w.x, w.t, w.ends() ? kEnds : kGoesOn);
                if (slot) named1 = name;
                else named0 = name;
            }
            const int head = w.x * G + row_head;
            const float inv = l == 0.f ? 0.f : 1.f / l;  // (NaN stays NaN)
            T *O = static_cast<T *>(a.o.ptr) + (a.seqs.cu ? int64_t(w.u.first + ti) * a.o.ss : w.n * a.o.sb + ti * a.o.ss) +
                   head * a.o.sh;
            const int64_t part = (int64_t(blockIdx.x) * 2 + slot) * (kSplit ? BM : 2 * BM) + (kSplit ? 0 : grp * BM) + r;
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
                    const float ga = done ? fa * inv : fa, gb = done ? fb * inv : fb;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            y[k] = __uint_as_float(va[e + k]) * ga;
                            if (kSplit) y[k] = fmaf(__uint_as_float(vb[e + k]), gb, y[k]);
                        }
                        if (done) {
                            *reinterpret_cast<uint4 *>(O + o0 + e) =
                                make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
                        } else {
                            float4 *dst = reinterpret_cast<float4 *>(a.part_o + part * D + o0 + e);
                            dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                            dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                        }
                    }
                }
            }
            if (row_ok && (!kSplit || grp == 0)) {
                if (!done)
                    a.part_ml[part] = make_float2(m, l);
                else if (a.lse)
                    a.lse[a.seqs.cu ? int64_t(head) * a.seqs.tokens + w.u.first + ti : (int64_t(w.n) * a.h + head) * a.seqs.s_q + ti] =
                        lse_of(m, l);
            }
            k_base += st.stages;
            // the next piece's first product overwrites O once this group's P of it is there, which is behind these
            // reads; with kSplit the other group's reads too
            if (kSplit) named_bar_sync(3, 256);
        }
        if (threadIdx.x == 128) {
            a.rec[2 * blockIdx.x] = named0;
            a.rec[2 * blockIdx.x + 1] = named1;
        }
    } else if (kEight) {
        // ================================================= e4m3 -> 16 bit (warps 12..15)
        regs_decrease<kRegsConvert>();
        // a thread's row k of the stage, of which it takes every other 16 bytes from col on: eight lanes eight rows, whose
        // swizzled 16-byte pieces lie in different banks on both sides
        constexpr int N = D / 32;
        const int wt = threadIdx.x - 384, k = wt & 63, col = wt >> 6;
        const float c = a.scale * kLog2e;
        float *scales = reinterpret_cast<float *>(smem + Cfg::OFF_KS);
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok && !(ok = mbar_wait(bar, parity, abort))) flag_abort(abort, nullptr);
            ok = __all_sync(0xffffffffu, ok);
        };
        uint32_t n = 0, s = 0, par = 1, es = 0, epar = 0;  // stages so far; positions and phases in the two rings
        Walk<kChunkCost> w(sched, *range);
        while (w.next()) {
            const Steps st = steps_of(w);
            for (int j = 0; j < st.stages; ++j, ++n) {
                const int left = w.k1 - (w.k0 + j * HN);  // rows behind: zeros
                wait(&e_full[es], epar);
                wait(&e_full[NE + es], epar);
                const float *size = reinterpret_cast<const float *>(smem + Cfg::OFF_ES) + 2 * es * HN;
                const uint32_t eb = exponent_bits(size[HN + k]);
                const float f = size[HN + k] * exponent_inv(eb);
                const uint32_t factor = pack2<__half>(f, f);
                float *to = scales + n % NKS * 3 * HN + k;
                if (col == 0) {
                    *to = size[k] * c;
                } else {
                    to[HN] = exponent_of(eb);
                    to[2 * HN] = exponent_inv(eb);
                }
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    const uint8_t *src = smem + Cfg::OFF_E + (2 * es + side) * Cfg::E_BYTES;
                    uint4 x[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int c16 = col + 2 * i, at = D == 128 ? c16 ^ (k & 7) : c16 ^ (k >> 1 & 3);
                        x[i] = *reinterpret_cast<const uint4 *>(src + k * D + at * 16);
                        if (k >= left) x[i] = make_uint4(0, 0, 0, 0);
                    }
                    if (n >= uint32_t(NS)) wait(side ? &v_empty[s] : &k_empty[s], par);
                    if (ok) {
                        const uint32_t dst = smem_u32(side ? sV(s) : sK(s)) + k * 128;
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const int c16 = col + 2 * i;
                            const uint32_t to = dst + (c16 >> 2) * HN * 128, c0 = (c16 & 3) * 2;  // 16-byte piece of 128 bytes
                            uint32_t y[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t u = (e / 2 == 0 ? x[i].x : e / 2 == 1 ? x[i].y : e / 2 == 2 ? x[i].z : x[i].w) >> (16 * (e & 1));
                                y[e] = side ? mul_half2(half_pair(u), factor) : widen<T>(u);
                            }
                            st_shared_v4(to + ((c0 ^ (k & 7)) << 4), y[0], y[1], y[2], y[3]);
                            st_shared_v4(to + (((c0 + 1) ^ (k & 7)) << 4), y[4], y[5], y[6], y[7]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&e_empty[side * NE + es]);
                        mbar_arrive(side ? &v_full[s] : &k_full[s]);
                        if (!side) mbar_arrive(&ks_full[n % NKS]);
                    }
                }
                if (++s == NS) {
                    s = 0;
                    par ^= 1;
                }
                if (++es == NE) {
                    es = 0;
                    epar ^= 1;
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) a.flags[blockIdx.x] = (*bad_page ? ATTN_DEV_INDEX_RANGE : 0u) | (*abort ? ATTN_DEV_TIMEOUT : 0u);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::T_COLS);
    }
}

// ===================================================================== host

namespace {

// Pages [n_pages][h_kv][page][d]: boxes of up to 128 tokens x 64 16-bit elements or 64 x d e4m3 ones, with the swizzle of the box's
// width.
bool tmap_pages(CUtensorMap *m, void *ptr, const PagedCache &c, int dtype, int d, int h_kv)
{
    auto enc = tmap_encoder();
    if (!enc) return false;
    const bool eight = c.type == ATTN_E4M3;
    const int page = 1 << c.shift, size = eight ? 1 : 2;
    cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(page), cuuint64_t(h_kv), cuuint64_t(c.none)};
    cuuint64_t strides[3] = {cuuint64_t(c.ss) * size, cuuint64_t(c.sh) * size, cuuint64_t(c.sp) * size};
    cuuint32_t box[4] = {cuuint32_t(eight ? d : 64), cuuint32_t(page < (eight ? 64 : 128) ? page : (eight ? 64 : 128)), 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = eight ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : dtype == ATTN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return enc(m, type, 4, ptr, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               eight && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, tmap_promotion(d * size),
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries as (d, head, token, sequence): boxes of 64 elements x a kv head's query heads x `tokens` tokens, whose rows lie
// in shared memory in that order.
bool tmap_queries(CUtensorMap *m, const View &v, int dtype, int d, int h, int64_t s, int64_t b, int group, int tokens)
{
    auto enc = tmap_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(h), cuuint64_t(s), cuuint64_t(b)};
    cuuint64_t strides[3] = {cuuint64_t(v.sh * 2), cuuint64_t(v.ss * 2), cuuint64_t((b > 1 ? v.sb : 0) * 2)};
    cuuint32_t box[4] = {64, cuuint32_t(group), cuuint32_t(tokens), 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, dtype == ATTN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.ptr, dims, strides,
               box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int D, bool kEight, bool kSplit> cudaError_t run(const PagedAttnArgs &a, cudaStream_t s)
{
    using Cfg = ChunkCfg<D, kEight, kSplit>;
    ChunkParams prm;
    prm.a = a;
    const int group = a.h / a.h_kv;
    prm.tokens = Cfg::BM / group;
    const bool packed = a.seqs.cu != nullptr;
    if (!tmap_queries(&prm.tm_q, a.q, a.dtype, D, a.h, packed ? a.seqs.tokens : a.seqs.s_q, packed ? 1 : a.seqs.b, group, prm.tokens))
        return cudaErrorInvalidValue;
    if (!tmap_pages(&prm.tm_k, a.cache.k, a.cache, a.dtype, D, a.h_kv) ||
             !tmap_pages(&prm.tm_v, a.cache.v, a.cache, a.dtype, D, a.h_kv))
        return cudaErrorInvalidValue;
    auto k = paged_chunk_kernel<T, D, kEight, kSplit>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    return launch_kernel(k, dim3(kPagedCtas), dim3(Cfg::THREADS), Cfg::SMEM_ALLOC, s, false, prm);
}

template <class T, int D> cudaError_t pick(const PagedAttnArgs &a, bool split, cudaStream_t s)
{
    if (a.cache.type == ATTN_E4M3) return split ? run<T, D, true, true>(a, s) : run<T, D, true, false>(a, s);
    return split ? run<T, D, false, true>(a, s) : run<T, D, false, false>(a, s);
}

}  // namespace

PagedShape paged_chunk_shape(int64_t h, int64_t h_kv, int64_t s_q)
{
    PagedShape p;
    p.chunk = true;
    p.heads = int(h / h_kv);
    p.tokens = 128 / p.heads;
    p.groups = s_q <= p.tokens ? 1 : 2;  // chunks that fit 128 rows: kSplit
    p.rows = 128 * p.groups;
    p.shares = kPagedCtas;
    p.row_blocks = 1;
    return p;
}

cudaError_t launch_paged_chunk(const PagedAttnArgs &a, const PagedShape &shape, cudaStream_t s)
{
    const bool split = shape.groups == 1;
    if (a.d == 64) return a.dtype == ATTN_F16 ? pick<__half, 64>(a, split, s) : pick<__nv_bfloat16, 64>(a, split, s);
    return a.dtype == ATTN_F16 ? pick<__half, 128>(a, split, s) : pick<__nv_bfloat16, 128>(a, split, s);
}

}  // namespace attn
