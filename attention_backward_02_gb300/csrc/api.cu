// api.cu -- the C ABI: argument checks, workspace layout, launch order.
//
// Every check runs on the host before the first launch, so a call that
// returns an error has launched nothing.  Launch order on the caller's
// stream: preprocess -> main backward -> dQ finalize (dense), and
// preprocess -> block lists -> main -> finalizes (NSA); each kernel is
// chained to its predecessor with programmatic dependent launch.  With a relative
// bias the expansion of its table goes first (forward: then the main kernel), and the
// dQ finalize sums the table's gradient too.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "attnbwd.h"
#include "paged.h"
#include "plan.h"
#include "qk_norm.h"
#include "relbias.h"
#include "relbias_decode.h"

using namespace attn;

namespace {

constexpr int64_t kTilePad = 128;       // NSA: rows a tile may run past the last token
constexpr int kDefaultDqSplits = 8;     // deterministic dense dQ partial buffers

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Element strides of a 16-bit tensor must be multiples of 8 (16 bytes).
bool strides_ok(const attn_view_t &v) { return v.sb % 8 == 0 && v.sh % 8 == 0 && v.ss % 8 == 0; }

struct DenseShape {
    bool packed;
    int64_t nseq, t_q, t_kv;
};

attn_status_t check_cu(const int64_t *cu, int64_t n, int64_t *total)
{
    int64_t prev = 0;
    for (int64_t b = 0; b < n; ++b) {
        if (cu[b] < prev) return ATTN_ERR_INVALID;
        prev = cu[b];
    }
    *total = prev;
    return ATTN_OK;
}

attn_status_t check_dense_desc(const attn_sdpa_desc_t *d, DenseShape *sh)
{
    if (!d) return ATTN_ERR_NULLPTR;
    if (d->dtype != ATTN_F16 && d->dtype != ATTN_BF16) return ATTN_ERR_INVALID;
    if (d->b < 1 || d->h < 1 || d->h_kv < 1 || d->h % d->h_kv != 0 || d->d < 1) return ATTN_ERR_INVALID;
    if (!std::isfinite(d->scale)) return ATTN_ERR_INVALID;
    if (d->mask != ATTN_MASK_NONE && d->mask != ATTN_CAUSAL_TOP_LEFT && d->mask != ATTN_CAUSAL_BOTTOM_RIGHT)
        return ATTN_ERR_INVALID;
    if ((d->cu_seqlens_q == nullptr) != (d->cu_seqlens_kv == nullptr)) return ATTN_ERR_NULLPTR;
    if (d->deterministic < 0 || d->deterministic > 2) return ATTN_ERR_INVALID;
    if (d->dq_splits < 0) return ATTN_ERR_INVALID;
    sh->packed = d->cu_seqlens_q != nullptr;
    sh->nseq = d->b;
    if (sh->packed) {
        if (d->b > kMaxSeq) return ATTN_ERR_UNSUPPORTED;
        attn_status_t st = check_cu(d->cu_seqlens_q, d->b, &sh->t_q);
        if (st) return st;
        st = check_cu(d->cu_seqlens_kv, d->b, &sh->t_kv);
        if (st) return st;
    } else {
        if (d->s_q < 0 || d->s_kv < 0) return ATTN_ERR_INVALID;
        if (d->b > 65535) return ATTN_ERR_UNSUPPORTED;  // grid z
        sh->t_q = d->b * d->s_q;
        sh->t_kv = d->b * d->s_kv;
    }
    if (d->d != 64 && d->d != 128) return ATTN_ERR_UNSUPPORTED;
    // 32-bit row indices inside the kernels
    if (sh->t_q * d->h >= (int64_t(1) << 31) || sh->t_kv * d->h_kv >= (int64_t(1) << 31))
        return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

int dense_parts(const attn_sdpa_desc_t *d)
{
    if (d->deterministic != 1) return 1;
    return d->dq_splits > 0 ? d->dq_splits : kDefaultDqSplits;
}

struct DenseLayout {
    size_t status, lse2, dvec, dqacc, sem, total;
    int64_t t_pad;
};

// Workspace rows: every sequence's query rows rounded up to kWsRowAlign.
int64_t ws_rows(const attn_sdpa_desc_t *d, const DenseShape &sh)
{
    if (!sh.packed) return d->b * ws_round(d->s_q);
    int64_t n = 0;
    for (int64_t b = 0; b < d->b; ++b) n += ws_round(d->cu_seqlens_q[b] - (b ? d->cu_seqlens_q[b - 1] : 0));
    return n;
}

DenseLayout dense_layout(const attn_sdpa_desc_t *d, const DenseShape &sh)
{
    DenseLayout L;
    L.t_pad = ws_rows(d, sh);
    size_t rows = size_t(d->h) * size_t(L.t_pad);
    L.status = 0;
    L.lse2 = Workspace::align(64 * sizeof(uint32_t));
    L.dvec = L.lse2 + Workspace::align(rows * sizeof(float));
    L.dqacc = L.dvec + Workspace::align(rows * sizeof(float));
    L.sem = L.dqacc + Workspace::align(size_t(dense_parts(d)) * rows * size_t(d->d) * sizeof(float));
    // ordered dQ mode: one add counter per (head, 64 workspace rows)
    L.total = L.sem + (d->deterministic == 2 ? Workspace::align(rows / 64 * sizeof(uint32_t)) : 0);
    return L;
}

View to_view(const attn_view_t &v, bool packed)
{
    View w;
    w.ptr = v.ptr;
    w.sb = packed ? 0 : v.sb;
    w.sh = v.sh;
    w.ss = v.ss;
    return w;
}

attn_status_t check_view(const attn_view_t &v, int64_t rows)
{
    if (rows == 0) return ATTN_OK;
    if (!v.ptr) return ATTN_ERR_NULLPTR;
    if (!aligned16(v.ptr) || !strides_ok(v)) return ATTN_ERR_ALIGN;
    return ATTN_OK;
}

attn_status_t check_ws(const void *ws, size_t have, size_t need)
{
    if (need == 0) return ATTN_OK;
    if (!ws || have < need || (reinterpret_cast<uintptr_t>(ws) & (Workspace::kAlign - 1))) return ATTN_ERR_WORKSPACE;
    return ATTN_OK;
}

void fill_geo(const attn_sdpa_desc_t *d, const DenseShape &sh, FixedGeo *fg, PackedGeo *pg)
{
    fg->nseq = d->b;
    fg->s_q = d->s_q;
    fg->s_kv = d->s_kv;
    if (sh.packed) {
        pg->nseq = d->b;
        pg->cu_q[0] = pg->cu_kv[0] = pg->ws_q[0] = 0;
        for (int64_t b = 0; b < d->b; ++b) {
            pg->cu_q[b + 1] = d->cu_seqlens_q[b];
            pg->cu_kv[b + 1] = d->cu_seqlens_kv[b];
            pg->ws_q[b + 1] = pg->ws_q[b] + ws_round(pg->cu_q[b + 1] - pg->cu_q[b]);
        }
    }
}

// Text of the CUDA error behind the last ATTN_ERR_CUDA of this host thread.
thread_local const char *g_last_error = "";

attn_status_t cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return ATTN_OK;
    g_last_error = cudaGetErrorString(e);
    return ATTN_ERR_CUDA;
}

thread_local cudaEvent_t g_ev_before = nullptr, g_ev_after = nullptr;

// Records a timing event; under stream capture as an external event node, so replays record it.
cudaError_t mark(cudaEvent_t ev, cudaStream_t s)
{
    if (!ev) return cudaSuccess;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(s, &cs);
    if (e != cudaSuccess) return e;
    return cudaEventRecordWithFlags(ev, s, cs == cudaStreamCaptureStatusActive ? cudaEventRecordExternal : 0);
}

}  // namespace

attn_status_t attn::record_cuda_error(cudaError_t e) { return cuda_status(e); }

extern "C" {

const char *attn_last_error(void) { return g_last_error; }

const char *attn_status_string(attn_status_t s)
{
    switch (s) {
    case ATTN_OK: return "ATTN_OK";
    case ATTN_ERR_NULLPTR: return "ATTN_ERR_NULLPTR";
    case ATTN_ERR_INVALID: return "ATTN_ERR_INVALID";
    case ATTN_ERR_UNSUPPORTED: return "ATTN_ERR_UNSUPPORTED";
    case ATTN_ERR_WORKSPACE: return "ATTN_ERR_WORKSPACE";
    case ATTN_ERR_ALIGN: return "ATTN_ERR_ALIGN";
    case ATTN_ERR_CUDA: return "ATTN_ERR_CUDA";
    case ATTN_ERR_DEVICE: return "ATTN_ERR_DEVICE";
    }
    return "ATTN_ERR_UNKNOWN";
}

attn_status_t sdpa_workspace_size(const attn_sdpa_desc_t *desc, size_t *fwd_bytes, size_t *bwd_bytes)
{
    DenseShape sh;
    attn_status_t st = check_dense_desc(desc, &sh);
    if (st) return st;
    if (fwd_bytes) *fwd_bytes = Workspace::align(64 * sizeof(uint32_t));
    if (bwd_bytes) *bwd_bytes = dense_layout(desc, sh).total;
    return ATTN_OK;
}

}  // extern "C"

namespace {

// -------------------------------------------------- relative position bias

// base^power (base at most 65536, power at most 64: 1025 bits) times what is in w, in words of 32 bits.
constexpr int kRelWords = 34;
void rel_multiply(uint32_t (&w)[kRelWords], uint64_t base, int power)
{
    for (; power > 0; --power) {
        uint64_t carry = 0;
        for (uint32_t &x : w) {
            carry += x * base;
            x = uint32_t(carry);
            carry >>= 32;
        }
    }
}

// Whether distance x (e .. max_distance) has reached step m < k of the k = n - e buckets past the exact ones:
// log(x / e) / log(max_distance / e) k >= m.  By logarithms where the two sides are further apart than their
// rounding (below 1e-12; whole distances come much closer than 1e-9 to a border without reaching it), else by
// x^k >= max_distance^m e^(k - m) in integers, each side below 2^1025.
bool rel_reached(const RelBias &r, int64_t max_distance, int64_t x, int m)
{
    const int k = r.n - r.e;
    const double step = std::log(double(x) / r.e) / std::log(double(max_distance) / r.e) * k;
    if (std::fabs(step - m) > 1e-9) return step > m;
    uint32_t left[kRelWords] = {1}, right[kRelWords] = {1};
    rel_multiply(left, uint64_t(x), k);
    rel_multiply(right, uint64_t(max_distance), m);
    rel_multiply(right, uint64_t(r.e), k - m);
    for (int i = kRelWords - 1; i >= 0; --i)
        if (left[i] != right[i]) return left[i] > right[i];
    return true;
}

attn_status_t check_relbias(const attn_relbias_t *b, RelBias *r)
{
    if (!b) return ATTN_ERR_NULLPTR;
    if (b->bidirectional != 0 && b->bidirectional != 1) return ATTN_ERR_INVALID;
    if (b->table_type != ATTN_F16 && b->table_type != ATTN_BF16 && b->table_type != ATTN_F32) return ATTN_ERR_INVALID;
    if (b->num_buckets < 2 || (b->bidirectional && (b->num_buckets < 4 || b->num_buckets % 2 != 0)))
        return ATTN_ERR_INVALID;
    const int64_t n = b->bidirectional ? b->num_buckets / 2 : b->num_buckets;
    if (b->max_distance <= n / 2) return ATTN_ERR_INVALID;
    if (b->num_buckets > kRelMaxBuckets || b->max_distance > kRelMaxDistance) return ATTN_ERR_UNSUPPORTED;
    // the borders of the last bucket layout (a hundred logarithms, several microseconds of a small call)
    static thread_local RelBias last;
    static thread_local int64_t last_distance = 0;
    if (last.buckets == b->num_buckets && last_distance == b->max_distance && last.bidirectional == b->bidirectional) {
        *r = last;
        r->table = b->table;
        r->table_type = b->table_type;
        return ATTN_OK;
    }
    std::memset(r, 0, sizeof *r);
    r->buckets = int(b->num_buckets);
    r->n = int(n);
    r->e = int(n / 2);
    r->bidirectional = b->bidirectional;
    r->nthr = r->n - r->e - 1;
    const double far = double(b->max_distance);
    for (int m = 1; m <= r->nthr; ++m) {  // the first distance of step m: a guess, then by the definition
        int64_t x = int64_t(r->e * std::pow(far / r->e, double(m) / (r->n - r->e)));
        if (x < r->e) x = r->e;
        while (x > r->e && rel_reached(*r, b->max_distance, x - 1, m)) --x;
        while (!rel_reached(*r, b->max_distance, x, m)) ++x;
        r->thr[m - 1] = int32_t(x);
    }
    const int w = r->nthr ? r->thr[r->nthr - 1] : r->e;
    r->lo = -w;
    r->hi = r->bidirectional ? w : 1;  // (1: a causal mask may part it from 0)
    last = *r;
    last_distance = b->max_distance;
    r->table = b->table;
    r->table_type = b->table_type;
    return ATTN_OK;
}

attn_status_t check_rel_table(const RelBias &r)
{
    if (!r.table) return ATTN_ERR_NULLPTR;
    const uintptr_t size = r.table_type == ATTN_F32 ? 4 : 2;
    return reinterpret_cast<uintptr_t>(r.table) & (size - 1) ? ATTN_ERR_ALIGN : ATTN_OK;
}

// Workspace of the calls with a bias, behind `base` bytes of the call without one: the expanded table and, for
// the backward, its bucket codes, the shares of the table's gradient and those of dK and dV.
struct RelLayout {
    size_t rel, code, part, kv, total;
    int shares;
};

// Units that share the query heads of a (key tile, kv head) in the backward: more than one where the units are few
// and large, so that some SMs would wait for others.  The estimate: the longest sum of a CTA's units, taken as
// the largest of the mean and, for each k, k + 1 units of the k * 152 + 1st size (half a query tile takes 0.85 us
// at d = 128, 1.2 at d = 64; a unit's start is one of them), and the shares' way through the workspace at 2.2 TB/s.
// The split and ordered dQ modes keep one unit: their order of adds is by key tiles.  A constant 152 SMs: the
// workspace size must not depend on a CUDA call.  Measured (us, whole call, causal, 32 buckets to 128 unless said; 1, 2,
// 4, 8 shares, the choice in brackets): b1 h32/8 s2048 d128 209 [135] 155; b1 h32/8 s4096 [398] 502 438; b2 h32/4 s1024
// 216 131 [101] 120; b1 h16/1 s1024 d64 283 152 84 [53]; b1 h8/1 s512, 4096 keys 117 71 [49] 53; b4 h32/8 s1024 [161]
// 190 222; b1 h32/8 s1301, 2285 keys [148] 159 157, and with 64 buckets to 1024 [177] 188 174; b2 h12/4 s777 d64
// without a mask [88], 3 shares 64.  The estimate counts all blocks of scores alike, though one that crosses a bucket's
// border costs more (half of them do with 64 buckets to 1024, a tenth with 32 to 128), and it errs in the last two.
int rel_shares(const attn_sdpa_desc_t *d, const DenseShape &sh)
{
    const int64_t G = d->h / d->h_kv, sms = 152;
    constexpr int kTiles = 1024;
    if (G == 1 || d->deterministic || sh.t_q == 0 || sh.t_kv == 0) return 1;
    const int64_t BM = d->d == 64 ? 128 : 64, copies = sh.packed ? d->h_kv : d->h_kv * d->b;
    int32_t nq[kTiles];  // query tiles of each key tile
    int n = 0;
    for (int64_t b = 0; b < (sh.packed ? d->b : 1); ++b) {
        const int64_t lq = sh.packed ? d->cu_seqlens_q[b] - (b ? d->cu_seqlens_q[b - 1] : 0) : d->s_q;
        const int64_t lkv = sh.packed ? d->cu_seqlens_kv[b] - (b ? d->cu_seqlens_kv[b - 1] : 0) : d->s_kv;
        for (int64_t j0 = 0; j0 < lkv; j0 += 128) {
            if (n == kTiles) return 1;
            const int64_t lo = first_query_seeing(d->mask, j0, lq, lkv);
            nq[n++] = int32_t(lq <= 0 || lo >= lq ? 0 : (lq + BM - 1) / BM - lo / BM);
        }
    }
    if (n * copies > 8 * sms) return 1;
    std::sort(nq, nq + n, [](int32_t x, int32_t y) { return x > y; });
    int best = 1;
    double best_us = 0;
    for (int64_t s = 1; s <= G && s <= 8; ++s) {
        if (G % s) continue;
        double total = 0, most = 0;
        for (int k = 0; k < n; ++k) total += double(2 * (G / s) * nq[k] + 2) * double(copies * s);
        for (int64_t k = 0; k * sms < n * copies * s; ++k) {
            const double sum = double(k + 1) * double(2 * (G / s) * nq[k * sms / (copies * s)] + 2);
            most = sum > most ? sum : most;
        }
        if (most < total / double(sms)) most = total / double(sms);
        const double us = most * (d->d == 64 ? 1.2 : 0.85) + (s > 1 ? double(s * 2 * sh.t_kv * d->h_kv * d->d * 8) / 2.2e6 + 4 : 0.);
        if (s == 1 || us < 0.95 * best_us) {
            best = int(s);
            best_us = us;
        }
    }
    return best;
}

RelLayout rel_layout(const attn_sdpa_desc_t *d, const DenseShape &sh, const RelBias &r, size_t base, bool backward)
{
    RelLayout L;
    const size_t line = size_t(rel_stride(r));
    L.rel = base;
    L.code = L.rel + Workspace::align(size_t(d->h) * line * sizeof(float));
    L.part = L.code + (backward ? Workspace::align(line * sizeof(uint32_t)) : 0);
    const size_t rows = size_t(sh.t_kv / 128 + d->b + 1);
    L.kv = L.part + (backward ? Workspace::align(rows * size_t(d->h) * 8 * size_t(r.buckets) * sizeof(float)) : 0);
    L.shares = backward ? rel_shares(d, sh) : 1;
    L.total = L.kv + (L.shares > 1 ? Workspace::align(size_t(2 * L.shares) * size_t(sh.t_kv * d->h_kv * d->d) * sizeof(float)) : 0);
    return L;
}

void fill_rel(RelArgs *a, const attn_sdpa_desc_t *d, const DenseShape &sh, const RelBias &r, const RelLayout &L, void *workspace,
              bool backward, float *dtable)
{
    std::memset(a, 0, sizeof *a);
    char *ws = static_cast<char *>(workspace);
    a->b = r;
    a->h = d->h;
    a->rel = reinterpret_cast<float *>(ws + L.rel);
    a->stride = rel_stride(r);
    a->status = reinterpret_cast<uint32_t *>(ws);
    if (backward) {
        a->causal = d->mask != ATTN_MASK_NONE;
        a->code = reinterpret_cast<uint32_t *>(ws + L.code);
        a->part = reinterpret_cast<float *>(ws + L.part);
        a->part_rows = sh.t_kv / 128 + d->b + 1;
        a->dtable = dtable;
        a->shares = L.shares;
        a->kv_part = reinterpret_cast<float *>(ws + L.kv);
    }
}

// 32-bit entries of the expanded table inside the kernels, and the grid of the small ones
attn_status_t check_rel_heads(const attn_sdpa_desc_t *d) { return d->h > 65535 ? ATTN_ERR_UNSUPPORTED : ATTN_OK; }

// sdpa_fwd_stats (bias NULL) and sdpa_relbias_fwd_stats
attn_status_t dense_fwd_call(const attn_sdpa_desc_t *desc, const RelBias *bias, attn_view_t q, attn_view_t k, attn_view_t v,
                             attn_view_t o, float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    DenseShape sh;
    attn_status_t st = check_dense_desc(desc, &sh);
    if (st) return st;
    if (bias && ((st = check_rel_heads(desc)) || (st = check_rel_table(*bias)))) return st;
    if ((st = check_view(q, sh.t_q)) || (st = check_view(o, sh.t_q)) || (st = check_view(k, sh.t_kv)) ||
        (st = check_view(v, sh.t_kv)))
        return st;
    if (sh.t_q && !lse) return ATTN_ERR_NULLPTR;
    size_t need = Workspace::align(64 * sizeof(uint32_t));
    RelLayout RL = {};
    if (bias) {
        RL = rel_layout(desc, sh, *bias, need, false);
        need = RL.total;
    }
    if ((st = check_ws(workspace, workspace_bytes, need))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (sh.t_q == 0) return bias ? cuda_status(cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s)) : ATTN_OK;

    DenseArgs a;
    std::memset(&a, 0, sizeof a);
    a.dtype = desc->dtype;
    a.nseq = desc->b; a.h = desc->h; a.h_kv = desc->h_kv; a.d = desc->d;
    a.t_q = sh.t_q; a.t_kv = sh.t_kv; a.t_pad = ws_rows(desc, sh);
    a.scale = float(desc->scale);
    a.mask = desc->mask;
    a.packed = sh.packed;
    a.q = to_view(q, sh.packed); a.k = to_view(k, sh.packed); a.v = to_view(v, sh.packed);
    a.o = to_view(o, sh.packed);
    a.lse_out = lse;
    a.status = static_cast<uint32_t *>(workspace);
    FixedGeo fg;
    static thread_local PackedGeo pg;
    fill_geo(desc, sh, &fg, &pg);
    if (!bias) return cuda_status(sh.packed ? launch_dense_fwd(a, pg, s) : launch_dense_fwd(a, fg, s));
    RelArgs rel;
    fill_rel(&rel, desc, sh, *bias, RL, workspace, false, nullptr);
    if ((st = cuda_status(launch_rel_expand(rel, s)))) return st;
    return cuda_status(sh.packed ? launch_relbias_fwd(a, rel, pg, s) : launch_relbias_fwd(a, rel, fg, s));
}

// sdpa_bwd (bias NULL) and sdpa_relbias_bwd
attn_status_t dense_bwd_call(const attn_sdpa_desc_t *desc, const RelBias *bias, attn_view_t q, attn_view_t k, attn_view_t v,
                             attn_view_t o, attn_view_t dO, const float *lse, attn_view_t dQ, attn_view_t dK,
                             attn_view_t dV, float *dtable, void *workspace, size_t workspace_bytes, void *stream)
{
    DenseShape sh;
    attn_status_t st = check_dense_desc(desc, &sh);
    if (st) return st;
    if (bias) {
        if ((st = check_rel_heads(desc)) || (st = check_rel_table(*bias))) return st;
        if (!dtable) return ATTN_ERR_NULLPTR;
        if (reinterpret_cast<uintptr_t>(dtable) & 3) return ATTN_ERR_ALIGN;
    }
    if ((st = check_view(q, sh.t_q)) || (st = check_view(o, sh.t_q)) || (st = check_view(dO, sh.t_q)) ||
        (st = check_view(dQ, sh.t_q)) || (st = check_view(k, sh.t_kv)) || (st = check_view(v, sh.t_kv)) ||
        (st = check_view(dK, sh.t_kv)) || (st = check_view(dV, sh.t_kv)))
        return st;
    if (sh.t_q && !lse) return ATTN_ERR_NULLPTR;
    DenseLayout L = dense_layout(desc, sh);
    // 32-bit row coordinates of the fp32 dQ accumulator inside the kernels
    if (int64_t(dense_parts(desc)) * desc->h * L.t_pad >= (int64_t(1) << 31)) return ATTN_ERR_UNSUPPORTED;
    if (desc->deterministic == 2) {  // ordered dQ: every work unit is planned on the host
        int64_t max_kv = desc->s_kv;
        if (sh.packed) {
            max_kv = 0;
            for (int64_t b = 0; b < desc->b; ++b) {
                const int64_t l = desc->cu_seqlens_kv[b] - (b ? desc->cu_seqlens_kv[b - 1] : 0);
                max_kv = l > max_kv ? l : max_kv;
            }
        }
        if ((max_kv + 127) / 128 * desc->b * desc->h_kv > kOrderedMaxUnits) return ATTN_ERR_UNSUPPORTED;
    }
    RelLayout RL = {};
    if (bias) RL = rel_layout(desc, sh, *bias, L.total, true);
    if ((st = check_ws(workspace, workspace_bytes, bias ? RL.total : L.total))) return st;

    DenseArgs a;
    std::memset(&a, 0, sizeof a);
    a.dtype = desc->dtype;
    a.nseq = desc->b; a.h = desc->h; a.h_kv = desc->h_kv; a.d = desc->d;
    a.t_q = sh.t_q; a.t_kv = sh.t_kv; a.t_pad = L.t_pad;
    a.scale = float(desc->scale);
    a.mask = desc->mask;
    a.deterministic = desc->deterministic == 1;
    a.ordered = desc->deterministic == 2;
    a.n_part = dense_parts(desc);
    a.packed = sh.packed;
    a.q = to_view(q, sh.packed); a.k = to_view(k, sh.packed); a.v = to_view(v, sh.packed);
    a.o = to_view(o, sh.packed); a.dO = to_view(dO, sh.packed);
    a.dQ = to_view(dQ, sh.packed); a.dK = to_view(dK, sh.packed); a.dV = to_view(dV, sh.packed);
    a.lse = lse;
    char *ws = static_cast<char *>(workspace);
    a.status = reinterpret_cast<uint32_t *>(ws + L.status);
    a.lse2 = reinterpret_cast<float *>(ws + L.lse2);
    a.dvec = reinterpret_cast<float *>(ws + L.dvec);
    a.dqacc = reinterpret_cast<float *>(ws + L.dqacc);
    a.sem = reinterpret_cast<uint32_t *>(ws + L.sem);
    a.sem_stride = L.t_pad / 64;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (sh.t_q == 0 && sh.t_kv == 0 && !bias) return ATTN_OK;

    FixedGeo fg;
    static thread_local PackedGeo pg;
    fill_geo(desc, sh, &fg, &pg);
    RelArgs rel;
    const RelArgs *rp = bias ? &rel : nullptr;
    cudaError_t e;
    if (bias) {
        fill_rel(&rel, desc, sh, *bias, RL, workspace, true, dtable);
        if ((e = launch_rel_expand(rel, s)) != cudaSuccess) return cuda_status(e);
    }
    if (sh.packed) {
        if ((e = launch_dense_preprocess(a, pg, s, bias != nullptr)) != cudaSuccess) return cuda_status(e);
        if ((e = mark(g_ev_before, s)) != cudaSuccess) return cuda_status(e);
        if ((e = launch_dense_bwd_main(a, pg, s, rp)) != cudaSuccess) return cuda_status(e);
        if ((e = mark(g_ev_after, s)) != cudaSuccess) return cuda_status(e);
        return cuda_status(launch_dq_finalize(a, pg, s, rp));
    }
    if ((e = launch_dense_preprocess(a, fg, s, bias != nullptr)) != cudaSuccess) return cuda_status(e);
    if ((e = mark(g_ev_before, s)) != cudaSuccess) return cuda_status(e);
    if ((e = launch_dense_bwd_main(a, fg, s, rp)) != cudaSuccess) return cuda_status(e);
    if ((e = mark(g_ev_after, s)) != cudaSuccess) return cuda_status(e);
    return cuda_status(launch_dq_finalize(a, fg, s, rp));
}

}  // namespace

extern "C" {

attn_status_t sdpa_fwd_stats(const attn_sdpa_desc_t *desc, attn_view_t q, attn_view_t k, attn_view_t v,
                             attn_view_t o, float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    return dense_fwd_call(desc, nullptr, q, k, v, o, lse, workspace, workspace_bytes, stream);
}

attn_status_t sdpa_bwd(const attn_sdpa_desc_t *desc, attn_view_t q, attn_view_t k, attn_view_t v, attn_view_t o,
                       attn_view_t dO, const float *lse, attn_view_t dQ, attn_view_t dK, attn_view_t dV,
                       void *workspace, size_t workspace_bytes, void *stream)
{
    return dense_bwd_call(desc, nullptr, q, k, v, o, dO, lse, dQ, dK, dV, nullptr, workspace, workspace_bytes, stream);
}

attn_status_t attn_relbias_bucket(const attn_relbias_t *bias, int64_t delta, int64_t *bucket)
{
    RelBias r;
    const attn_status_t st = check_relbias(bias, &r);
    if (st) return st;
    if (!bucket) return ATTN_ERR_NULLPTR;
    const int64_t far = int64_t(1) << 40;  // beyond any border
    *bucket = r.bucket(delta < -far ? -far : (delta > far ? far : delta));
    return ATTN_OK;
}

attn_status_t sdpa_relbias_workspace_size(const attn_sdpa_desc_t *desc, const attn_relbias_t *bias, size_t *fwd_bytes,
                                          size_t *bwd_bytes)
{
    DenseShape sh;
    RelBias r;
    attn_status_t st = check_dense_desc(desc, &sh);
    if (st || (st = check_rel_heads(desc)) || (st = check_relbias(bias, &r))) return st;
    if (fwd_bytes) *fwd_bytes = rel_layout(desc, sh, r, Workspace::align(64 * sizeof(uint32_t)), false).total;
    if (bwd_bytes) *bwd_bytes = rel_layout(desc, sh, r, dense_layout(desc, sh).total, true).total;
    return ATTN_OK;
}

attn_status_t sdpa_relbias_fwd_stats(const attn_sdpa_desc_t *desc, const attn_relbias_t *bias, attn_view_t q,
                                     attn_view_t k, attn_view_t v, attn_view_t o, float *lse, void *workspace,
                                     size_t workspace_bytes, void *stream)
{
    RelBias r;
    const attn_status_t st = check_relbias(bias, &r);
    if (st) return st;
    return dense_fwd_call(desc, &r, q, k, v, o, lse, workspace, workspace_bytes, stream);
}

attn_status_t sdpa_relbias_bwd(const attn_sdpa_desc_t *desc, const attn_relbias_t *bias, attn_view_t q, attn_view_t k,
                               attn_view_t v, attn_view_t o, attn_view_t dO, const float *lse, attn_view_t dQ,
                               attn_view_t dK, attn_view_t dV, float *dtable, void *workspace, size_t workspace_bytes,
                               void *stream)
{
    RelBias r;
    const attn_status_t st = check_relbias(bias, &r);
    if (st) return st;
    return dense_bwd_call(desc, &r, q, k, v, o, dO, lse, dQ, dK, dV, dtable, workspace, workspace_bytes, stream);
}

// ------------------------------------------------------------------- NSA

namespace {

struct NsaShape {
    int64_t t1, t2, nblk_max, words_max, maxlen_q, dv;
};

attn_status_t check_nsa_desc(const attn_nsa_desc_t *d, NsaShape *sh)
{
    if (!d) return ATTN_ERR_NULLPTR;
    if (!d->cu_seqlens_q || !d->cu_seqlens_kv) return ATTN_ERR_NULLPTR;
    if (d->dtype != ATTN_F16 && d->dtype != ATTN_BF16) return ATTN_ERR_INVALID;
    if (d->b < 1) return ATTN_ERR_INVALID;
    if (d->b > kMaxSeq) return ATTN_ERR_UNSUPPORTED;
    if (d->n1 < 1 || d->n2 < 1 || d->n1 > 128 || d->n2 > 128 || d->n1 % d->n2 != 0 || d->n1 / d->n2 > 32)
        return ATTN_ERR_INVALID;
    if (!std::isfinite(d->scale)) return ATTN_ERR_INVALID;
    if (d->block_size < 16 || d->block_size > 128 || d->block_size % 16 != 0) return ATTN_ERR_INVALID;
    if (d->block_count < 1 || d->block_count > 128 || d->block_count * d->block_size >= 8192)
        return ATTN_ERR_INVALID;
    if (d->sparse_mode != 0 && d->sparse_mode != 2) return ATTN_ERR_INVALID;
    if (d->deterministic < 0 || d->deterministic > 2) return ATTN_ERR_INVALID;
    if (d->d != 128 && d->d != 192) return ATTN_ERR_INVALID;
    if (d->d_v != 0 && d->d_v != 128 && d->d_v != 192) return ATTN_ERR_INVALID;
    if (d->grad_fp32 != 0 && d->grad_fp32 != 1) return ATTN_ERR_INVALID;
    if (check_cu(d->cu_seqlens_q, d->b, &sh->t1) || check_cu(d->cu_seqlens_kv, d->b, &sh->t2))
        return ATTN_ERR_INVALID;
    sh->nblk_max = 0;
    sh->maxlen_q = 0;
    for (int64_t b = 0; b < d->b; ++b) {
        int64_t lkv = d->cu_seqlens_kv[b] - (b ? d->cu_seqlens_kv[b - 1] : 0);
        int64_t lq = d->cu_seqlens_q[b] - (b ? d->cu_seqlens_q[b - 1] : 0);
        if (lkv % d->block_size != 0 || lkv < d->block_count * d->block_size) return ATTN_ERR_INVALID;
        if (lkv / d->block_size > sh->nblk_max) sh->nblk_max = lkv / d->block_size;
        if (lq > sh->maxlen_q) sh->maxlen_q = lq;
    }
    sh->words_max = (sh->maxlen_q + 31) / 32;
    sh->dv = d->d_v ? d->d_v : d->d;
    if (d->atten_mask) {  // the mask covers every sequence's local positions
        if (d->mask_rows < sh->maxlen_q || d->mask_cols < 0) return ATTN_ERR_INVALID;
        for (int64_t b = 0; b < d->b; ++b)
            if (d->cu_seqlens_kv[b] - (b ? d->cu_seqlens_kv[b - 1] : 0) > d->mask_cols) return ATTN_ERR_INVALID;
    }
    if (sh->t1 * d->n1 >= (int64_t(1) << 31) || sh->t2 * d->n2 >= (int64_t(1) << 31)) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

struct NsaLayout {
    size_t status, lse2, dvec, bitmap, offsets, pieces, tokens, dqacc, dkacc, dvacc, dqpart, sem, rank, kvpart, total;
    int64_t t1_pad, nrows;
};

NsaLayout nsa_layout(const attn_nsa_desc_t *d, const NsaShape &sh)
{
    NsaLayout L;
    L.t1_pad = sh.t1 + kTilePad;
    L.nrows = d->b * d->n2 * sh.nblk_max;
    size_t rows = size_t(d->n1) * size_t(L.t1_pad);
    L.status = 0;
    L.lse2 = Workspace::align(64 * sizeof(uint32_t));
    L.dvec = L.lse2 + Workspace::align(rows * sizeof(float));
    L.bitmap = L.dvec + Workspace::align(rows * sizeof(float));
    L.offsets = L.bitmap + Workspace::align(size_t(L.nrows) * size_t(sh.words_max) * sizeof(uint32_t));
    L.pieces = L.offsets + Workspace::align(size_t(L.nrows + 1) * sizeof(int32_t));
    L.tokens = L.pieces + Workspace::align(size_t(L.nrows + 1) * sizeof(int32_t));
    L.dqacc = L.tokens + Workspace::align(size_t(sh.t1) * size_t(d->n2 * d->block_count) * sizeof(int32_t) + 4);
    L.dkacc = L.dqacc + Workspace::align(rows * size_t(d->d) * sizeof(float));
    L.dvacc = L.dkacc + Workspace::align(size_t(sh.t2) * size_t(d->n2 * d->d) * sizeof(float));
    L.dqpart = L.dvacc + Workspace::align(size_t(sh.t2) * size_t(d->n2 * sh.dv) * sizeof(float));
    // deterministic 1: dQ per (token, selected slot); 2: one add counter per (token, kv head)
    const size_t part_bytes = d->deterministic == 1
                                  ? size_t(sh.t1) * size_t(d->n1) * size_t(d->block_count) * size_t(d->d) * sizeof(float)
                                  : 0;
    L.sem = L.dqpart + Workspace::align(part_bytes);
    const bool ord = d->deterministic == 2;
    L.rank = L.sem + (ord ? Workspace::align(size_t(sh.t1) * size_t(d->n2) * sizeof(uint32_t)) : 0);
    L.kvpart = L.rank + (ord ? Workspace::align(size_t(sh.t1) * size_t(d->n2 * d->block_count) * sizeof(int32_t)) : 0);
    // deterministic mode 1: each work unit's dK / dV rows (block_size keys x (d + d_v) fp32)
    const size_t kv_bytes = d->deterministic == 1 ? size_t(nsa_max_pieces(L.nrows, sh.t1, d->n2, d->block_count,
                                                                           d->n1 / d->n2)) *
                                                        size_t(d->block_size) * size_t(d->d + sh.dv) * sizeof(float)
                                                  : 0;
    L.total = L.kvpart + Workspace::align(kv_bytes);
    return L;
}

// The forward runs on the tensor cores for d = d_v = 128 and blocks of 64 (the backward's block lists,
// its lse2 / dvec rows for the row maxima and sums and its dQ accumulator for O); otherwise on CUDA
// cores, which need the status word alone.
bool nsa_fwd_on_tc(const attn_nsa_desc_t *d, const NsaShape &sh)
{
    return d->d == 128 && sh.dv == 128 && d->block_size == 64;
}

NsaLayout nsa_fwd_layout(const attn_nsa_desc_t *d, const NsaShape &sh)
{
    attn_nsa_desc_t c = *d;
    c.deterministic = 0;  // no per-slot partials or add counters in the forward
    return nsa_layout(&c, sh);
}

size_t nsa_fwd_bytes(const attn_nsa_desc_t *d, const NsaShape &sh)
{
    return nsa_fwd_on_tc(d, sh) ? nsa_fwd_layout(d, sh).total : Workspace::align(64 * sizeof(uint32_t));
}

void nsa_ws_pointers(NsaArgs *a, const NsaLayout &L, void *workspace)
{
    char *ws = static_cast<char *>(workspace);
    a->status = reinterpret_cast<uint32_t *>(ws + L.status);
    a->lse2 = reinterpret_cast<float *>(ws + L.lse2);
    a->dvec = reinterpret_cast<float *>(ws + L.dvec);
    a->bitmap = reinterpret_cast<uint32_t *>(ws + L.bitmap);
    a->offsets = reinterpret_cast<int32_t *>(ws + L.offsets);
    a->tokens = reinterpret_cast<int32_t *>(ws + L.tokens);
    a->pieces = reinterpret_cast<int32_t *>(ws + L.pieces);
    a->dqacc = reinterpret_cast<float *>(ws + L.dqacc);
    a->dkacc = reinterpret_cast<float *>(ws + L.dkacc);
    a->dvacc = reinterpret_cast<float *>(ws + L.dvacc);
    a->dqpart = reinterpret_cast<float *>(ws + L.dqpart);
    a->sem = reinterpret_cast<uint32_t *>(ws + L.sem);
    a->rank = reinterpret_cast<int32_t *>(ws + L.rank);
    a->kvpart = reinterpret_cast<float *>(ws + L.kvpart);
}

}  // namespace

attn_status_t nsa_workspace_size(const attn_nsa_desc_t *desc, size_t *bytes)
{
    NsaShape sh;
    attn_status_t st = check_nsa_desc(desc, &sh);
    if (st) return st;
    if (!bytes) return ATTN_ERR_NULLPTR;
    *bytes = nsa_layout(desc, sh).total;
    return ATTN_OK;
}

attn_status_t nsa_selected_attn_bwd(const attn_nsa_desc_t *desc, const void *q, const void *k, const void *v,
                                    const void *o, const void *dO, const float *softmax_max,
                                    const float *softmax_sum, const int32_t *topk, void *dq, void *dk, void *dv,
                                    void *workspace, size_t workspace_bytes, void *stream)
{
    NsaShape sh;
    attn_status_t st = check_nsa_desc(desc, &sh);
    if (st) return st;
    if (sh.t1 > 0 && (!q || !o || !dO || !softmax_max || !softmax_sum || !topk || !dq)) return ATTN_ERR_NULLPTR;
    if (sh.t2 > 0 && (!k || !v || !dk || !dv)) return ATTN_ERR_NULLPTR;
    for (const void *p : {q, k, v, o, dO, (const void *)dq, (const void *)dk, (const void *)dv})
        if (p && !aligned16(p)) return ATTN_ERR_ALIGN;
    if ((topk && (reinterpret_cast<uintptr_t>(topk) & 3)) || (softmax_max && !aligned16(softmax_max)) ||
        (softmax_sum && !aligned16(softmax_sum)))
        return ATTN_ERR_ALIGN;
    NsaLayout L = nsa_layout(desc, sh);
    if ((st = check_ws(workspace, workspace_bytes, L.total))) return st;
    if (sh.t1 == 0 && sh.t2 == 0) return ATTN_OK;

    NsaArgs a;
    std::memset(&a, 0, sizeof a);
    a.dtype = desc->dtype;
    a.nseq = desc->b; a.n1 = desc->n1; a.n2 = desc->n2; a.d = desc->d; a.dv = sh.dv;
    a.grad_fp32 = desc->grad_fp32;
    a.bs = desc->block_size; a.cnt = desc->block_count;
    a.mask = desc->atten_mask; a.mask_cols = desc->mask_cols;
    a.t1 = sh.t1; a.t2 = sh.t2; a.t1_pad = L.t1_pad;
    a.nblk_max = sh.nblk_max; a.words_max = sh.words_max; a.nrows = L.nrows;
    a.scale = float(desc->scale);
    a.sparse_mode = desc->sparse_mode;
    a.deterministic = desc->deterministic;
    a.n_part = 1;
    a.q = q; a.k = k; a.v = v; a.o = o; a.dO = dO;
    a.smax = softmax_max; a.ssum = softmax_sum; a.topk = topk;
    a.dq = dq; a.dk = dk; a.dvp = dv;
    char *ws = static_cast<char *>(workspace);
    a.status = reinterpret_cast<uint32_t *>(ws + L.status);
    a.lse2 = reinterpret_cast<float *>(ws + L.lse2);
    a.dvec = reinterpret_cast<float *>(ws + L.dvec);
    a.bitmap = reinterpret_cast<uint32_t *>(ws + L.bitmap);
    a.offsets = reinterpret_cast<int32_t *>(ws + L.offsets);
    a.tokens = reinterpret_cast<int32_t *>(ws + L.tokens);
    a.pieces = reinterpret_cast<int32_t *>(ws + L.pieces);
    a.dqacc = reinterpret_cast<float *>(ws + L.dqacc);
    a.dkacc = reinterpret_cast<float *>(ws + L.dkacc);
    a.dvacc = reinterpret_cast<float *>(ws + L.dvacc);
    a.dqpart = reinterpret_cast<float *>(ws + L.dqpart);
    a.sem = reinterpret_cast<uint32_t *>(ws + L.sem);
    a.rank = reinterpret_cast<int32_t *>(ws + L.rank);
    a.kvpart = reinterpret_cast<float *>(ws + L.kvpart);
    // the CUDA-core kernel (a head dim of 192) adds dK / dV atomically from many blocks
    if (a.deterministic && !nsa_tc_supported(a)) return ATTN_ERR_UNSUPPORTED;
    static thread_local PackedGeo pg;
    pg.nseq = desc->b;
    pg.cu_q[0] = pg.cu_kv[0] = 0;
    for (int64_t b = 0; b < desc->b; ++b) {
        pg.cu_q[b + 1] = desc->cu_seqlens_q[b];
        pg.cu_kv[b + 1] = desc->cu_seqlens_kv[b];
    }
    return cuda_status(launch_nsa_bwd(a, pg, static_cast<cudaStream_t>(stream), g_ev_before, g_ev_after));
}

attn_status_t nsa_fwd_workspace_size(const attn_nsa_desc_t *desc, size_t *bytes)
{
    NsaShape sh;
    attn_status_t st = check_nsa_desc(desc, &sh);
    if (st) return st;
    if (!bytes) return ATTN_ERR_NULLPTR;
    *bytes = nsa_fwd_bytes(desc, sh);
    return ATTN_OK;
}

attn_status_t nsa_selected_attn_fwd(const attn_nsa_desc_t *desc, const void *q, const void *k, const void *v,
                                    const int32_t *topk, void *o, float *softmax_max, float *softmax_sum,
                                    void *workspace, size_t workspace_bytes, void *stream)
{
    NsaShape sh;
    attn_status_t st = check_nsa_desc(desc, &sh);
    if (st) return st;
    if (sh.t1 > 0 && (!q || !o || !softmax_max || !softmax_sum || !topk)) return ATTN_ERR_NULLPTR;
    if (sh.t2 > 0 && (!k || !v)) return ATTN_ERR_NULLPTR;
    for (const void *p : {q, k, v, (const void *)o})
        if (p && !aligned16(p)) return ATTN_ERR_ALIGN;
    if ((topk && (reinterpret_cast<uintptr_t>(topk) & 3)) || (softmax_max && !aligned16(softmax_max)) ||
        (softmax_sum && !aligned16(softmax_sum)))
        return ATTN_ERR_ALIGN;
    if ((st = check_ws(workspace, workspace_bytes, nsa_fwd_bytes(desc, sh)))) return st;
    if (sh.t1 == 0) return ATTN_OK;
    NsaArgs a;
    std::memset(&a, 0, sizeof a);
    if (nsa_fwd_on_tc(desc, sh)) {
        const NsaLayout L = nsa_fwd_layout(desc, sh);
        a.t1_pad = L.t1_pad;
        a.nblk_max = sh.nblk_max; a.words_max = sh.words_max; a.nrows = L.nrows;
        nsa_ws_pointers(&a, L, workspace);
    } else {
        a.status = static_cast<uint32_t *>(workspace);
    }
    a.dtype = desc->dtype;
    a.nseq = desc->b; a.n1 = desc->n1; a.n2 = desc->n2; a.d = desc->d; a.dv = sh.dv;
    a.bs = desc->block_size; a.cnt = desc->block_count;
    a.mask = desc->atten_mask; a.mask_cols = desc->mask_cols;
    a.t1 = sh.t1; a.t2 = sh.t2;
    a.scale = float(desc->scale);
    a.sparse_mode = desc->sparse_mode;
    a.q = q; a.k = k; a.v = v; a.topk = topk;
    a.o_out = o; a.smax_out = softmax_max; a.ssum_out = softmax_sum;
    static thread_local PackedGeo pg;
    pg.nseq = desc->b;
    pg.cu_q[0] = pg.cu_kv[0] = 0;
    for (int64_t b = 0; b < desc->b; ++b) {
        pg.cu_q[b + 1] = desc->cu_seqlens_q[b];
        pg.cu_kv[b + 1] = desc->cu_seqlens_kv[b];
    }
    return cuda_status(launch_nsa_fwd(a, pg, static_cast<cudaStream_t>(stream)));
}

attn_status_t nsa_block_lists(const attn_nsa_desc_t *desc, const int32_t *topk, int32_t *offsets, int32_t *tokens,
                              int64_t *nblk_max_out, void *workspace, size_t workspace_bytes, void *stream)
{
    NsaShape sh;
    attn_status_t st = check_nsa_desc(desc, &sh);
    if (st) return st;
    if (!offsets || !tokens || !nblk_max_out || (sh.t1 > 0 && !topk)) return ATTN_ERR_NULLPTR;
    if (reinterpret_cast<uintptr_t>(topk) & 3) return ATTN_ERR_ALIGN;
    NsaLayout L = nsa_layout(desc, sh);
    if ((st = check_ws(workspace, workspace_bytes, L.total))) return st;
    *nblk_max_out = sh.nblk_max;
    NsaArgs a;
    std::memset(&a, 0, sizeof a);
    a.dtype = desc->dtype;
    a.nseq = desc->b; a.n1 = desc->n1; a.n2 = desc->n2; a.d = desc->d; a.dv = sh.dv;
    a.grad_fp32 = desc->grad_fp32;
    a.bs = desc->block_size; a.cnt = desc->block_count;
    a.mask = desc->atten_mask; a.mask_cols = desc->mask_cols;
    a.t1 = sh.t1; a.t2 = sh.t2; a.t1_pad = L.t1_pad;
    a.nblk_max = sh.nblk_max; a.words_max = sh.words_max; a.nrows = L.nrows;
    a.sparse_mode = desc->sparse_mode;
    a.topk = topk;
    char *ws = static_cast<char *>(workspace);
    a.status = reinterpret_cast<uint32_t *>(ws + L.status);
    a.bitmap = reinterpret_cast<uint32_t *>(ws + L.bitmap);
    a.offsets = offsets;
    a.tokens = tokens;
    static thread_local PackedGeo pg;
    pg.nseq = desc->b;
    pg.cu_q[0] = pg.cu_kv[0] = 0;
    for (int64_t b = 0; b < desc->b; ++b) {
        pg.cu_q[b + 1] = desc->cu_seqlens_q[b];
        pg.cu_kv[b + 1] = desc->cu_seqlens_kv[b];
    }
    return cuda_status(launch_nsa_block_lists(a, pg, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------- one token with the relative bias

namespace {

attn_status_t check_decode(const attn_sdpa_desc_t *d, const attn_relbias_t *bias, RelBias *r)
{
    DenseShape sh;
    attn_status_t st = check_dense_desc(d, &sh);
    if (st || (st = check_relbias(bias, r))) return st;
    if (d->s_q != 1 || d->mask != ATTN_CAUSAL_BOTTOM_RIGHT) return ATTN_ERR_INVALID;
    if (sh.packed) return ATTN_ERR_UNSUPPORTED;
    if (d->h > 65535 || d->b > 65535 || d->s_kv > INT32_MAX) return ATTN_ERR_UNSUPPORTED;  // grid y and z, int32 lengths
    return ATTN_OK;
}

struct DecodeLayout {
    int64_t chunk;
    size_t ml, o, total;
};

DecodeLayout decode_layout(const attn_sdpa_desc_t *d)
{
    DecodeLayout L;
    L.chunk = decode_chunk(d->b, d->h, d->h_kv, d->s_kv, d->d);
    const int64_t chunks = decode_chunks(d->s_kv, L.chunk);
    const size_t rows = chunks > 1 ? size_t(d->b) * size_t(d->h) * size_t(chunks) : 0;
    L.ml = Workspace::align(64 * sizeof(uint32_t));
    L.o = L.ml + Workspace::align(rows * 2 * sizeof(float));
    L.total = L.o + Workspace::align(rows * size_t(d->d) * sizeof(float));
    return L;
}

}  // namespace

attn_status_t sdpa_relbias_decode_workspace_size(const attn_sdpa_desc_t *desc, const attn_relbias_t *bias, size_t *bytes)
{
    RelBias r;
    const attn_status_t st = check_decode(desc, bias, &r);
    if (st) return st;
    if (!bytes) return ATTN_ERR_NULLPTR;
    *bytes = decode_layout(desc).total;
    return ATTN_OK;
}

attn_status_t sdpa_relbias_decode(const attn_sdpa_desc_t *desc, const attn_relbias_t *bias, attn_view_t q, attn_view_t k,
                                  attn_view_t v, const int32_t *lens, attn_view_t o, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    DecodeArgs a;
    std::memset(&a, 0, sizeof a);
    attn_status_t st = check_decode(desc, bias, &a.bias);
    if (st || (st = check_rel_table(a.bias))) return st;
    const int64_t keys = desc->b * desc->s_kv;
    if ((st = check_view(q, desc->b)) || (st = check_view(o, desc->b)) || (st = check_view(k, keys)) ||
        (st = check_view(v, keys)))
        return st;
    if (reinterpret_cast<uintptr_t>(lens) & 3) return ATTN_ERR_ALIGN;
    const DecodeLayout L = decode_layout(desc);
    if ((st = check_ws(workspace, workspace_bytes, L.total))) return st;
    a.dtype = desc->dtype;
    a.b = desc->b; a.h = desc->h; a.h_kv = desc->h_kv; a.d = desc->d; a.cap = desc->s_kv;
    a.chunk = L.chunk;
    a.scale = float(desc->scale);
    a.q = to_view(q, false); a.k = to_view(k, false); a.v = to_view(v, false); a.o = to_view(o, false);
    a.lens = lens;
    char *ws = static_cast<char *>(workspace);
    a.status = reinterpret_cast<uint32_t *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(ws + L.ml);
    a.part_o = reinterpret_cast<float *>(ws + L.o);
    return cuda_status(launch_relbias_decode(a, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ paged cache

namespace {

constexpr int64_t kPagedMost = int64_t(1) << 30;  // cached tokens of a sequence

bool offset_fits(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t d)
{
    const int64_t lim = int64_t(1) << 31;
    return s1 < lim && s2 < lim && (n1 - 1) * s1 + (n2 - 1) * s2 + d < lim;
}

attn_status_t check_paged(const attn_sdpa_desc_t *d, const attn_paged_cache_t *c, PagedCache *out)
{
    if (!d || !c) return ATTN_ERR_NULLPTR;
    if (d->dtype != ATTN_F16 && d->dtype != ATTN_BF16) return ATTN_ERR_INVALID;
    if (d->b < 1 || d->h < 1 || d->h_kv < 1 || d->h % d->h_kv != 0 || d->d < 1) return ATTN_ERR_INVALID;
    if (d->s_q < 0 || d->s_kv < 0 || !std::isfinite(d->scale)) return ATTN_ERR_INVALID;
    if (d->mask != ATTN_MASK_NONE && d->mask != ATTN_CAUSAL_TOP_LEFT && d->mask != ATTN_CAUSAL_BOTTOM_RIGHT)
        return ATTN_ERR_INVALID;
    if (c->type != int(d->dtype) && c->type != ATTN_E4M3) return ATTN_ERR_INVALID;
    if (c->n_pages < 0 || c->page_size < 1) return ATTN_ERR_INVALID;
    const bool eight = c->type == ATTN_E4M3;
    if (c->sp < 0 || c->sh < 0 || c->ss < 0) return ATTN_ERR_INVALID;
    if (eight && (c->scale_sp < 0 || c->scale_sh < 0 || c->scale_ss < 0)) return ATTN_ERR_INVALID;
    if (d->mask == ATTN_CAUSAL_TOP_LEFT || d->cu_seqlens_q || d->cu_seqlens_kv) return ATTN_ERR_UNSUPPORTED;
    if ((d->d != 64 && d->d != 128) || d->h / d->h_kv > kPagedMaxGroup) return ATTN_ERR_UNSUPPORTED;
    if (d->b > 65535 || d->h > 65535 || d->s_q > kPagedMost || d->s_kv > kPagedMost) return ATTN_ERR_UNSUPPORTED;
    int shift = 4;
    while (shift < 9 && (int64_t(1) << shift) != c->page_size) ++shift;
    if (shift == 9 || c->n_pages > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
    if (c->sp >= int64_t(1) << 38 || !offset_fits(c->page_size, c->ss, d->h_kv, c->sh, d->d)) return ATTN_ERR_UNSUPPORTED;
    if (eight && !offset_fits(c->page_size, c->scale_ss, d->h_kv, c->scale_sh, 1)) return ATTN_ERR_UNSUPPORTED;
    const int64_t unit = eight ? 16 : 8;
    if (c->sp % unit || c->sh % unit || c->ss % unit) return ATTN_ERR_ALIGN;
    out->k = c->k; out->v = c->v;
    out->k_scale = c->k_scale; out->v_scale = c->v_scale;
    out->type = c->type;
    out->n_pages = int(c->n_pages);
    out->shift = shift;
    out->none = out->n_pages > 0 ? out->n_pages : 1;
    out->sp = c->sp; out->sh = int(c->sh); out->ss = int(c->ss);
    out->sc_sp = eight ? c->scale_sp : 0; out->sc_sh = eight ? int(c->scale_sh) : 0; out->sc_ss = eight ? int(c->scale_ss) : 0;
    return ATTN_OK;
}

// The cache's memory and the sequences, of a call.
attn_status_t check_paged_call(const attn_sdpa_desc_t *d, const attn_paged_cache_t *c, const attn_paged_seqs_t *s, PagedSeqs *out)
{
    if (c->n_pages > 0) {
        if (!c->k || !c->v || (c->type == ATTN_E4M3 && (!c->k_scale || !c->v_scale))) return ATTN_ERR_NULLPTR;
        if (!aligned16(c->k) || !aligned16(c->v)) return ATTN_ERR_ALIGN;
        if (c->type == ATTN_E4M3 && ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3))
            return ATTN_ERR_ALIGN;
    }
    if (!s || !s->lens) return ATTN_ERR_NULLPTR;
    if (d->s_kv > 0 && !s->page_table) return ATTN_ERR_NULLPTR;
    if (s->table_stride < 0 || s->table_pages < (d->s_kv + c->page_size - 1) / c->page_size) return ATTN_ERR_INVALID;
    if (s->cu_new && s->tokens < 0) return ATTN_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(s->page_table) | reinterpret_cast<uintptr_t>(s->lens) |
         reinterpret_cast<uintptr_t>(s->cu_new)) & 3)
        return ATTN_ERR_ALIGN;
    // 32-bit row indices inside the kernels, which round them up to a block's rows and the number of blocks
    const int64_t tokens = s->cu_new ? s->tokens : d->b * d->s_q, lim = (int64_t(1) << 31) - 4096;
    if (tokens > lim || tokens * (d->h > 2 * d->h_kv ? d->h : 2 * d->h_kv) > lim) return ATTN_ERR_UNSUPPORTED;
    out->table = s->page_table;
    out->table_stride = s->table_stride;
    out->lens = s->lens;
    out->cu = s->cu_new;
    out->b = int(d->b); out->s_q = int(d->s_q); out->tokens = int(tokens);
    out->cap = int(d->s_kv);
    return ATTN_OK;
}

// A cache to be written has a place for every row and every scale: no stride of 0, which a cache that is read may have (one
// scale for all rows), along what it has several of.
bool own_places(const attn_sdpa_desc_t *d, const attn_paged_cache_t *c)
{
    auto apart = [&](int64_t sp, int64_t ss, int64_t sh) {
        return (c->n_pages < 2 || sp > 0) && (c->page_size < 2 || ss > 0) && (d->h_kv < 2 || sh > 0);
    };
    return apart(c->sp, c->ss, c->sh) && (c->type != ATTN_E4M3 || apart(c->scale_sp, c->scale_ss, c->scale_sh));
}

constexpr size_t kPagedCopyBytes = 256;

attn_status_t paged_copy_call(bool write, const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache,
                              const attn_paged_seqs_t *seqs, attn_view_t k, attn_view_t v, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    PagedCopyArgs a;
    std::memset(&a, 0, sizeof a);
    attn_status_t st = check_paged(desc, cache, &a.cache);
    if (st || (st = check_paged_call(desc, cache, seqs, &a.seqs))) return st;
    if (write && !own_places(desc, cache)) return ATTN_ERR_INVALID;
    if ((st = check_view(k, a.seqs.tokens)) || (st = check_view(v, a.seqs.tokens))) return st;
    if ((st = check_ws(workspace, workspace_bytes, kPagedCopyBytes))) return st;
    a.dtype = desc->dtype;
    a.h_kv = int(desc->h_kv); a.d = int(desc->d);
    a.k = to_view(k, a.seqs.cu != nullptr); a.v = to_view(v, a.seqs.cu != nullptr);
    a.status = static_cast<uint32_t *>(workspace);
    return cuda_status(launch_paged_copy(a, write, static_cast<cudaStream_t>(stream)));
}

struct PagedLayout {
    size_t flags, rec, ml, o, total;
};

// The kernel a call takes, by its rows (new tokens x query heads of a kv head): the tensor-core one from 17 on, or from 49
// over an e4m3 cache, whose conversion takes it longer than the other takes to read the keys once for every 16 rows.
// (us, cold L2, 16 sequences of 500 to 6000 tokens, 32 / 8 heads of 128, mma.sync / tcgen05: 16 bits, 16 rows 60 / 80, 24 rows
// 82 / 82, 48 rows 110 / 83; e4m3, 16 rows 46 / 109, 48 rows 89 / 112, 64 rows 108 / 109.)
PagedShape paged_shape(const attn_sdpa_desc_t *d, bool eight)
{
    if (d->s_q * (d->h / d->h_kv) > (eight ? 48 : 16)) return paged_chunk_shape(d->h, d->h_kv, d->s_q);
    return paged_decode_shape(d->h, d->h_kv, d->d, d->s_q, eight);
}

PagedLayout paged_layout(const attn_sdpa_desc_t *d, const PagedShape &p)
{
    const size_t parts = size_t(p.shares) * 2;
    PagedLayout L;
    L.flags = Workspace::align(64 * sizeof(uint32_t));
    L.rec = L.flags + Workspace::align(size_t(p.shares) * sizeof(uint32_t));
    L.ml = L.rec + Workspace::align(parts * sizeof(int4));
    L.o = L.ml + Workspace::align(parts * size_t(p.rows) * sizeof(float2));
    L.total = L.o + Workspace::align(parts * size_t(p.rows) * size_t(d->d) * sizeof(float));
    return L;
}

}  // namespace

attn_status_t paged_cache_workspace_size(const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache, size_t *bytes)
{
    PagedCache c;
    const attn_status_t st = check_paged(desc, cache, &c);
    if (st) return st;
    if (!bytes) return ATTN_ERR_NULLPTR;
    *bytes = kPagedCopyBytes;
    return ATTN_OK;
}

attn_status_t paged_cache_write(const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache,
                                const attn_paged_seqs_t *seqs, attn_view_t k, attn_view_t v, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    return paged_copy_call(true, desc, cache, seqs, k, v, workspace, workspace_bytes, stream);
}

attn_status_t paged_cache_read(const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache,
                               const attn_paged_seqs_t *seqs, attn_view_t k, attn_view_t v, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    return paged_copy_call(false, desc, cache, seqs, k, v, workspace, workspace_bytes, stream);
}

attn_status_t sdpa_paged_workspace_size(const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache, size_t *bytes)
{
    PagedCache c;
    const attn_status_t st = check_paged(desc, cache, &c);
    if (st) return st;
    if (!bytes) return ATTN_ERR_NULLPTR;
    // (a call without tokens takes the other kernel, whose partial results are always smaller)
    *bytes = paged_layout(desc, paged_shape(desc, c.type == ATTN_E4M3)).total;
    return ATTN_OK;
}

attn_status_t sdpa_paged_fwd(const attn_sdpa_desc_t *desc, const attn_paged_cache_t *cache,
                             const attn_paged_seqs_t *seqs, attn_view_t q, attn_view_t o, float *lse, void *workspace,
                             size_t workspace_bytes, void *stream)
{
    PagedAttnArgs a;
    std::memset(&a, 0, sizeof a);
    attn_status_t st = check_paged(desc, cache, &a.cache);
    if (st || (st = check_paged_call(desc, cache, seqs, &a.seqs))) return st;
    if ((st = check_view(q, a.seqs.tokens)) || (st = check_view(o, a.seqs.tokens))) return st;
    if (reinterpret_cast<uintptr_t>(lse) & 3) return ATTN_ERR_ALIGN;
    const bool eight = a.cache.type == ATTN_E4M3;
    PagedShape shape = paged_shape(desc, eight);
    if ((st = check_ws(workspace, workspace_bytes, paged_layout(desc, shape).total))) return st;
    // no queries to make a tensor map of: the other kernel writes the status
    if (shape.chunk && a.seqs.tokens == 0) shape = paged_decode_shape(desc->h, desc->h_kv, desc->d, 1, eight);
    const PagedLayout L = paged_layout(desc, shape);
    a.dtype = desc->dtype;
    a.h = int(desc->h); a.h_kv = int(desc->h_kv); a.d = int(desc->d);
    a.causal = desc->mask == ATTN_CAUSAL_BOTTOM_RIGHT;
    a.scale = float(desc->scale);
    a.q = to_view(q, a.seqs.cu != nullptr); a.o = to_view(o, a.seqs.cu != nullptr);
    a.lse = lse;
    char *ws = static_cast<char *>(workspace);
    a.status = reinterpret_cast<uint32_t *>(ws);
    if (a.cache.n_pages == 0) a.cache.k = a.cache.v = ws;  // (for the tensor maps: an address, which nothing reads)
    a.flags = reinterpret_cast<uint32_t *>(ws + L.flags);
    a.rec = reinterpret_cast<int4 *>(ws + L.rec);
    a.part_ml = reinterpret_cast<float2 *>(ws + L.ml);
    a.part_o = reinterpret_cast<float *>(ws + L.o);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = shape.chunk ? launch_paged_chunk(a, shape, s) : launch_paged_decode(a, shape, s);
    return cuda_status(e != cudaSuccess ? e : launch_paged_join(a, shape, s));
}

// --------------------------------------------------- query / key norm and rotation

namespace {

attn_status_t check_qk_desc(const attn_qk_norm_desc_t *d)
{
    if (!d) return ATTN_ERR_NULLPTR;
    if (d->dtype != ATTN_F16 && d->dtype != ATTN_BF16) return ATTN_ERR_INVALID;
    if (d->b < 1 || d->s < 0 || d->h < 0 || d->h_kv < 0 || d->h + d->h_kv < 1) return ATTN_ERR_INVALID;
    if (d->rotary_dim < 0 || d->rotary_dim > d->d) return ATTN_ERR_INVALID;
    if ((d->interleaved != 0 && d->interleaved != 1) || (d->weight_fp32 != 0 && d->weight_fp32 != 1))
        return ATTN_ERR_INVALID;
    if (!std::isfinite(d->eps) || !(float(d->eps) > 0.f)) return ATTN_ERR_INVALID;
    if (d->rotary_dim > 0 && (d->max_pos < 1 || d->max_pos > INT32_MAX)) return ATTN_ERR_INVALID;
    if (d->d != 64 && d->d != 128 && d->d != 192) return ATTN_ERR_UNSUPPORTED;
    if (d->rotary_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
    // 32-bit work item indices inside the kernels
    const int64_t lim = int64_t(1) << 31;
    if (d->h >= lim || d->h_kv >= lim || d->b >= lim || d->s >= lim || d->b * d->s >= lim) return ATTN_ERR_UNSUPPORTED;
    const int64_t hmax = d->h > d->h_kv ? d->h : d->h_kv;
    if (d->s > 0 && d->b * d->s > (lim - 1) / hmax) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

size_t qk_part_offset() { return Workspace::align(64 * sizeof(uint32_t)); }
size_t qk_bwd_bytes(const attn_qk_norm_desc_t *d)
{
    return qk_part_offset() + Workspace::align(size_t(kQkBlocks + 2) * size_t(d->d) * sizeof(float));
}

attn_status_t qk_norm_call(const attn_qk_norm_desc_t *d, bool backward, attn_view_t q, attn_view_t k, attn_view_t dyq,
                           attn_view_t dyk, const void *wq, const void *wk, const float *cos, const float *sin,
                           const int32_t *positions, attn_view_t yq, attn_view_t yk, float *dwq, float *dwk,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    attn_status_t st = check_qk_desc(d);
    if (st) return st;
    const int64_t rows_q = d->b * d->s * d->h, rows_k = d->b * d->s * d->h_kv;
    if ((st = check_view(q, rows_q)) || (st = check_view(k, rows_k)) || (st = check_view(yq, rows_q)) ||
        (st = check_view(yk, rows_k)))
        return st;
    if (backward && ((st = check_view(dyq, rows_q)) || (st = check_view(dyk, rows_k)))) return st;
    if (d->rotary_dim > 0 && d->s > 0) {
        if (!cos || !sin) return ATTN_ERR_NULLPTR;
        if (!aligned16(cos) || !aligned16(sin) || (reinterpret_cast<uintptr_t>(positions) & 3)) return ATTN_ERR_ALIGN;
    }
    if ((d->h && !aligned16(wq)) || (d->h_kv && !aligned16(wk))) return ATTN_ERR_ALIGN;
    if ((reinterpret_cast<uintptr_t>(dwq) & 3) || (reinterpret_cast<uintptr_t>(dwk) & 3)) return ATTN_ERR_ALIGN;
    if ((st = check_ws(workspace, workspace_bytes, backward ? qk_bwd_bytes(d) : qk_part_offset()))) return st;
    QkNormArgs a;
    std::memset(&a, 0, sizeof a);
    a.dtype = d->dtype; a.weight_fp32 = d->weight_fp32; a.interleaved = d->interleaved;
    a.b = d->b; a.s = d->s; a.d = d->d; a.rot = d->rotary_dim; a.max_pos = d->max_pos;
    a.eps = float(d->eps);
    a.cos = cos; a.sin = sin; a.pos = positions;
    char *ws = static_cast<char *>(workspace);
    a.status = reinterpret_cast<uint32_t *>(ws);
    QkSide &sq = a.side[0], &sk = a.side[1];
    sq.x = to_view(q, false); sq.dy = to_view(dyq, false); sq.y = to_view(yq, false);
    sk.x = to_view(k, false); sk.dy = to_view(dyk, false); sk.y = to_view(yk, false);
    sq.w = wq; sk.w = wk;
    sq.h = d->h; sk.h = d->h_kv;
    sq.dw = d->h ? dwq : nullptr; sk.dw = d->h_kv ? dwk : nullptr;
    // the query side's shares first, the key side's behind them (split when the blocks are dealt)
    sq.part = sk.part = reinterpret_cast<float *>(ws + qk_part_offset());
    return cuda_status(launch_qk_norm(a, backward, static_cast<cudaStream_t>(stream)));
}

}  // namespace

attn_status_t qk_norm_rope_workspace_size(const attn_qk_norm_desc_t *desc, size_t *fwd_bytes, size_t *bwd_bytes)
{
    const attn_status_t st = check_qk_desc(desc);
    if (st) return st;
    if (fwd_bytes) *fwd_bytes = qk_part_offset();
    if (bwd_bytes) *bwd_bytes = qk_bwd_bytes(desc);
    return ATTN_OK;
}

attn_status_t qk_norm_rope_fwd(const attn_qk_norm_desc_t *desc, attn_view_t q, attn_view_t k, const void *q_weight,
                               const void *k_weight, const float *cos, const float *sin, const int32_t *positions,
                               attn_view_t q_out, attn_view_t k_out, void *workspace, size_t workspace_bytes,
                               void *stream)
{
    const attn_view_t none = {nullptr, 0, 0, 0};
    return qk_norm_call(desc, false, q, k, none, none, q_weight, k_weight, cos, sin, positions, q_out, k_out, nullptr,
                        nullptr, workspace, workspace_bytes, stream);
}

attn_status_t qk_norm_rope_bwd(const attn_qk_norm_desc_t *desc, attn_view_t q, attn_view_t k, attn_view_t dq_out,
                               attn_view_t dk_out, const void *q_weight, const void *k_weight, const float *cos,
                               const float *sin, const int32_t *positions, attn_view_t dq, attn_view_t dk,
                               float *dq_weight, float *dk_weight, void *workspace, size_t workspace_bytes,
                               void *stream)
{
    return qk_norm_call(desc, true, q, k, dq_out, dk_out, q_weight, k_weight, cos, sin, positions, dq, dk, dq_weight,
                        dk_weight, workspace, workspace_bytes, stream);
}

attn_status_t attn_set_main_kernel_events(void *before, void *after)
{
    g_ev_before = static_cast<cudaEvent_t>(before);
    g_ev_after = static_cast<cudaEvent_t>(after);
    return ATTN_OK;
}

attn_status_t attn_query_status(void *workspace, void *stream, uint32_t *device_flags)
{
    if (!workspace || !device_flags) return ATTN_ERR_NULLPTR;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if ((e = cudaStreamSynchronize(s)) != cudaSuccess) return cuda_status(e);
    uint32_t flags = 0;
    if ((e = cudaMemcpy(&flags, workspace, sizeof flags, cudaMemcpyDeviceToHost)) != cudaSuccess) return cuda_status(e);
    // on the stream: cudaMemset may return first, and would then race with the next call's status on this stream
    if (flags && (e = cudaMemsetAsync(workspace, 0, sizeof flags, s)) != cudaSuccess) return cuda_status(e);
    *device_flags = flags;
    return flags ? ATTN_ERR_DEVICE : ATTN_OK;
}

}  // extern "C"
