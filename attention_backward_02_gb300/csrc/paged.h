// paged.h -- argument bundles of the paged key / value cache: its write and read
// kernels and the attention of new tokens over it.
#pragma once

#include "plan.h"

namespace attn {

constexpr int kPagedMaxGroup = 128;  // query heads that may share a key / value head
constexpr int kPagedCtas = 152;      // SMs: a constant, as the workspace size must not depend on a CUDA call

// Pages of k and v (same strides, in elements) and, for e4m3, the fp32 scales of their rows.
struct PagedCache {
    void *k, *v;
    float *k_scale, *v_scale;
    int type;                     // ATTN_F16, ATTN_BF16 or ATTN_E4M3
    int n_pages, shift;           // page size: 1 << shift tokens
    int none;                     // a page coordinate out of every range: max(n_pages, 1)
    int64_t sp, sc_sp;            // stride of a page; within one, offsets fit 32 bits:
    int sh, ss, sc_sh, sc_ss;     // strides of a head and a token
};

// Where the sequences and their new tokens lie.
struct PagedSeqs {
    const int32_t *table;         // [b] rows of page ids
    int64_t table_stride;
    const int32_t *lens;          // [b] tokens cached, the new ones among them
    const int32_t *cu;            // [b + 1] first rows of the sequences' new tokens (NULL: s_q each)
    int b, s_q, tokens;           // tokens: rows of all new tokens
    int cap;                      // most tokens a sequence may have cached

    // First row and number of new tokens of sequence n, in bounds whatever cu holds; *bad is set where that changed them.
    __host__ __device__ __forceinline__ void rows(int n, int *first, int *m, bool *bad) const
    {
        if (!cu) {
            *first = n * s_q;
            *m = s_q;
            return;
        }
        const int a = cu[n], e = cu[n + 1];
        *first = a < 0 ? 0 : (a > tokens ? tokens : a);
        const int end = e < *first ? *first : (e > tokens ? tokens : e);
        *m = end - *first;
        if (*first != a || end != e) *bad = true;
    }
    // Its cached tokens, in [0, cap].
    __host__ __device__ __forceinline__ int len(int n, bool *bad) const
    {
        const int l = lens[n], c = l < 0 ? 0 : (l > cap ? cap : l);
        if (c != l) *bad = true;
        return c;
    }
};

struct PagedCopyArgs {
    int dtype;
    int h_kv, d;
    View k, v;                    // rows of the new tokens
    PagedCache cache;
    PagedSeqs seqs;
    uint32_t *status;
};

// Workspace of the attention (all offsets 256-byte aligned), for C work shares of R rows:
//   status uint32[64];  flags uint32[C]   what a share found wrong
//   rec    int32 [C][8]                   its two partial results' units
//   ml     f32   [C][2][R][2]             their maxima (log2 units) and sums
//   o      f32   [C][2][R][d]             their unnormalised outputs
struct PagedAttnArgs {
    int dtype;
    int h, h_kv, d, causal;
    float scale;
    View q, o;
    float *lse;                   // [b][h][s_q], packed [h][tokens]; NULL: not wanted
    PagedCache cache;
    PagedSeqs seqs;
    uint32_t *status, *flags;
    int4 *rec;
    float2 *part_ml;
    float *part_o;
};

// The kernel that a call takes: rows of a share's partial result, shares, and how a unit's rows name new tokens and
// query heads.  A unit has `row_blocks` head blocks to a kv head and `groups` groups of rows; row r of a group is token
// r / heads and head r % heads of the block, for `tokens` tokens.
struct PagedShape {
    bool chunk;                   // paged_chunk.cu (else paged_decode.cu)
    int rows, shares;
    int groups, tokens, heads, row_blocks;
};
PagedShape paged_decode_shape(int64_t h, int64_t h_kv, int64_t d, int64_t s_q, bool eight);
PagedShape paged_chunk_shape(int64_t h, int64_t h_kv, int64_t s_q);

cudaError_t launch_paged_copy(const PagedCopyArgs &a, bool write, cudaStream_t s);
cudaError_t launch_paged_decode(const PagedAttnArgs &a, const PagedShape &shape, cudaStream_t s);
cudaError_t launch_paged_chunk(const PagedAttnArgs &a, const PagedShape &shape, cudaStream_t s);
cudaError_t launch_paged_join(const PagedAttnArgs &a, const PagedShape &shape, cudaStream_t s);

}  // namespace attn
