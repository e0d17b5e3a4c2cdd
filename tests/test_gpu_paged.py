"""GPU parity of the paged cache's calls with their definitions (oracle/paged.py); the attention's bounds are derived in
tests/paged_problem.py, the cache's rows are compared bit by bit."""
import numpy as np
import pytest

from oracle import paged as P
from tests.paged_problem import Problem

pytestmark = pytest.mark.gpu


def _bits(t):
    import torch
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32).cpu()


# ------------------------------------------------------------------------------------ write and read

COPIES = [
    # dtype, cache, lens, new, hk, d, kw
    ("float16", "same", [1], [1], 1, 64, dict(packed=False)),
    ("bfloat16", "e4m3", [1], [1], 1, 128, dict(packed=False)),
    ("bfloat16", "e4m3", [5, 17, 16, 300], [5, 2, 0, 33], 8, 128, dict(page=16)),
    ("float16", "e4m3", [129, 64, 640], [100, 64, 1], 3, 64, dict(page=64, layout="hnd", scales_by_head=True)),
    ("bfloat16", "same", [70, 260], [70, 259], 12, 128, dict(page=32, layout="kv")),
    ("float16", "e4m3", [1000, 2000, 513], [512] * 3, 8, 128, dict(page=256, packed=False)),
    ("bfloat16", "e4m3", [3, 0, 9], [5, 4, 9], 2, 64, dict()),           # more new tokens than cached ones
    ("float16", "same", [40] * 300, [1] * 300, 70, 64, dict(packed=False)),  # more heads than a block's rows
    ("bfloat16", "e4m3", [2500, 4000], [2500, 3999], 16, 128, dict(page=64, extra_rows=37)),
]


def _rows(p, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(p.rows, p.hk, p.d, generator=g) * torch.exp(2 * torch.randn(p.rows, p.hk, 1, generator=g))
    return x.to(p.dt)


def _expected_pool(p, i, x):
    """Pool and scales i after the write of rows x, as bit patterns by slot."""
    import torch
    pool = _bits(p.pool[i]).reshape(-1, p.hk, p.d).clone()
    scales = _bits(p.scales[i]).reshape(-1, p.hk).clone() if p.eight else None
    for n, m in enumerate(p.new):
        c = len(p.rows_of[n])
        for t in range(m):
            pos = c - m + t
            if pos < 0:
                continue
            row, slot = x[p.starts[n] + t], p.rows_of[n][pos]
            if p.eight:
                code, sc = P.quantise(row.float().numpy())
                pool[slot] = torch.from_numpy(code)
                scales[slot] = _bits(torch.from_numpy(sc))
            else:
                pool[slot] = _bits(row)
    return pool, scales


@pytest.mark.parametrize("case", COPIES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", "")[:80])
def test_write_then_read(case):
    import torch
    dtype, cache, lens, new, hk, d, kw = case
    p = Problem(dtype, cache, lens, new, hk, hk, d, seed=len(lens) + d, **kw)
    x = [_rows(p, s) for s in (1, 2)]
    ws = p.ab.paged_cache_write(p.desc, p.cache, p.dtable, p.dlens, *(p.dense(t) for t in x), cu_new=p.cu)
    assert p.ab.attn_query_status(ws) == 0
    want = [_expected_pool(p, i, x[i]) for i in range(2)]
    for i in range(2):
        assert torch.equal(_bits(p.cpool[i]).reshape(-1, hk, d), want[i][0])
        if p.eight:
            assert torch.equal(_bits(p.cscales[i]).reshape(-1, hk), want[i][1])
    out = [torch.full_like(p.dense(t), 7.0) for t in x]
    ws = p.ab.paged_cache_read(p.desc, p.cache, p.dtable, p.dlens, *out, cu_new=p.cu)
    assert p.ab.attn_query_status(ws) == 0
    for i in range(2):
        got = p.packed_of(out[i]).cpu()
        for n, m in enumerate(new):
            for t in range(0, m, max(1, m // 50)):
                pos, row = len(p.rows_of[n]) - m + t, got[p.starts[n] + t]
                if pos < 0:
                    assert bool((row == 0).all())
                elif p.eight:
                    slot = p.rows_of[n][pos]
                    val = P.values(want[i][0][slot].numpy(), want[i][1][slot].view(torch.float32).numpy())
                    assert torch.equal(row, torch.from_numpy(val).to(p.dt))
                else:
                    assert torch.equal(row, x[i][p.starts[n] + t])
        assert bool((got[p.starts[-1]:] == 7).all())  # rows behind the last sequence


def test_rows_of_special_values():
    """All zeros; a NaN; infinities beside finite elements; nothing finite; the type's largest and smallest numbers."""
    import torch
    for dtype in ("bfloat16", "float16"):
        p = Problem(dtype, "e4m3", [8], [8], 1, 1, 64, packed=False)
        x = torch.randn(8, 1, 64).to(p.dt)
        x[0] = 0
        x[1, 0, 3] = float("nan")
        x[2, 0, 5], x[2, 0, 6] = float("inf"), -float("inf")
        x[3] = float("inf")
        x[4] = float("nan")
        x[5] = torch.finfo(p.dt).max
        x[6] = torch.finfo(p.dt).smallest_normal * (x[6] > 0)
        x[7] = 2.0 ** (-133 if dtype == "bfloat16" else -24)  # subnormal
        ws = p.ab.paged_cache_write(p.desc, p.cache, p.dtable, p.dlens, p.dense(x), p.dense(x))
        assert p.ab.attn_query_status(ws) == 0
        code, sc = P.quantise(x.float().numpy())
        slots = p.rows_of[0]
        got = _bits(p.cpool[0]).reshape(-1, 1, 64)[slots].numpy()
        nan = (code & 127) == 127
        assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], code[~nan])
        assert np.array_equal(p.cscales[0].cpu().numpy().reshape(-1, 1)[slots], sc)
        assert bool(np.all(got[0] & 127 == 0)) and bool(np.all(got[3] == 0x7e))


def test_bad_pages_lengths_and_counts_are_flagged():
    import torch
    # a page id that is none: its tokens are not written and read as zeros, the others are
    p = Problem("bfloat16", "e4m3", [40, 33], [40, 33], 2, 2, 64)
    p.dtable[0, 1] = p.cpool[0].shape[0]
    p.dtable[1, 0] = -1
    before = [_bits(t).clone() for t in p.cpool]
    x = _rows(p, 3)
    ws = p.ab.paged_cache_write(p.desc, p.cache, p.dtable, p.dlens, p.dense(x), p.dense(x), cu_new=p.cu)
    assert p.ab.attn_query_status(ws) == 2
    after = _bits(p.cpool[0]).reshape(-1, 2, 64)
    lost = set(p.rows_of[0][16:32]) | set(p.rows_of[1][:16])
    for n in range(2):
        for t, slot in enumerate(p.rows_of[n]):
            old = before[0].reshape(-1, 2, 64)[slot]
            new = torch.from_numpy(P.quantise(x[p.starts[n] + t].float().numpy())[0])
            assert torch.equal(after[slot], old if slot in lost else new)
    out = [torch.full_like(p.dense(x), 7.0) for _ in range(2)]
    ws = p.ab.paged_cache_read(p.desc, p.cache, p.dtable, p.dlens, *out, cu_new=p.cu)
    assert p.ab.attn_query_status(ws) == 2
    assert bool((out[0][16:32] == 0).all()) and bool((out[0][40:56] == 0).all()) and bool((out[0][:16] != 0).any())
    # lengths and counts out of range
    p = Problem("float16", "same", [20, 20], [20, 20], 2, 2, 64)
    x = _rows(p, 4)
    for lens, cu, flag in (([-1, 20], [0, 20, 40], 2), ([20, 1 << 30], [0, 20, 40], 2), ([20, 20], [0, 50, 40], 2),
                           ([20, 20], [-5, 20, 40], 2), ([20, 20], [0, 20, 40], 0)):
        p.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        p.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        ws = p.ab.paged_cache_write(p.desc, p.cache, p.dtable, p.dlens, p.dense(x), p.dense(x), cu_new=p.cu)
        assert p.ab.attn_query_status(ws) == flag, (lens, cu)
        ws = p.ab.paged_cache_read(p.desc, p.cache, p.dtable, p.dlens, *(torch.empty_like(p.dense(x)) for _ in range(2)), cu_new=p.cu)
        assert p.ab.attn_query_status(ws) == flag, (lens, cu)
        o = torch.empty_like(p.dense(p.q))
        ws = p.ab.sdpa_paged_fwd(p.desc, p.cache, p.dtable, p.dlens, p.dense(p.q), o, cu_new=p.cu)
        assert p.ab.attn_query_status(ws) == flag, (lens, cu)


# ----------------------------------------------------------------------------------------- attention

CASES = [
    # dtype, cache, lens, new, h, hk, d, kw
    ("float16", "same", [1], [1], 1, 1, 64, dict(packed=False)),
    ("bfloat16", "e4m3", [1], [1], 1, 1, 128, dict(packed=False)),
    ("bfloat16", "same", [1, 2, 15, 16, 17, 63, 64, 65, 0], [1] * 9, 4, 2, 128, dict(packed=False)),
    ("float16", "e4m3", [1, 2, 31, 32, 33, 127, 128, 129, 0], [1] * 9, 4, 2, 64, dict(packed=False, page=32)),
    ("float16", "same", [1000], [1], 12, 12, 64, dict(packed=False)),
    ("bfloat16", "e4m3", [5000, 1, 777, 2048], [1] * 4, 32, 8, 128, dict(packed=False, page=64, layout="hnd", scales_by_head=True)),
    ("bfloat16", "same", [3000, 129, 640], [1, 4, 2], 8, 1, 128, dict(layout="kv", page=128)),
    ("float16", "e4m3", [700, 300, 5], [3, 0, 5], 10, 2, 128, dict(page=256)),
    ("bfloat16", "same", [301, 9], [2, 1], 35, 1, 64, dict()),             # 35 query heads a kv head
    ("float16", "same", [200, 90], [7, 5], 6, 2, 128, dict(causal=False)),
    ("bfloat16", "e4m3", [200, 90], [16, 13], 5, 5, 64, dict(causal=False, packed=True, extra_rows=9)),
    ("float16", "same", [3, 0, 20], [5, 4, 20], 4, 2, 64, dict()),          # rows before the first cached token
    ("bfloat16", "same", [150] * 200, [1] * 200, 2, 1, 64, dict(packed=False, page=32)),  # more units than shares
    # chunks
    ("float16", "same", [64, 200], [64, 200], 4, 4, 64, dict()),
    ("bfloat16", "same", [257, 128, 129], [257, 100, 1], 4, 1, 128, dict(page=64)),
    ("bfloat16", "e4m3", [1500, 700], [333, 700], 8, 2, 128, dict(page=32, layout="hnd")),
    ("float16", "e4m3", [900, 300], [300, 300], 12, 12, 64, dict(page=16, packed=False)),
    ("bfloat16", "same", [520, 30, 77], [130, 60, 0], 40, 8, 128, dict(page=128, extra_rows=11)),  # 30 rows without keys
    ("float16", "same", [1030], [515], 71, 1, 64, dict(packed=False, page=256)),
    ("bfloat16", "e4m3", [400, 131], [200, 131], 3, 1, 64, dict(causal=False, page=64)),
    ("bfloat16", "same", [2000], [1000], 128, 1, 128, dict(page=64)),
    ("float16", "same", [3000], [150], 16, 2, 128, dict(packed=False, page=16, layout="hnd")),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", "")[:80])
def test_attention_parity(case):
    import torch
    p = Problem(*case[:7], seed=case[6] + len(case[2]), **case[7])
    o, lse = p.attend()
    p.check(o, lse)
    assert bool(p.packed_of(o)[p.starts[-1]:].isnan().all())  # rows behind the last sequence
    again, lse2 = p.attend()
    assert torch.equal(o.nan_to_num(9), again.nan_to_num(9)) and torch.equal(lse.nan_to_num(9), lse2.nan_to_num(9))
    alone, _ = p.attend(lse=False)
    assert torch.equal(o.nan_to_num(9), alone.nan_to_num(9))


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale", [-0.17, 0.0, 3.0])
def test_scales_of_every_sign(cache, new, scale):
    """A negative scale, one of zero (the mean of the visible values) and a large one."""
    p = Problem("bfloat16", cache, [200, 77], [new, new], 4, 2, 64, packed=False, seed=11)
    p.desc.scale = scale
    p.scale = scale
    p.check(*p.attend())


@pytest.mark.parametrize("new", [3, 50])
def test_padded_in_front_and_queries_by_head(new):
    """Fixed-length calls whose sequences have fewer cached tokens than new ones, with [B, h, S, D] storage."""
    import torch
    p = Problem("float16", "e4m3", [2, 0, 60], [new] * 3, 8, 2, 128, packed=False, seed=12)
    q = p.dense(p.q).contiguous()
    o, lse = p.attend(q=q, o=torch.full_like(q, float("nan")))
    p.check(o, lse)
    x = _rows(p, 13)
    ws = p.ab.paged_cache_write(p.desc, p.cache, p.dtable, p.dlens, p.dense(x).contiguous(), p.dense(x), cu_new=p.cu)
    assert p.ab.attn_query_status(ws) == 0
    for i in range(2):
        pool, scales = _expected_pool(p, i, x)
        assert torch.equal(_bits(p.cpool[i]).reshape(-1, 2, 128), pool)


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("hint,new", [(1, [300, 1, 7]), (1000, [1, 2, 1]), (0, [5, 40, 1])])
def test_an_expected_count_only_chooses_the_kernel(cache, hint, new):
    """desc.s_q of packed calls: longer and shorter chunks than it says are computed all the same."""
    p = Problem("bfloat16", cache, [400, 90, 50], new, 8, 2, 64, seed=14)
    p.desc.s_q = hint
    p.check(*p.attend())


def test_a_cache_without_room():
    """s_kv = 0: nothing is read, every row is empty."""
    import torch
    for new in (1, 40):
        p = Problem("float16", "same", [3, 2], [new, new], 4, 2, 64, packed=False)
        p.desc.s_kv = 0
        table, lens = torch.empty(2, 0, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
        q = p.dense(p.q)
        o, lse = torch.full_like(q, 3), torch.empty(2, 4, new, device="cuda")
        ws = p.ab.sdpa_paged_fwd(p.desc, p.cache, table, lens, q, o, lse=lse)
        assert p.ab.attn_query_status(ws) == 0
        assert bool((o == 0).all()) and bool(lse.isposinf().all())
        lens[1] = 1
        ws = p.ab.sdpa_paged_fwd(p.desc, p.cache, table, lens, q, o, lse=lse)
        assert p.ab.attn_query_status(ws) == 2


def test_two_threads_on_two_streams():
    """Two host threads, each with a stream and a workspace, over one cache handle."""
    import threading
    import torch
    p = Problem("bfloat16", "e4m3", [3000, 700], [60, 60], 8, 2, 128, packed=False, seed=15)
    one = Problem("bfloat16", "e4m3", [3000, 700], [1, 1], 8, 2, 128, packed=False, seed=15)
    one.cache, one.dtable = p.cache, p.dtable  # (the same seed: the same pages)
    want = [p.attend()[0], one.attend()[0]]
    got, errors = [[], []], []

    def work(i, x):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(30):
                    got[i].append(x.attend(flags=None, stream=s)[0])
                s.synchronize()
        except Exception as e:
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i, x)) for i, x in enumerate((p, one))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for i in range(2):
        assert len(got[i]) == 30 and all(torch.equal(o, want[i]) for o in got[i])


def test_packed_views_are_refused():
    import torch
    p = Problem("float16", "same", [5], [5], 2, 2, 64)
    v = p.ab.attn_view_t(p.dense(p.q).data_ptr(), 0, 64, 128)
    with pytest.raises(ValueError):
        p.ab.sdpa_paged_fwd(p.desc, p.cache, p.dtable, p.dlens, v, v, cu_new=p.cu)
    with pytest.raises(ValueError):  # a page table of another type
        p.ab.sdpa_paged_fwd(p.desc, p.cache, p.dtable.long(), p.dlens, p.dense(p.q), p.dense(p.q), cu_new=p.cu)
    with pytest.raises(ValueError):  # rows of another head count
        p.ab.paged_cache_write(p.desc, p.cache, p.dtable, p.dlens, p.dense(p.q)[:, :1], p.dense(p.q)[:, :1], cu_new=p.cu)
    with pytest.raises(p.ab.AttnError):  # too small a workspace
        p.ab.sdpa_paged_fwd(p.desc, p.cache, p.dtable, p.dlens, p.dense(p.q), p.dense(p.q), cu_new=p.cu,
                            workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("new", [1, 40])
def test_a_bad_page_reads_as_zeros(new):
    p = Problem("bfloat16", "same", [200, 300], [new, new], 4, 2, 128, seed=3)
    for n, i in ((0, 2), (1, 0)):
        p.dtable[n, i] = -3
        p.pool[0].reshape(-1, 2, 128)[p.rows_of[n][16 * i:16 * i + 16]] = 0
        p.pool[1].reshape(-1, 2, 128)[p.rows_of[n][16 * i:16 * i + 16]] = 0
    o, lse = p.attend(flags=2)
    p.check(o, lse)


@pytest.mark.parametrize("eight", [False, True])
def test_no_pages_and_no_tokens(eight):
    """A cache without pages: every key reads as zeros, and the call says so.  A call without new tokens: its status."""
    import torch
    import attention_backward_02_gb300 as ab
    pool = torch.empty(0, 16, 2, 64, dtype=torch.uint8 if eight else torch.float16, device="cuda")
    pool = pool.view(torch.float8_e4m3fn) if eight else pool
    sc = torch.empty(0, 16, 2, device="cuda") if eight else None
    cache = ab.paged_cache(pool, pool, k_scale=sc, v_scale=sc)
    table, lens = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.tensor([60], dtype=torch.int32, device="cuda")
    for new in (1, 50):
        desc = ab.sdpa_desc(dtype=ab.ATTN_F16, b=1, h=4, h_kv=2, s_q=new, s_kv=64, d=64, scale=0.125, mask=ab.ATTN_MASK_NONE)
        q = torch.randn(1, 4, new, 64, dtype=torch.float16, device="cuda")
        o, lse = torch.full_like(q, 3), torch.empty(1, 4, new, device="cuda")
        ws = ab.sdpa_paged_fwd(desc, cache, table, lens, q, o, lse=lse)
        assert ab.attn_query_status(ws) == 2
        assert bool((o == 0).all()) and bool(((lse - np.log(60.0)).abs() <= 2.0 ** -18).all())
        cu = torch.zeros(2, dtype=torch.int32, device="cuda")
        none = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
        ws = ab.sdpa_paged_fwd(desc, cache, table, lens, none, none, cu_new=cu)
        assert ab.attn_query_status(ws) == 0
        lens[0] = 65
        ws = ab.sdpa_paged_fwd(desc, cache, table, lens, none, none, cu_new=cu, workspace=ws)
        assert ab.attn_query_status(ws) == 2
        lens[0] = 60


@pytest.mark.parametrize("new", [1, 6, 90])
def test_shared_pages_and_strided_rows(new):
    """Two sequences with the same first pages; queries as a slice of a fused projection, outputs into one."""
    import torch
    p = Problem("float16", "same", [96 + new, 96 + new], [new, new], 4, 2, 64, packed=False, seed=5)
    p.dtable[1, :6] = p.dtable[0, :6]
    p.rows_of[1][:96] = p.rows_of[0][:96]
    fused = torch.full((2, new, 8, 64), float("nan"), dtype=p.dt, device="cuda")
    fused[:, :, :4] = p.q.view(2, new, 4, 64).cuda()
    o, lse = p.attend(q=fused[:, :, :4].permute(0, 2, 1, 3), o=fused[:, :, 4:].permute(0, 2, 1, 3))
    p.check(o, lse)
    assert torch.equal(fused[:, :, :4], p.q.view(2, new, 4, 64).cuda())


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("new", [1, 5, 70])
@pytest.mark.parametrize("dim", [0, 1, 2])
def test_inputs_that_repeat(cache, new, dim):
    """Queries, and rows to write, that are the same for all sequences, heads or tokens (a stride of 0, as expand makes
    them): the bits of the same calls on copies."""
    import torch
    runs = []
    for copies in (False, True):
        p = Problem("bfloat16", cache, [90 + new, 7 + new, 200], [new] * 3, 8, 2, 128, packed=False, seed=15)
        g = torch.Generator().manual_seed(16)
        def rows(heads):
            shape = [3, heads, new, 128]
            x = torch.randn(*(1 if i == dim else n for i, n in enumerate(shape)), generator=g).to(p.dt).cuda().expand(*shape)
            return x.contiguous() if copies else x
        ws = p.ab.paged_cache_write(p.desc, p.cache, p.dtable, p.dlens, rows(2), rows(2))
        assert p.ab.attn_query_status(ws) == 0
        q = rows(8)
        runs.append([*p.cpool, *p.attend(q=q, o=torch.full((3, 8, new, 128), float("nan"), dtype=p.dt, device="cuda"))])
    for a, b in zip(*runs):
        assert torch.equal(_bits(a), _bits(b))


def test_extreme_scores_and_scales():
    """Scores far apart and values of very different size: e4m3 scales from 2^-20 to 2^10 in one sequence."""
    import torch
    for dtype in ("float16", "bfloat16"):
        for new in (1, 50):
            p = Problem(dtype, "e4m3", [900], [new], 4, 2, 64, seed=6)
            sc = torch.exp2(torch.arange(p.scales[1].numel()).reshape(p.scales[1].shape) % 31 - 20.0)
            if dtype == "float16":
                sc = sc * 2.0 ** -3  # values within the type's range
            live = ~p.scales[1].isnan()
            p.scales[1][live] = sc[live]
            p.cscales[1].copy_(p.scales[1])
            p.q *= 6
            p.check(*p.attend())


def test_a_nan_and_an_infinity_stay_in_their_sequence():
    import torch
    for new in (1, 70):
        p = Problem("bfloat16", "same", [100, 100, 100], [new] * 3, 2, 2, 64, seed=7)
        for t in p.cpool:
            t.reshape(-1, 2, 64)[p.rows_of[1][5]] = float("nan") if t is p.cpool[0] else float("inf")
        o, lse = p.attend()
        p.check(o, lse, only=(0, 2))
        assert bool(o[p.starts[1]:p.starts[2]].isnan().all())


def test_streams_threads_and_graphs():
    """On a stream of its own; two graphs with one workspace, replayed in turn as the cache grows."""
    import torch
    p = Problem("bfloat16", "e4m3", [0, 0], [1, 1], 8, 2, 128, packed=False, cap=200, page=16, seed=8)
    ab = p.ab
    pages = torch.randperm(26)[:26].int()
    p.dtable[:, :13] = pages.view(2, 13).cuda()
    raw = [torch.randn(200, 2, 2, 128).to(p.dt).cuda() for _ in range(2)]
    pool = [torch.zeros(26, 16, 2, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    sc = [torch.zeros(26, 16, 2, device="cuda") for _ in range(2)]
    cache = ab.paged_cache(*pool, k_scale=sc[0], v_scale=sc[1])
    ws = torch.empty(max(ab.sdpa_paged_workspace_size(p.desc, cache), ab.paged_cache_workspace_size(p.desc, cache)),
                     dtype=torch.uint8, device="cuda")
    k, v = (torch.empty(2, 2, 1, 128, dtype=p.dt, device="cuda") for _ in range(2))
    q, o = p.dense(p.q), torch.empty_like(p.dense(p.q))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        ab.paged_cache_write(p.desc, cache, p.dtable, p.dlens, k, v, workspace=ws)
        ab.sdpa_paged_fwd(p.desc, cache, p.dtable, p.dlens, q, o, workspace=ws)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        graphs.append(g)
    keys = [np.zeros((2, 200, 2, 128)) for _ in range(2)]
    for t in range(200):
        for i, x in enumerate((k, v)):
            x.copy_(raw[i][t].view(2, 2, 1, 128))
            keys[i][:, t] = P.values(*P.quantise(raw[i][t].float().cpu().numpy()))
        p.dlens.fill_(t + 1)
        graphs[t % 2].replay()
        if t in (0, 15, 16, 63, 128, 199):
            torch.cuda.synchronize()
            for n in range(2):
                ref = P.attention(p.q[n:n + 1].double().numpy(), keys[0][n, :t + 1], keys[1][n, :t + 1], 128 ** -0.5, True)[0]
                err = np.abs(o[n].permute(1, 0, 2).double().cpu().numpy() - ref)
                assert err.max() <= 2.0 ** -6 * np.abs(keys[1][n, :t + 1]).max()
    assert ab.attn_query_status(ws) == 0


def test_prompt_in_chunks_then_tokens():
    """A prompt written and attended to in chunks, then token by token, against the dense forward over the read-back
    rows: the same attention by another kernel (two roundings of the weights and of the output: 4 half steps of the
    largest value)."""
    import torch
    import attention_backward_02_gb300 as ab
    h, hk, d, total = 8, 2, 128, 700
    g = torch.Generator().manual_seed(9)
    dt = torch.bfloat16
    q, k, v = (torch.randn(1, total, n, d, generator=g).to(dt).cuda() for n in (h, hk, hk))
    for eight in (False, True):
        pages = 50
        kind = torch.uint8 if eight else dt
        pool = [torch.zeros(pages, 16, hk, d, dtype=kind, device="cuda") for _ in range(2)]
        pool = [t.view(torch.float8_e4m3fn) if eight else t for t in pool]
        sc = [torch.zeros(pages, 16, hk, device="cuda") if eight else None for _ in range(2)]
        cache = ab.paged_cache(*pool, k_scale=sc[0], v_scale=sc[1])
        table = torch.randperm(pages, generator=g).int()[None, :44].contiguous().cuda()
        out = torch.empty_like(q)
        at = 0
        for m in (256, 1, 300, 7, 129, 1, 1, 5):
            desc = ab.sdpa_desc(dtype=ab.ATTN_BF16, b=1, h=h, h_kv=hk, s_q=m, s_kv=total, d=d, scale=d ** -0.5,
                                mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
            lens = torch.tensor([at + m], dtype=torch.int32, device="cuda")
            rows = [t[:, at:at + m].permute(0, 2, 1, 3) for t in (q, k, v, out)]
            ab.paged_cache_write(desc, cache, table, lens, rows[1], rows[2])
            ws = ab.sdpa_paged_fwd(desc, cache, table, lens, rows[0], rows[3])
            assert ab.attn_query_status(ws) == 0
            at += m
        assert at == total
        desc = ab.sdpa_desc(dtype=ab.ATTN_BF16, b=1, h=h, h_kv=hk, s_q=total, s_kv=total, d=d, scale=d ** -0.5,
                            mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
        back = [torch.empty_like(t) for t in (k, v)]
        ab.paged_cache_read(desc, cache, table, lens, *(t.permute(0, 2, 1, 3) for t in back))
        if not eight:
            assert torch.equal(back[0], k) and torch.equal(back[1], v)
        want, lse = torch.empty_like(q), torch.empty(1, h, total, device="cuda")
        ab.sdpa_fwd_stats(desc, *(t.permute(0, 2, 1, 3) for t in (q, *back, want)), lse)
        # (the dense forward's keys are rounded once more than e4m3 numbers are: half a step of a score of up to 5)
        lim = (4 if not eight else 16) * 2.0 ** -8 * float(back[1].abs().max())
        assert float((out.float() - want.float()).abs().max()) <= lim


@pytest.mark.parametrize("eight,new", [(False, 1), (True, 1), (False, 40), (True, 40)])
def test_offsets_past_32_bits(eight, new):
    """Pages beyond 2^31 elements of the pools: a few tokens in the last ones."""
    import torch
    import attention_backward_02_gb300 as ab
    hk, d, page = 16, 128, 256
    pages = 4300 if not eight else 8300  # 2.25e9 elements, 4.35e9 bytes
    dt = torch.bfloat16
    pool = [torch.zeros(pages, page, hk, d, dtype=torch.uint8 if eight else dt, device="cuda") for _ in range(2)]
    assert pool[0].numel() > 2 ** 31
    pool = [t.view(torch.float8_e4m3fn) if eight else t for t in pool]
    sc = [torch.zeros(pages, page, hk, device="cuda") if eight else None for _ in range(2)]
    cache = ab.paged_cache(*pool, k_scale=sc[0], v_scale=sc[1])
    g = torch.Generator().manual_seed(10)
    n = 300
    k, v = (torch.randn(1, hk, n, d, generator=g).to(dt).cuda() for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    def desc(m):
        return ab.sdpa_desc(dtype=ab.ATTN_BF16, b=1, h=hk, h_kv=hk, s_q=m, s_kv=512, d=d, scale=d ** -0.5,
                            mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
    ws = ab.paged_cache_write(desc(n), cache, table, lens, k, v)
    assert ab.attn_query_status(ws) == 0
    back = [torch.empty_like(t) for t in (k, v)]
    ab.paged_cache_read(desc(n), cache, table, lens, *back)
    if not eight:
        assert torch.equal(back[0], k) and torch.equal(back[1], v)
    q = torch.randn(1, hk, new, d, generator=g).to(dt).cuda()
    o = torch.empty_like(q)
    ws = ab.sdpa_paged_fwd(desc(new), cache, table, lens, q, o)
    assert ab.attn_query_status(ws) == 0
    s = q.double() @ back[0].double().transpose(2, 3) * d ** -0.5
    s = s.masked_fill(torch.ones(new, n, dtype=torch.bool, device="cuda").triu(n - new + 1), -float("inf"))
    w = s.softmax(-1)
    want, mag = w @ back[1].double(), w @ back[1].double().abs()
    # weights 2^-8, values 2^-8 (read back, and rounded), scores of e4m3 keys off by the read back's rounding: 2^-8 of |q||k|
    slack = 4 if not eight else 4 + 2 * float((q.double().abs() @ back[0].double().abs().transpose(2, 3)).max()) * d ** -0.5
    assert bool(((o.double() - want).abs() <= 2.0 ** -8 * (want.abs() + slack * mag)).all())
