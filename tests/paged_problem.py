"""A paged cache with its sequences for the tests: pages in a random order, NaN wherever nothing may look, and the error
bounds of the attention.

Bounds (h: half a step of the 16-bit type, u = 2^-23).  The exponent of a key's weight is off by at most
e = (d + 8) u (sum |q k| scale + |s| + |largest s|), the exponential by 2^-21; the weights are rounded to 16 bits
(h); values of an e4m3 cache may be half-precision numbers times their scale, both rounded (2^-11 each, together g); a
half-precision weight is also off by 2^-25 of the largest, and such a value by 2^-25 of the largest value scale
rounded up to a power of two, once for the scale's rounding and once for the product's:
    |O err| <= h |O| + sum_j (h + g + 2 max e + 2^-20 + n u) P_j |v_j| + 2^-25 a,
    a = sum_j |v_j|, e4m3: 3 * 2 (largest scale) sum_j max(|code_j|, 1)
    |LSE err| <= max e + 2^-20 + n u + 4 u |LSE|."""
import numpy as np

from oracle import paged as P

U = 2.0 ** -23
HALF = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


class Problem:
    def __init__(self, dtype, cache, lens, new, h, hk, d, page=16, layout="nhd", packed=True, causal=True, extra_rows=0,
                 seed=0, cap=None, scales_by_head=False, size=1.0):
        import torch
        import attention_backward_02_gb300 as ab
        self.ab, self.torch, self.dtype = ab, torch, dtype
        self.dt = dt = torch.float16 if dtype == "float16" else torch.bfloat16
        self.lens, self.new = list(lens), list(new)
        self.h, self.hk, self.d, self.page, self.packed, self.causal, self.eight = h, hk, d, page, packed, causal, cache == "e4m3"
        self.scale = d ** -0.5
        b = len(self.lens)
        self.cap = cap if cap is not None else max(1, max(self.lens))
        g = torch.Generator().manual_seed(seed)
        used = [-(-max(min(n, self.cap), 0) // page) for n in self.lens]
        pages = sum(used) + 2
        order = torch.randperm(pages, generator=g)
        self.table = torch.full((b, -(-self.cap // page) + 1), -7, dtype=torch.int32)  # (a column nobody needs)
        at = 0
        for n, c in enumerate(used):
            self.table[n, :c] = order[at:at + c].int()
            at += c
        self.rows_of = [[int(self.table[n, i // page]) * page + i % page for i in range(max(min(c, self.cap), 0))]
                        for n, c in enumerate(self.lens)]
        # the cache's contents, [slot, head, d], NaN where no sequence has a token
        self.pool, self.scales = [], []
        live = torch.zeros(pages * page, dtype=torch.bool)
        for r in self.rows_of:
            live[r] = True
        for _ in range(2):
            x = torch.randn(pages * page, hk, d, generator=g) * torch.exp(0.5 * torch.randn(pages * page, hk, 1, generator=g)) * size
            x = x.to(dt)
            if self.eight:
                code, sc = P.quantise(x.float().numpy())
                code[~live.numpy()] = 0x7f
                sc[~live.numpy()] = np.nan
                x, sc = torch.from_numpy(code).view(pages, page, hk, d), torch.from_numpy(sc).view(pages, page, hk)
            else:
                x[~live] = float("nan")
                x, sc = x.view(pages, page, hk, d), None
            self.pool.append(x)
            self.scales.append(sc)
        lay = self._by_head if layout == "hnd" else self._side_by_side if layout == "kv" else (lambda a, b: [a.cuda(), b.cuda()])
        self.cpool = lay(*self.pool)
        if self.eight:
            self.cpool = [t.view(torch.float8_e4m3fn) for t in self.cpool]
            self.cscales = (self._by_head if scales_by_head else (lambda a, b: [a.cuda(), b.cuda()]))(*self.scales)
        else:
            self.cscales = [None, None]
        self.cache = ab.paged_cache(*self.cpool, k_scale=self.cscales[0], v_scale=self.cscales[1])
        self.dtable, self.dlens = self.table.cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.starts = np.concatenate([[0], np.cumsum(self.new)]).tolist()
        self.rows = self.starts[-1] + extra_rows
        self.cu = torch.tensor(self.starts, dtype=torch.int32, device="cuda") if packed else None
        assert packed or len(set(self.new)) <= 1
        self.desc = self._desc()
        self.q = (torch.randn(self.rows, h, d, generator=g)).to(dt)

    @staticmethod
    def _by_head(a, b):
        return [t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in (a, b)]

    @staticmethod
    def _side_by_side(a, b):
        import torch
        both = torch.stack([a, b], 1).contiguous().cuda()
        return [both[:, 0], both[:, 1]]

    def _desc(self):
        ab = self.ab
        return ab.sdpa_desc(dtype=ab.ATTN_F16 if self.dtype == "float16" else ab.ATTN_BF16, b=len(self.lens), h=self.h,
                            h_kv=self.hk, s_q=max(self.new, default=0), s_kv=self.cap, d=self.d, scale=self.d ** -0.5,
                            mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT if self.causal else ab.ATTN_MASK_NONE)

    def dense(self, t):
        """Packed rows [T, heads, d] as the calls take them."""
        t = t.cuda()
        return t if self.packed else t.view(len(self.new), -1, *t.shape[1:]).permute(0, 2, 1, 3)

    def packed_of(self, t):
        return t if self.packed else t.permute(0, 2, 1, 3).reshape(self.rows, *t.shape[1:2], t.shape[3])

    def attend(self, flags=0, lse=True, q=None, o=None, **kw):
        torch = self.torch
        q = self.dense(self.q) if q is None else q
        o = torch.full_like(q, float("nan")) if o is None else o
        stats = torch.full((self.h, self.rows) if self.packed else (len(self.new), self.h, self.new[0]), float("nan"),
                           device="cuda") if lse else None
        ws = self.ab.sdpa_paged_fwd(self.desc, self.cache, self.dtable, self.dlens, q, o, lse=stats, cu_new=self.cu, **kw)
        if flags is not None:
            assert self.ab.attn_query_status(ws, kw.get("stream")) == flags
        return o, stats

    def contents(self, n):
        """k, v [len, hk, d] of sequence n in 64 bits, and the sums' |code| rows with the largest scale."""
        out = []
        for x, sc in zip(self.pool, self.scales):
            r = self.rows_of[n]
            x = x.reshape(-1, self.hk, self.d)[r]
            if self.eight:
                sc = sc.reshape(-1, self.hk)[r]
                out.append(P.E4M3[x.numpy()] * sc.double().numpy()[..., None])
            else:
                out.append(x.double().numpy())
        return out

    def check(self, o, lse=None, only=None):
        o = self.packed_of(o).double().cpu().numpy()
        if lse is not None:
            lse = lse.double().cpu().numpy() if self.packed else lse.permute(1, 0, 2).reshape(self.h, -1).double().cpu().numpy()
        grp = self.h // self.hk
        for n, m in enumerate(self.new):
            if only is not None and n not in only:
                continue
            k, v = self.contents(n)
            if self.eight:
                r = self.rows_of[n]
                code = np.abs(P.E4M3[self.pool[1].reshape(-1, self.hk, self.d)[r].numpy()])
                code = np.where(code > 0, np.maximum(code, 1), 0)
                tiny = 6 * (self.scales[1].reshape(-1, self.hk)[r].double().numpy().max(0, initial=0)[:, None] * code.sum(0))
            else:
                tiny = np.abs(v).sum(0)
            tiny = np.repeat(tiny, grp, 0) * 2.0 ** -25
            av = np.repeat(np.abs(v), grp, 1)
            hf = HALF[self.dtype]
            for i0 in range(0, m, 64):  # rows in pieces: the bounds' arrays are large
                rows = slice(self.starts[n] + i0, self.starts[n] + min(m, i0 + 64))
                upto = len(k) - m + min(m, i0 + 64) if self.causal else len(k)
                upto = max(upto, 0)
                q = self.q[rows].double().numpy()
                if not self.causal:
                    ref, rl, p, mag, s = P.attention(q, k, v, self.scale, False)
                else:
                    ref, rl, p, mag, s = P.attention(q, k[:upto], v[:upto], self.scale, True)
                e = (self.d + 8) * U * (mag + np.abs(s) + np.abs(s).max(-1, initial=0, keepdims=True))
                e = e.max(-1, initial=0)
                w = hf + (2.0 ** -10 if self.eight else 0) + 2 * e + 2.0 ** -20 + len(k) * U
                bound = hf * np.abs(ref) + w[..., None] * np.einsum("mhn,nhd->mhd", p, av[:upto] if self.causal else av) + tiny + 2.0 ** -24
                err = np.abs(o[rows] - ref)
                assert np.all(err <= bound), (n, i0, float(np.nanmax(err)), float(np.nanmax(err - bound)), int(np.isnan(err).sum()))
                empty = np.isinf(rl)
                assert np.all(o[rows][empty] == 0)
                if lse is not None:
                    got = lse[:, rows].T
                    assert np.array_equal(np.isposinf(got), empty)
                    err = np.abs(np.where(empty, 0, got) - np.where(empty, 0, rl))
                    lim = e + 2.0 ** -20 + len(k) * U + 4 * U * np.abs(np.where(empty, 0, rl))
                    assert np.all(err <= lim), (n, i0, float(err.max()), float((err - lim).max()))
