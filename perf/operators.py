"""The position operators as a user's program calls them: their plain forms in torch, the library's
calls, and the cases over which they are measured.

Two operators in five forms:

* ``qknorm_fwd`` / ``qknorm_bwd``: RMS norm of every query and key head with the rotary position
  embedding in the same pass, and its gradient;
* ``relbias_fwd`` / ``relbias_bwd``: scaled dot-product attention with a learned relative position
  bias by buckets added to the scores (training forward with its log-sum-exp stats; gradients of Q, K,
  V and of the bias table);
* ``relbias_decode``: the same attention for one new token per sequence over a key/value cache.

Tensors are stored [batch, seq, head, dim] (or packed [token, head, dim]).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token for each of 8 sequences of a grouped-query decoder: latency
        dict(name="qknorm-fwd-token", op="qknorm_fwd", dtype="bf16", b=8, s=1, h=32, h_kv=8, d=128, rot=128,
             interleaved=False, max_pos=8192),
        # the attention layer of a GPT-2-sized training step, half of each head rotated in adjacent pairs
        dict(name="qknorm-fwd-gpt", op="qknorm_fwd", dtype="fp16", b=4, s=1024, h=12, h_kv=12, d=64, rot=32,
             interleaved=True, max_pos=2048),
        # a packed varlen batch of a grouped-query model (20442 tokens, an odd count per sequence)
        dict(name="qknorm-fwd-packed", op="qknorm_fwd", dtype="bf16", b=1, s=20442, h=32, h_kv=8, d=128, rot=128,
             interleaved=False, max_pos=4096),
        # gradient of a ragged small layer with head dim 192, the NSA head dim
        dict(name="qknorm-bwd-ragged", op="qknorm_bwd", dtype="fp16", b=3, s=777, h=16, h_kv=1, d=192, rot=64,
             interleaved=False, max_pos=1024),
        # gradient of the packed batch
        dict(name="qknorm-bwd-packed", op="qknorm_bwd", dtype="bf16", b=1, s=20442, h=32, h_kv=8, d=128, rot=128,
             interleaved=False, max_pos=4096),
        # an encoder layer: no mask, both directions have buckets
        dict(name="relbias-fwd-encoder", op="relbias_fwd", dtype="fp16", b=4, h=12, h_kv=12, s_q=1024, s_kv=1024, d=64,
             mask="none", bidirectional=True, buckets=32, max_distance=128),
        # a long causal decoder layer
        dict(name="relbias-fwd-long", op="relbias_fwd", dtype="bf16", b=2, h=32, h_kv=32, s_q=4096, s_kv=4096, d=128,
             mask="causal", bidirectional=False, buckets=32, max_distance=128),
        # gradients of the encoder layer
        dict(name="relbias-bwd-encoder", op="relbias_bwd", dtype="fp16", b=4, h=12, h_kv=12, s_q=1024, s_kv=1024, d=64,
             mask="none", bidirectional=True, buckets=32, max_distance=128),
        # gradients of a grouped-query layer, fewer queries than keys, neither a multiple of a tile, far buckets
        dict(name="relbias-bwd-ragged", op="relbias_bwd", dtype="bf16", b=1, h=32, h_kv=8, s_q=1301, s_kv=2285, d=128,
             mask="causal", bidirectional=False, buckets=64, max_distance=1024),
        # gradients of the long causal layer
        dict(name="relbias-bwd-long", op="relbias_bwd", dtype="bf16", b=2, h=32, h_kv=32, s_q=4096, s_kv=4096, d=128,
             mask="causal", bidirectional=False, buckets=32, max_distance=128),
        # one token of one sequence, 1000 tokens in: latency
        dict(name="relbias-decode-one", op="relbias_decode", dtype="fp16", b=1, h=12, h_kv=12, cap=1024, d=64,
             len_lo=1000, len_hi=1000, bidirectional=False, buckets=32, max_distance=128),
        # a serving batch of 32 sequences between 1 and 8192 tokens long
        dict(name="relbias-decode-batch", op="relbias_decode", dtype="bf16", b=32, h=32, h_kv=8, cap=8192, d=128,
             len_lo=1, len_hi=8192, bidirectional=False, buckets=32, max_distance=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["qknorm_fwd", "qknorm_bwd", "relbias_fwd", "relbias_bwd", "relbias_decode"])
    dtype = rng.choice(["bf16", "fp16"])
    if op.startswith("qknorm"):
        d = rng.choice([64, 128, 192])
        h, h_kv = rng.choice([(12, 12), (16, 1), (32, 8), (32, 32), (5, 5), (24, 3)])
        most = 20442 * 40 * 128 // ((h + h_kv) * d)
        tokens = _log_int(rng, 1, most)
        b = min(rng.choice([1, 1, 2, 3, 8]), tokens)
        s = tokens // b
        return dict(op=op, dtype=dtype, b=b, s=s, h=h, h_kv=h_kv, d=d,
                    rot=rng.choice([r for r in (0, 16, 32, 64, 96, 128, 192) if r <= d]),
                    interleaved=rng.random() < 0.4, max_pos=max(64, s) + rng.randint(0, 512))
    buckets, far = rng.choice([(32, 128), (32, 64), (64, 256), (16, 100), (64, 1024), (128, 1000)])
    d = rng.choice([64, 128])
    h, h_kv = rng.choice([(12, 12), (32, 8), (32, 32), (16, 1), (5, 5), (12, 4)])
    if op == "relbias_decode":
        b = _log_int(rng, 1, 48)
        most = min(32768, 32 * 8192 * 8 * 128 // (b * h_kv * d))
        cap = _log_int(rng, 16, most)
        hi = rng.randint(max(1, cap // 2), cap)
        return dict(op=op, dtype=dtype, b=b, h=h, h_kv=h_kv, cap=cap, d=d, len_lo=rng.randint(1, hi), len_hi=hi,
                    bidirectional=rng.random() < 0.2, buckets=buckets, max_distance=far)
    s_kv = _log_int(rng, 33, 4096)
    s_q = s_kv if rng.random() < 0.5 else max(1, min(4096, _log_int(rng, max(1, s_kv // 4), s_kv * 2)))
    most = 32 * 4096 * 4096 // (h * s_q * s_kv)
    b = max(1, min(_log_int(rng, 1, 16), most))
    return dict(op=op, dtype=dtype, b=b, h=h, h_kv=h_kv, s_q=s_q, s_kv=s_kv, d=d,
                mask=rng.choice(["none", "causal", "causal"]), bidirectional=rng.random() < 0.5, buckets=buckets,
                max_distance=far)


# ------------------------------------------------------------------------------------------ inputs

def _cache_lens(case):
    """The lengths of the cached sequences, spread evenly from len_lo to len_hi."""
    b, lo, hi = case["b"], case["len_lo"], case["len_hi"]
    return [hi if b == 1 else lo + (hi - lo) * n // (b - 1) for n in range(b)]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 42)
    dt = DT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)

    st = dict(case)
    d, h, hk = case["d"], case["h"], case["h_kv"]
    if case["op"].startswith("qknorm"):
        b, s, rot = case["b"], case["s"], case["rot"]
        # projections of a hidden state: another size for each token
        size = torch.exp(torch.randn(b, s, 1, 1, generator=g, device=DEV) * 0.5)
        st["q"] = (normal(b, s, h, d, dtype=torch.float32) * size).to(dt)
        st["k"] = (normal(b, s, hk, d, dtype=torch.float32) * size).to(dt)
        st["wq"] = (1 + 0.2 * normal(d, dtype=torch.float32)).to(dt)
        st["wk"] = (1 + 0.2 * normal(d, dtype=torch.float32)).to(dt)
        st["eps"] = 1e-6
        st["pos"] = torch.randint(0, case["max_pos"], (b, s), generator=g, device=DEV, dtype=torch.int32)
        if rot:
            inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
            ang = torch.arange(case["max_pos"], dtype=torch.float64, device=DEV)[:, None] * inv
            st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        else:
            st["cos"] = st["sin"] = None
        st["out"] = [torch.empty_like(st["q"]), torch.empty_like(st["k"])]
        if case["op"] == "qknorm_bwd":
            st["dyq"], st["dyk"] = normal(b, s, h, d), normal(b, s, hk, d)
            st["out"] += [torch.empty(d, dtype=torch.float32, device=DEV) for _ in range(2)]
        if own:
            import attention_backward_02_gb300 as ab
            st["desc"] = ab.qk_norm_rope_desc(dtype=_code(ab, dt), b=b, s=s, h=h, h_kv=hk, d=d, rotary_dim=rot,
                                              interleaved=case["interleaved"], eps=st["eps"], max_pos=case["max_pos"])
            need = ab.qk_norm_rope_workspace_size(st["desc"])[case["op"] == "qknorm_bwd"]
            st["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        return st
    st["scale"] = 1.0 / math.sqrt(d)
    st["table"] = normal(case["buckets"], h, scale=1.5, dtype=torch.float32)
    if case["op"] == "relbias_decode":
        b, cap = case["b"], case["cap"]
        st["q"], st["k"], st["v"] = normal(b, 1, h, d), normal(b, cap, hk, d), normal(b, cap, hk, d)
        st["lens"] = torch.tensor(_cache_lens(case), dtype=torch.int32, device=DEV)
        st["out"] = [torch.empty_like(st["q"])]
        if own:
            import attention_backward_02_gb300 as ab
            st["bias"] = ab.relbias(st["table"], max_distance=case["max_distance"],
                                    bidirectional=case["bidirectional"])
            st["desc"] = ab.sdpa_desc(dtype=_code(ab, dt), b=b, h=h, h_kv=hk, s_q=1, s_kv=cap, d=d, scale=st["scale"],
                                      mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT)
            st["ws"] = torch.empty(ab.sdpa_relbias_decode_workspace_size(st["desc"], st["bias"]), dtype=torch.uint8,
                                   device=DEV)
        return st
    b, sq, sk = case["b"], case["s_q"], case["s_kv"]
    st["q"], st["k"], st["v"] = normal(b, sq, h, d), normal(b, sk, hk, d), normal(b, sk, hk, d)
    st["out"] = [torch.empty_like(st["q"]), torch.empty(b, h, sq, dtype=torch.float32, device=DEV)]
    if case["op"] == "relbias_bwd":
        st["do"] = normal(b, sq, h, d)
        o, lse = _plain_fwd(st)
        st["o"], st["lse"] = o, lse
        st["out"] = [torch.empty_like(st["q"]), torch.empty_like(st["k"]), torch.empty_like(st["v"]),
                     torch.empty_like(st["table"])]
    if own:
        import attention_backward_02_gb300 as ab
        st["bias"] = ab.relbias(st["table"], max_distance=case["max_distance"], bidirectional=case["bidirectional"])
        st["desc"] = ab.sdpa_desc(dtype=_code(ab, dt), b=b, h=h, h_kv=hk, s_q=sq, s_kv=sk, d=d, scale=st["scale"],
                                  mask=ab.ATTN_CAUSAL_BOTTOM_RIGHT if case["mask"] == "causal" else ab.ATTN_MASK_NONE)
        need = ab.sdpa_relbias_workspace_size(st["desc"], st["bias"])[case["op"] == "relbias_bwd"]
        st["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return st


def _code(ab, dt):
    return ab.ATTN_BF16 if dt is torch.bfloat16 else ab.ATTN_F16


# --------------------------------------------------------------------------------------------- run

def run(state):
    return _OWN[state["op"]](state) if own else _PLAIN[state["op"]](state)


def _bhsd(t):
    return t.permute(0, 2, 1, 3)


def _own_qknorm_fwd(st):
    import attention_backward_02_gb300 as ab
    yq, yk = st["out"]
    ab.qk_norm_rope_fwd(st["desc"], _bhsd(st["q"]), _bhsd(st["k"]), st["wq"], st["wk"], st["cos"], st["sin"],
                        _bhsd(yq), _bhsd(yk), positions=st["pos"], workspace=st["ws"])
    return yq, yk


def _own_qknorm_bwd(st):
    import attention_backward_02_gb300 as ab
    dq, dk, dwq, dwk = st["out"]
    ab.qk_norm_rope_bwd(st["desc"], _bhsd(st["q"]), _bhsd(st["k"]), _bhsd(st["dyq"]), _bhsd(st["dyk"]), st["wq"],
                        st["wk"], st["cos"], st["sin"], _bhsd(dq), _bhsd(dk), dwq, dwk, positions=st["pos"],
                        workspace=st["ws"])
    return dq, dk, dwq, dwk


def _own_relbias_fwd(st):
    import attention_backward_02_gb300 as ab
    o, lse = st["out"]
    ab.sdpa_relbias_fwd_stats(st["desc"], st["bias"], _bhsd(st["q"]), _bhsd(st["k"]), _bhsd(st["v"]), _bhsd(o), lse,
                              workspace=st["ws"])
    return o, lse


def _own_relbias_bwd(st):
    import attention_backward_02_gb300 as ab
    dq, dk, dv, dt = st["out"]
    ab.sdpa_relbias_bwd(st["desc"], st["bias"], _bhsd(st["q"]), _bhsd(st["k"]), _bhsd(st["v"]), _bhsd(st["o"]),
                        _bhsd(st["do"]), st["lse"], _bhsd(dq), _bhsd(dk), _bhsd(dv), dt, workspace=st["ws"])
    return dq, dk, dv, dt


def _own_relbias_decode(st):
    import attention_backward_02_gb300 as ab
    o, = st["out"]
    ab.sdpa_relbias_decode(st["desc"], st["bias"], _bhsd(st["q"]), _bhsd(st["k"]), _bhsd(st["v"]), st["lens"],
                           _bhsd(o), workspace=st["ws"])
    return o


_OWN = dict(qknorm_fwd=_own_qknorm_fwd, qknorm_bwd=_own_qknorm_bwd, relbias_fwd=_own_relbias_fwd,
            relbias_bwd=_own_relbias_bwd, relbias_decode=_own_relbias_decode)


# ------------------------------------------------------------------------------------- plain forms

def _rotate(z, st, sign):
    """z [b, s, h, d] rotated by the angle of its token (sign = -1: back)."""
    rot = st["rot"]
    if rot == 0:
        return z
    pos = st["pos"].long()
    cos, sin = st["cos"][pos].unsqueeze(2), sign * st["sin"][pos].unsqueeze(2)
    if st["interleaved"]:
        a, c = z[..., 0:rot:2], z[..., 1:rot:2]
        r = torch.stack([a * cos - c * sin, c * cos + a * sin], -1).flatten(-2)
    else:
        a, c = z[..., :rot // 2], z[..., rot // 2:rot]
        r = torch.cat([a * cos - c * sin, c * cos + a * sin], -1)
    return torch.cat([r, z[..., rot:]], -1)


def _plain_qknorm_fwd(st):
    outs = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        xf = x.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + st["eps"])
        outs.append(_rotate(xf * r * w.float(), st, 1).to(x.dtype))
    return tuple(outs)


def _plain_qknorm_bwd(st):
    dxs, dws = [], []
    for x, dy, w in ((st["q"], st["dyq"], st["wq"]), (st["k"], st["dyk"], st["wk"])):
        xf = x.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + st["eps"])
        xh = xf * r
        dz = _rotate(dy.float(), st, -1)
        dws.append((dz * xh).flatten(0, -2).sum(0, dtype=torch.float64).float())
        g = dz * w.float()
        dxs.append((r * (g - xh * (g * xh).mean(-1, keepdim=True))).to(x.dtype))
    return (*dxs, *dws)


def _bucket(delta, st):
    """Bucket of a key that lies `delta` positions after its query (int64 tensor)."""
    n = st["buckets"]
    base = torch.zeros_like(delta)
    if st["bidirectional"]:
        n //= 2
        base = (delta > 0).long() * n
        dist = delta.abs()
    else:
        dist = (-delta).clamp(min=0)
    exact = n // 2
    # in 64 bits, and a distance that lies on a border belongs to the bucket above it
    steps = torch.log(dist.clamp(min=1).double() / exact) / math.log(st["max_distance"] / exact) * (n - exact)
    far = (exact + torch.floor(steps + 1e-9).long()).clamp(max=n - 1)
    return base + torch.where(dist < exact, dist, far)


def _geometry(st):
    """(bucket [s_q, s_kv], visible [s_q, s_kv] or None)."""
    sq, sk = st["s_q"], st["s_kv"]
    shift = sk - sq if st["mask"] == "causal" else 0
    delta = torch.arange(sk, device=DEV)[None, :] - (torch.arange(sq, device=DEV)[:, None] + shift)
    return _bucket(delta, st), (delta <= 0) if st["mask"] == "causal" else None


def _scores(st, n, bias, visible):
    """Scores [h, s_q, s_kv] of sequence n, and its keys and values repeated for the query heads."""
    grp = st["h"] // st["h_kv"]
    q = st["q"][n].float().transpose(0, 1)
    k = st["k"][n].float().transpose(0, 1).repeat_interleave(grp, 0)
    v = st["v"][n].float().transpose(0, 1).repeat_interleave(grp, 0)
    s = (q @ k.transpose(1, 2)).mul_(st["scale"]).add_(bias)
    if visible is not None:
        s.masked_fill_(~visible, -math.inf)
    return q, k, v, s


def _plain_fwd(st):
    bucket, visible = _geometry(st)
    bias = st["table"].t()[:, bucket]
    os, lses = [], []
    for n in range(st["b"]):
        _, _, v, s = _scores(st, n, bias, visible)
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = s.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        o = torch.where(l > 0, (p @ v) / l, torch.zeros_like(v[:, :1]))
        os.append(o.transpose(0, 1).to(st["q"].dtype))
        lses.append(torch.where(l > 0, m + torch.log(l), torch.full_like(l, math.inf)).squeeze(-1))
        del s, p
    return torch.stack(os), torch.stack(lses)


def _plain_bwd(st):
    bucket, visible = _geometry(st)
    bias = st["table"].t()[:, bucket]
    sq, sk, h, hk, d = st["s_q"], st["s_kv"], st["h"], st["h_kv"], st["d"]
    grads = [[], [], []]
    by_delta = torch.zeros(h, sq + sk - 1, dtype=torch.float64, device=DEV)
    for n in range(st["b"]):
        q, k, v, s = _scores(st, n, bias, visible)
        do, o = st["do"][n].float().transpose(0, 1), st["o"][n].float().transpose(0, 1)
        p = s.sub_(st["lse"][n].unsqueeze(-1)).exp_()
        ds = (do @ v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
        dv = p.transpose(1, 2) @ do
        del s, p
        dq = (ds @ k) * st["scale"]
        dk = (ds.transpose(1, 2) @ q) * st["scale"]
        # sums along the diagonals: rows in reverse, each shifted by one more column
        skew = torch.zeros(h, sq, sk + sq, device=DEV)
        skew[:, :, :sk] = ds.flip(1)
        del ds
        skew = skew.reshape(h, -1)[:, :sq * (sk + sq - 1)].reshape(h, sq, sk + sq - 1)
        by_delta += skew.sum(1, dtype=torch.float64)
        del skew
        grads[0].append(dq.transpose(0, 1).to(st["q"].dtype))
        for i, x in ((1, dk), (2, dv)):  # the gradient of a shared head is the sum over its query heads
            grads[i].append(x.reshape(hk, h // hk, sk, d).sum(1).transpose(0, 1).to(st["k"].dtype))
    shift = sk - sq if st["mask"] == "causal" else 0
    delta = torch.arange(sk + sq - 1, device=DEV) - (sq - 1) - shift
    dt = torch.zeros(st["buckets"], h, dtype=torch.float64, device=DEV)
    dt.index_add_(0, _bucket(delta, st), by_delta.t().contiguous())
    return (*(torch.stack(x) for x in grads), dt.float())


def _plain_decode(st):
    grp = st["h"] // st["h_kv"]
    j = torch.arange(st["cap"], device=DEV)
    lens = st["lens"].long()
    delta = j[None, :] - (lens[:, None] - 1)  # the new token is the last of its sequence
    bias = st["table"][_bucket(delta, st)].permute(0, 2, 1)  # [b, h, cap]
    b, hk, d = st["b"], st["h_kv"], st["d"]
    q = st["q"].float().reshape(b, hk, grp, d)
    k, v = st["k"].float().permute(0, 2, 1, 3), st["v"].float().permute(0, 2, 1, 3)
    s = (q @ k.transpose(2, 3)) * st["scale"] + bias.reshape(b, hk, grp, -1)
    s = s.masked_fill((delta > 0)[:, None, None, :], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = (p @ v) / p.sum(-1, keepdim=True)
    return o.reshape(b, 1, st["h"], d).to(st["q"].dtype)


_PLAIN = dict(qknorm_fwd=_plain_qknorm_fwd, qknorm_bwd=_plain_qknorm_bwd, relbias_fwd=_plain_fwd,
              relbias_bwd=_plain_bwd, relbias_decode=_plain_decode)


# -------------------------------------------------------------------------------------------- work

def work(case):
    h, hk, d = case["h"], case["h_kv"], case["d"]
    if case["op"].startswith("qknorm"):
        t = case["b"] * case["s"]
        n = t * (h + hk) * d
        side = t * 4 + min(t, case["max_pos"]) * case["rot"] * 4 + 2 * d * 2  # positions, cos and sin rows, weights
        if case["op"] == "qknorm_fwd":
            return dict(bytes=2 * n * 2 + side, flops=7 * n)
        return dict(bytes=3 * n * 2 + side + 2 * d * 4, flops=16 * n)
    if case["op"] == "relbias_decode":
        keys = sum(_cache_lens(case))
        return dict(bytes=keys * hk * d * 4 + 2 * case["b"] * h * d * 2 + case["b"] * 4 + case["buckets"] * h * 4,
                    flops=4 * keys * h * d)
    b, sq, sk = case["b"], case["s_q"], case["s_kv"]
    if case["mask"] == "causal":
        pairs = sum(max(0, min(sk, i + sk - sq + 1)) for i in range(sq))
    else:
        pairs = sq * sk
    nq, nk = b * sq * h * d, b * sk * hk * d
    table = case["buckets"] * h * 4
    if case["op"] == "relbias_fwd":
        return dict(bytes=(2 * nq + 2 * nk) * 2 + b * h * sq * 4 + table, flops=4 * b * h * pairs * d)
    return dict(bytes=(4 * nq + 4 * nk) * 2 + b * h * sq * 4 + 2 * table, flops=10 * b * h * pairs * d)


# ------------------------------------------------------------------------------------------- exact

def _exact_buckets(case, largest):
    """The buckets of the distances 0 .. largest, by integer arithmetic: distance x reaches step m past
    the exact buckets when (x / e)^(n - e) >= (max_distance / e)^m."""
    n = case["buckets"] // 2 if case["bidirectional"] else case["buckets"]
    e, far, out, m = n // 2, case["max_distance"], [], 0
    for x in range(largest + 1):
        if x < e:
            out.append(x)
            continue
        while e + m < n - 1 and x ** (n - e) * e ** (m + 1) >= far ** (m + 1) * e ** (n - e):
            m += 1
        out.append(e + m)
    return out


def _exact_rows(case, sq, sk, shift):
    """Bucket of every (query, key), as int64 [sq, sk]."""
    known = torch.tensor(_exact_buckets(case, case["max_distance"]), device=DEV)
    i = torch.arange(sq, device=DEV) + shift
    ahead = torch.arange(sk, device=DEV)[None, :] - i[:, None]
    if case["bidirectional"]:
        return known[ahead.abs().clamp(max=case["max_distance"])] + torch.where(ahead > 0, case["buckets"] // 2, 0)
    return known[(-ahead).clamp(min=0, max=case["max_distance"])]


def exact(case, seed):
    st = prepare(case, seed)
    f = torch.float64
    if case["op"].startswith("qknorm"):
        if case["rot"]:
            c, s = st["cos"].to(f)[st["pos"].long()], st["sin"].to(f)[st["pos"].long()]
            # as complex numbers: a + ib times cos + i sin
            turn = torch.complex(c, s).unsqueeze(2)
        half = case["rot"] // 2

        def spin(x, w):
            if not half:
                return x
            head = x[..., :2 * half].unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
            a, b = head.unbind(-1 if case["interleaved"] else -2)
            y = torch.complex(a.contiguous(), b.contiguous()) * w
            y = torch.stack([y.real, y.imag], -1 if case["interleaved"] else -2).flatten(-2)
            return torch.cat([y, x[..., 2 * half:]], -1)

        outs, sums = [], []
        for x, w, dy in ((st["q"], st["wq"], st.get("dyq")), (st["k"], st["wk"], st.get("dyk"))):
            x, w = x.to(f), w.to(f)
            rms = ((x ** 2).sum(-1, keepdim=True) / case["d"] + st["eps"]).sqrt()
            if dy is None:
                outs.append(spin(x / rms * w, turn if half else None))
            else:
                up = spin(dy.to(f), turn.conj() if half else None)
                sums.append((up * x / rms).sum((0, 1, 2)))
                up = up * w
                outs.append(up / rms - x * (up * x).sum(-1, keepdim=True) / (case["d"] * rms ** 3))
        return (*outs, *sums)
    h, hk, d = case["h"], case["h_kv"], case["d"]
    grp = h // hk
    table = st["table"].to(f)
    if case["op"] == "relbias_decode":
        out = torch.empty(case["b"], 1, h, d, dtype=f, device=DEV)
        for n, length in enumerate(_cache_lens(case)):
            rows = _exact_rows(case, 1, length, length - 1)[0]
            for g in range(hk):
                q = st["q"][n, 0, g * grp:(g + 1) * grp].to(f)
                w = (q @ st["k"][n, :length, g].to(f).t() * st["scale"] + table[rows, g * grp:(g + 1) * grp].t()).softmax(-1)
                out[n, 0, g * grp:(g + 1) * grp] = w @ st["v"][n, :length, g].to(f)
        return out
    b, sq, sk = case["b"], case["s_q"], case["s_kv"]
    causal = case["mask"] == "causal"
    rows = _exact_rows(case, sq, sk, sk - sq if causal else 0)
    hidden = None
    if causal:
        hidden = torch.ones(sq, sk, dtype=torch.bool, device=DEV).triu(sk - sq + 1)
    if case["op"] == "relbias_fwd":
        o = torch.zeros(b, sq, h, d, dtype=f, device=DEV)
        lse = torch.empty(b, h, sq, dtype=f, device=DEV)
        for n in range(b):
            for x in range(h):
                s = st["q"][n, :, x].to(f) @ st["k"][n, :, x // grp].to(f).t() * st["scale"] + table[:, x][rows]
                if causal:
                    s = s.masked_fill(hidden, -math.inf)
                z = s.logsumexp(-1)
                dead = z == -math.inf
                z[dead] = math.inf
                lse[n, x] = z
                o[n, :, x] = torch.exp(s - z[:, None]) @ st["v"][n, :, x // grp].to(f)
        return o, lse
    dq = torch.empty(b, sq, h, d, dtype=f, device=DEV)
    dk, dv = (torch.zeros(b, sk, hk, d, dtype=f, device=DEV) for _ in range(2))
    dt = torch.zeros(case["buckets"], h, dtype=f, device=DEV)
    used = rows.unique().tolist()
    for n in range(b):
        for x in range(h):
            y = x // grp
            q, k, v = st["q"][n, :, x].to(f), st["k"][n, :, y].to(f), st["v"][n, :, y].to(f)
            do, o = st["do"][n, :, x].to(f), st["o"][n, :, x].to(f)
            p = torch.exp(q @ k.t() * st["scale"] + table[:, x][rows] - st["lse"][n, x].to(f)[:, None])
            if causal:
                p = p.masked_fill(hidden, 0.0)
            ds = p * (do @ v.t() - (do * o).sum(-1, keepdim=True))
            dv[n, :, y] += p.t() @ do
            dk[n, :, y] += ds.t() @ q * st["scale"]
            dq[n, :, x] = ds @ k * st["scale"]
            for u in used:
                dt[u, x] += (ds * (rows == u)).sum()
    return dq, dk, dv, dt
