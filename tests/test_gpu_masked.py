"""Dense attention with capped scores, a distance bias, document and prefix
masks (vsa_masked_attn_fwd, vsa_masked_attn_bwd) against the formula in 64 bits.

Tolerances, u = 2^-24, e = 2^-8 the largest rounding of a value to bf16 (half a
step: a value's rounding is at most e / 2 of its binade's top, 2^-8 relative).
  score  : a sum of 128 exact products in 32 bits, at most 128 u sum|q k| scale;
           the cap's tanh is formed as 1 - 2 / (1 + 2^y) with y, 2^y and the
           quotient within 2^-21 relative each: 8 u cap (1 + |s / cap|) more; the
           bias and the steps to log2 units round a few times: 8 u |score| more.
           ds <= 128 u smax + 16 u (cap + |s|max), smax = scale sum|q k|.
  P      : 2^(x - m): ds, 2 u |x - m| from the subtraction and 4 u from the
           exponential, relative: dp = ds + 64 u for every P that is not
           negligible (|x - m| < 24).
  lse    : ds + 64 u, and log2 and two products: + 4 u |lse| + 8 u.
  out    : P enters the second product rounded to bf16, 2^-8 relative, its sum is
           of the unrounded P; with p the probabilities: |out| error <= (2^-8 + 2 dp)
           sum p|v| + (128 + Sk / 128) u sum p|v| + the output's rounding 2^-8 |out|.
The gradients (the same P, in the same way):
  D      : sum dO O of the rounded output: 2^-8 sum|dO O| + 128 u sum|dO O|, and what
           out itself is off by, sum|dO| dout.
  dS     = P (dP - D): dP within 128 u sum|dO v|; dS enters its products as bf16.
           d(dS) <= |dS| (2^-8 + 2 dp) + P (128 u sum|dO v| + dD), and with a cap
           times 1 - t^2, within 16 u of it.
  dQ, dK : scale (sum d(dS) |k|, sum d(dS) |q|), sums in 32 bits, and rounding 2^-8.
  dV     : (2^-8 + 2 dp) sum P|dO| and rounding 2^-8.
  tiny   : an exponential below 2^-126 is 0, an absolute error below 2^-126 in P; dS
           multiplies it by at most sum|dO v| + |D| < 2 * 128 * 8 * 8 < 2^15, the
           products sum at most 2^11 of them times |k|, |q|, |dO| < 2^3 and the
           scale < 1: 2^-126 + 15 + 11 + 3 < 2^-96 everywhere.
All of these are evaluated with the reference's values below.
"""

import math

import pytest

from block_sparse_video_geometry_b200 import vsa

pytestmark = pytest.mark.gpu
U, E, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -96


def visible(B, Sq, Sk, causal=False, prefix=None, doc_q=None, doc_k=None):
    import torch
    i = torch.arange(Sq, device="cuda")[:, None] + Sk - Sq
    j = torch.arange(Sk, device="cuda")[None]
    see = torch.ones((B, Sq, Sk), dtype=torch.bool, device="cuda")
    if causal:
        p = prefix.view(-1, 1, 1) if prefix is not None else torch.zeros((B, 1, 1), device="cuda")
        see &= (j <= i)[None] | (j[None] < p)
    if doc_q is not None:
        see &= (doc_q[:, :, None] == doc_k[:, None, :]) & (doc_q[:, :, None] >= 0)
    return see


class Reference:
    """Values and bounds in float64, one (batch entry, query head) at a time."""

    def __init__(self, q, k, v, see, cap=0.0, slopes=None, scale=None, dout=None):
        import torch
        B, Sq, Hq, D = q.shape
        Sk, Hk = k.shape[1], k.shape[2]
        g = Hq // Hk
        scale = scale or 1 / math.sqrt(D)
        z = lambda *s: torch.zeros(s, dtype=torch.float64, device="cuda")  # noqa: E731
        self.out, self.t_out = z(B, Sq, Hq, D), z(B, Sq, Hq, D)
        self.lse, self.t_lse = z(B, Hq, Sq), z(B, Hq, Sq)
        if dout is not None:
            self.dq, self.t_dq = z(B, Sq, Hq, D), z(B, Sq, Hq, D)
            self.dk, self.t_dk, self.dv, self.t_dv = (z(B, Sk, Hk, D) for _ in range(4))
        i = torch.arange(Sq, device="cuda")[:, None] + Sk - Sq
        dist = (i - torch.arange(Sk, device="cuda")[None]).abs().double()
        for b in range(B):
            for h in range(Hq):
                Q, K, V = q[b, :, h].double(), k[b, :, h // g].double(), v[b, :, h // g].double()
                # hidden rows may hold anything: they take no part
                rows, cols = see[b].any(1), see[b].any(0)
                Q, K, V = (torch.where(m[:, None], x, torch.zeros_like(x)) for x, m in ((Q, rows), (K, cols), (V, cols)))
                s = scale * Q @ K.t()
                smax = scale * Q.abs() @ K.abs().t()
                slope = torch.ones_like(s)
                ds = 128 * U * smax
                if cap:
                    t = torch.tanh(s / cap)
                    slope = 1 - t * t
                    ds = ds + 16 * U * (cap + s.abs())
                    s = cap * t
                if slopes is not None:
                    s = s - slopes[h].double() * dist
                    ds = ds + 16 * U * s.abs()
                ds = (ds + 8 * U * s.abs()).masked_fill(~see[b], 0.0).amax(1, keepdim=True)
                s = s.masked_fill(~see[b], -math.inf)
                lse = torch.logsumexp(s, 1) if Sk else s.new_full((Sq,), -math.inf)
                P = torch.exp(s - lse.clamp_min(-1e300)[:, None])
                dp = ds + 64 * U
                o = P @ V
                self.out[b, :, h], self.lse[b, h] = o, lse
                to = (E + 2 * dp + (128 + Sk / 128) * U) * (P @ V.abs())
                self.t_out[b, :, h] = to + E * (o.abs() + to)
                self.t_lse[b, h] = (ds[:, 0] if Sk else 0) + 72 * U + 4 * U * lse.nan_to_num(neginf=0.0).abs()
                if dout is None:
                    continue
                dO = torch.where(rows[:, None], dout[b, :, h].double(), torch.zeros_like(Q))
                dP, adP = dO @ V.t(), dO.abs() @ V.abs().t()
                delta = (dO * o).sum(1, keepdim=True)
                dD = (128 * U * (dO * o).abs().sum(1, keepdim=True)
                      + (dO.abs() * self.t_out[b, :, h]).sum(1, keepdim=True))
                dS = P * (dP - delta) * slope
                tS = dS.abs() * (E + 2 * dp) + P * (128 * U * adP + dD) * slope \
                    + (16 * U * P * (dP - delta).abs() if cap else 0.0)
                tq = scale * (tS @ K.abs() + (128 + Sk / 128) * U * dS.abs() @ K.abs())
                tk = scale * (tS.t() @ Q.abs() + (128 + Sq / 128) * U * dS.abs().t() @ Q.abs())
                tv = ((E + 2 * dp + (128 + Sq / 128) * U) * P).t() @ dO.abs()
                self.dq[b, :, h] = scale * dS @ K
                self.t_dq[b, :, h] = tq
                self.dk[b, :, h // g] += scale * dS.t() @ Q
                self.t_dk[b, :, h // g] += tk
                self.dv[b, :, h // g] += P.t() @ dO
                self.t_dv[b, :, h // g] += tv
        if dout is not None:
            for n in ("dq", "dk", "dv"):
                x, t = getattr(self, n), getattr(self, "t_" + n)
                setattr(self, "t_" + n, t + E * (x.abs() + t))


def within(got, want, tol, what):
    import torch
    fine = torch.isfinite(want)
    assert torch.equal(got.double()[~fine], want[~fine]), what + ": infinities"
    err = (got.double() - want).abs()[fine]
    assert not torch.isnan(err).any(), what + ": NaN"
    worst = (err - tol[fine] - TINY).max().item() if err.numel() else 0.0
    assert worst <= 0, "%s: beyond its bound by %.3g (error %.3g)" % (what, worst, err.max().item())


def tensors(B, Sq, Sk, Hq, Hk, seed, size=1.3):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda S, H: (size * torch.randn((B, S, H, 128), generator=g, device="cuda")).bfloat16()  # noqa: E731
    return n(Sq, Hq), n(Sk, Hk), n(Sk, Hk), n(Sq, Hq)


def documents(B, S, lengths, seed=0):
    """Ids of consecutive documents, -1 behind the last; batch entries rotated."""
    import torch
    ids = torch.full((B, S), -1, dtype=torch.int32, device="cuda")
    at = 0
    for d, n in enumerate(lengths):
        ids[:, at:at + n] = d
        at += n
    for b in range(1, B):
        ids[b] = ids[b].roll(37 * b)
    return ids.contiguous()


def slopes_of(H):
    import torch
    return (2.0 ** (-2.0 - 6.0 * torch.arange(H, device="cuda") / H)).float()


def run(q, k, v, causal=False, cap=0.0, scale=0.0, dout=None, stream=None, **terms):
    """Outputs of the forward (and backward) pass with fresh workspaces."""
    import torch
    B, Sq, Hq, _ = q.shape
    Sk, Hk = k.shape[1], k.shape[2]
    attn = vsa.MaskedAttention(vsa.make_mask(causal=causal, softcap=cap, scale=scale), B, Sq, Sk, Hq, Hk)
    out = torch.full((B, Sq, Hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq, Sq), float("nan"), device="cuda")
    attn.forward(q, k, v, out, lse, stream=stream, **terms)
    for ws in attn.ws_fwd.values():
        assert vsa.masked_attn_status(ws, stream) == vsa.OK
    if dout is None:
        return out, lse
    grads = [torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for x in (q, k, v)]
    attn.backward(q, k, v, out, lse, dout, *grads, stream=stream, **terms)
    for ws in attn.ws_bwd.values():
        assert vsa.masked_attn_status(ws, stream) == vsa.OK
    return (out, lse, *grads)


CASES = [
    # B, Sq, Sk, Hq, Hk, causal, prefix, cap, bias, documents
    (1, 128, 128, 1, 1, False, None, 0.0, False, None),
    (1, 1, 1, 1, 1, False, None, 0.0, False, None),
    (2, 1, 300, 4, 2, True, None, 0.0, False, None),            # packed heads, one query, split keys
    (1, 5, 1500, 6, 2, True, None, 25.0, True, None),
    (1, 256, 128, 2, 2, False, None, 0.0, False, None),
    (1, 257, 129, 2, 1, False, None, 0.0, False, None),
    (2, 300, 517, 3, 1, True, (1, 400), 0.0, False, None),
    (1, 700, 700, 2, 2, True, None, 0.0, True, None),
    (1, 640, 640, 2, 2, False, None, 15.0, False, None),
    (2, 520, 520, 4, 2, False, None, 0.0, False, (100, 1, 130, 200)),
    (2, 520, 520, 2, 2, True, None, 20.0, True, (256, 128, 130)),
    (1, 300, 100, 2, 1, True, None, 0.0, False, None),          # the first 200 queries see nothing
    (1, 40, 400, 4, 4, True, (-5,), 0.0, False, None),
    (1, 40, 400, 2, 1, True, (10 ** 6,), 0.0, False, None),      # a prefix past the end
    (1, 1300, 1300, 1, 1, False, None, 0.0, False, (1, 2, 3, 500)),
]


def terms_of(case):
    import torch
    B, Sq, Sk, Hq, Hk, causal, prefix, cap, bias, docs = case
    t = {}
    if prefix is not None:
        t["prefix"] = torch.tensor([prefix[b % len(prefix)] for b in range(B)], dtype=torch.int32, device="cuda")
    if bias:
        t["slopes"] = slopes_of(Hq)
    if docs:
        ids = documents(B, Sk, docs)
        t.update(doc_q=ids[:, Sk - Sq:], doc_k=ids)
    return t


def reference(case, q, k, v, terms, dout=None):
    B, Sq, Sk, Hq, Hk, causal, prefix, cap, bias, docs = case
    see = visible(B, Sq, Sk, causal, terms.get("prefix"), terms.get("doc_q"), terms.get("doc_k"))
    return Reference(q, k, v, see, cap, terms.get("slopes"), dout=dout)


def ident(c):
    return "%dx%dx%d-%d-%d-%s%s%s%s%s" % (c[0], c[1], c[2], c[3], c[4], "c" if c[5] else "f", "p" if c[6] else "",
                                          "t" if c[7] else "", "b" if c[8] else "", "d" if c[9] else "")


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_forward_matches_the_formula(cuda_ok, case):
    q, k, v, _ = tensors(*case[:5], seed=1)
    terms = terms_of(case)
    out, lse = run(q, k, v, causal=case[5], cap=case[7], **terms)
    ref = reference(case, q, k, v, terms)
    within(lse, ref.lse, ref.t_lse, "lse")
    within(out, ref.out, ref.t_out, "out")


@pytest.mark.parametrize("case", CASES, ids=ident)
def test_gradients_match_the_formula(cuda_ok, case):
    q, k, v, dout = tensors(*case[:5], seed=2)
    terms = terms_of(case)
    out, lse, dq, dk, dv = run(q, k, v, causal=case[5], cap=case[7], dout=dout, **terms)
    ref = reference(case, q, k, v, terms, dout)
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(got, getattr(ref, name), getattr(ref, "t_" + name), name)


def with_padding(case=(2, 300, 300, 4, 2, True, None, 0.0, False, (70, 1, 129, 60))):
    """Documents with padding behind them, and the rows that hold padding."""
    q, k, v, dout = tensors(*case[:5], seed=3)
    terms = terms_of(case)
    return case, [q, k, v, dout], terms, terms["doc_k"] < 0


def test_infinities_and_nan_in_masked_places_change_nothing(cuda_ok):
    """Padding rows of q, k, v and dout that hold infinities and NaN: the same bits as with zeros there, and zero
    outputs and gradients in the padding rows themselves."""
    import torch
    case, clean, terms, pad = with_padding()
    for t in clean:
        t[pad] = 0
    want = run(*clean[:3], causal=True, dout=clean[3], **terms)
    dirty = [t.clone() for t in clean]
    for n, t in enumerate(dirty):
        rows = pad.nonzero()
        for i, (b, s) in enumerate(rows.tolist()):
            t[b, s, :, (i + n) % 128] = (float("inf"), float("-inf"), float("nan"))[i % 3]
            t[b, s, :, (i * 7 + 3) % 128] = -3e38
    got = run(*dirty[:3], causal=True, dout=dirty[3], **terms)
    for name, a, b in zip(("out", "lse", "dq", "dk", "dv"), got, want):
        assert torch.equal(a, b), name
    for g in (got[0], got[2], got[3], got[4]):
        assert not g[pad].float().any()
    assert torch.equal(got[1].transpose(1, 2)[pad], torch.full_like(got[1].transpose(1, 2)[pad], -math.inf))


@pytest.mark.parametrize("Sq", [1, 40, 333])
def test_later_keys_of_a_causal_mask_may_hold_anything(cuda_ok, Sq):
    """Keys behind the last query's position do not exist for the call; a key that only later queries see reaches
    no earlier one, in the forward and the backward pass."""
    import torch
    B, Sk, H = 1, 500, 2
    q, k, v, dout = tensors(B, Sq, Sk, H, H, seed=4)
    want = run(q, k, v, causal=True, dout=dout)
    j = Sk - Sq // 2 - 1                                     # its own query and later ones see it
    k2, v2 = k.clone(), v.clone()
    k2[:, j, :, 5] = float("nan")
    v2[:, j, :, 9] = float("inf")
    got = run(q, k2, v2, causal=True, dout=dout)
    before = j - (Sk - Sq)                                   # queries that do not see it
    assert torch.equal(got[0][:, :before], want[0][:, :before]) and torch.equal(got[1][..., :before], want[1][..., :before])
    assert torch.equal(got[2][:, :before], want[2][:, :before])
    assert torch.isnan(got[0][:, before:].float()).all()     # the documented answer of rows that see it


def test_visible_infinity_in_one_row_of_many(cuda_ok):
    import torch
    q, k, v, _ = tensors(1, 200, 200, 2, 2, seed=5)
    ids = documents(1, 200, (90, 110))
    want = run(q, k, v, doc_q=ids, doc_k=ids)
    v[0, 100, 1, 3] = float("inf")                            # document 1, head 1
    out, lse = run(q, k, v, doc_q=ids, doc_k=ids)
    assert torch.isnan(out[0, 90:, 1].float()).all()
    assert torch.equal(out[0, :90], want[0][0, :90]) and torch.equal(out[0, :, 0], want[0][0, :, 0])


@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_large_scores(cuda_ok, cap):
    """Scores of hundreds (one key takes nearly all of a row's weight) and, with a small cap, far into its bend."""
    case = (1, 200, 600, 2, 1, True, None, cap, True, None)
    q, k, v, dout = tensors(*case[:5], seed=6, size=8.0)
    terms = terms_of(case)
    out, lse, dq, dk, dv = run(q, k, v, causal=True, cap=cap, dout=dout, **terms)
    ref = reference(case, q, k, v, terms, dout)
    within(lse, ref.lse, ref.t_lse, "lse")
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(got, getattr(ref, name), getattr(ref, "t_" + name), name)


def test_growing_scores(cuda_ok):
    """Every key tile raises the maximum of the row by far more than the reference's slack of 2^32: towards the
    first keys, which the kernel takes last."""
    import torch
    q, k, v, dout = tensors(1, 130, 1000, 1, 1, seed=7)
    q[..., 0] = 40.0
    k[0, :, 0, 0] = torch.linspace(80, -80, 1000, device="cuda").bfloat16()
    out, lse, dq, dk, dv = run(q, k, v, dout=dout)
    ref = Reference(q, k, v, visible(1, 130, 1000), dout=dout)
    within(lse, ref.lse, ref.t_lse, "lse")
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(got, getattr(ref, name), getattr(ref, "t_" + name), name)


def test_strides_and_broadcast(cuda_ok):
    """Slices of a fused projection, heads-first outputs, heads and batch entries of k and v broadcast."""
    import torch
    B, S, H = 2, 200, 3
    g = torch.Generator(device="cuda").manual_seed(8)
    qkv = torch.randn((B, S, 3, H, 128), generator=g, device="cuda").bfloat16()
    dout = torch.randn((B, H, S, 128), generator=g, device="cuda").bfloat16().transpose(1, 2)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    prefix = torch.tensor([0, 77], dtype=torch.int32, device="cuda")
    want = run(*(t.contiguous() for t in (q, k, v)), causal=True, dout=dout.contiguous(), prefix=prefix)
    attn = vsa.MaskedAttention(vsa.make_mask(causal=True), B, S, S, H, H)
    out = torch.empty((B, H, S, 128), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    lse = torch.empty((B, H, S), device="cuda")
    attn.forward(q, k, v, out, lse, prefix=prefix)
    grads = torch.zeros((B, S, 3, H, 128), dtype=torch.bfloat16, device="cuda")
    attn.backward(q, k, v, out, lse, dout, grads[:, :, 0], grads[:, :, 1], grads[:, :, 2], prefix=prefix)
    for a, b in zip((out, lse, grads[:, :, 0], grads[:, :, 1], grads[:, :, 2]), want):
        assert torch.equal(a, b)
    one_k, one_v = k[:1, :, :1].expand(B, S, H, 128), v[:1, :, :1].expand(B, S, H, 128)
    got = run(q, one_k, one_v, causal=True, dout=dout, prefix=prefix)
    full = run(q, one_k.contiguous(), one_v.contiguous(), causal=True, dout=dout, prefix=prefix)
    assert all(torch.equal(a, b) for a, b in zip(got, full))


def test_scale_and_documents_of_a_longer_cache(cuda_ok):
    """A scale of its own, and queries that are the last of the cache's documents."""
    import torch
    B, Sq, Sk, H = 1, 70, 900, 2
    q, k, v, dout = tensors(B, Sq, Sk, H, H, seed=9)
    ids = documents(B, Sk, (300, 290, 310))
    terms = dict(doc_q=ids[:, Sk - Sq:], doc_k=ids)
    got = run(q, k, v, causal=True, scale=0.2, dout=dout, **terms)
    ref = Reference(q, k, v, visible(B, Sq, Sk, True, None, **terms), scale=float(torch.tensor(0.2)), dout=dout)
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), got):
        within(x, getattr(ref, name), getattr(ref, "t_" + name), name)


def test_unsorted_documents(cuda_ok):
    """Documents whose tokens are interleaved (no tile holds one only), 70 of them."""
    import torch
    B, S, H = 1, 390, 2
    q, k, v, dout = tensors(B, S, S, H, H, seed=10)
    ids = ((torch.arange(S, device="cuda") * 37) % 71 - 1).to(torch.int32)[None].contiguous()
    got = run(q, k, v, dout=dout, doc_q=ids, doc_k=ids)
    ref = Reference(q, k, v, visible(B, S, S, False, None, ids, ids), dout=dout)
    for name, x in zip(("out", "lse", "dq", "dk", "dv"), got):
        within(x, getattr(ref, name), getattr(ref, "t_" + name), name)


@pytest.mark.parametrize("B,Sq,Sk", [(1, 0, 5), (1, 5, 0), (0, 5, 5), (2, 0, 0)])
def test_nothing_to_attend(cuda_ok, B, Sq, Sk):
    import torch
    q, k, v, dout = tensors(B, Sq, Sk, 4, 2, seed=11)
    out, lse, dq, dk, dv = run(q, k, v, causal=True, dout=dout)
    assert not out.float().any() and not dq.float().any() and not dk.float().any() and not dv.float().any()
    assert torch.equal(lse, torch.full_like(lse, -math.inf))


def test_differences_agree(cuda_ok):
    """The gradients against central differences of sum(out * dout) in float64 on the formula, along a random
    direction: with a step h the difference is off by h^2 / 6 |L'''| < 1e-6 of the sums here; the kernel's part is
    bounded by the elementwise tolerances."""
    import torch
    case = (1, 90, 150, 2, 1, True, (20,), 5.0, True, None)
    q, k, v, dout = tensors(*case[:5], seed=12)
    terms = terms_of(case)
    _, _, dq, dk, dv = run(q, k, v, causal=True, cap=5.0, dout=dout, **terms)
    ref = reference(case, q, k, v, terms, dout)
    loss = lambda q, k, v: (reference(case, q, k, v, terms).out * dout.double()).sum().item()  # noqa: E731
    h = 1e-4
    for i, (name, got) in enumerate((("dq", dq), ("dk", dk), ("dv", dv))):
        at = [t.double() for t in (q, k, v)]
        e = torch.randn(at[i].shape, device="cuda", dtype=torch.float64)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * e, at[i] - h * e
        diff = (loss(*up) - loss(*down)) / (2 * h)
        have = (got.double() * e).sum().item()
        slack = (getattr(ref, "t_" + name) * e.abs()).sum().item() + 1e-6 * (got.double() * e).abs().sum().item()
        assert abs(have - diff) <= slack, (name, have, diff, slack)


def test_same_bits_again_and_two_streams(cuda_ok):
    """Equal inputs give equal bits; two calls at once on streams and workspaces of their own do not meet."""
    import torch
    sets = [tensors(1, 700, 700, 4, 2, seed=s) for s in (13, 14)]
    want = [run(*t[:3], causal=True, cap=20.0, dout=t[3]) for t in sets]
    assert all(torch.equal(a, b) for a, b in zip(run(*sets[0][:3], causal=True, cap=20.0, dout=sets[0][3]), want[0]))
    attns = [vsa.MaskedAttention(vsa.make_mask(causal=True, softcap=20.0), 1, 700, 700, 4, 2) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[torch.empty_like(x) for x in w] for w in want]
    torch.cuda.synchronize()
    for _ in range(3):
        for a, s, t, o in zip(attns, streams, sets, outs):
            a.forward(*t[:3], o[0], o[1], stream=s)
            a.backward(*t[:3], o[0], o[1], t[3], o[2], o[3], o[4], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(a, b) for a, b in zip(w, o))


def test_captured_calls_replay_on_new_inputs(cuda_ok):
    """Forward and backward in one graph, with documents, split keys (few queries) and changed inputs and masks."""
    import torch
    for Sq, Sk in ((300, 300), (3, 2000)):
        q, k, v, dout = tensors(1, Sq, Sk, 4, 2, seed=15)
        ids = documents(1, Sk, (Sk // 3, Sk - Sk // 3))
        attn = vsa.MaskedAttention(vsa.make_mask(), 1, Sq, Sk, 4, 2)
        terms = dict(doc_q=ids[:, Sk - Sq:], doc_k=ids)
        out, lse = attn.forward(q, k, v, **terms)                       # allocates the workspaces
        grads = attn.backward(q, k, v, out, lse, dout, **terms)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            attn.forward(q, k, v, out, lse, stream=s, **terms)
            attn.backward(q, k, v, out, lse, dout, *grads, stream=s, **terms)
        for seed, lengths in ((16, (Sk // 2,)), (17, (Sk - 2, 2))):
            for a, b in zip((q, k, v, dout), tensors(1, Sq, Sk, 4, 2, seed=seed)):
                a.copy_(b)
            ids.copy_(documents(1, Sk, lengths))
            graph.replay()
            torch.cuda.synchronize()
            ref = Reference(q, k, v, visible(1, Sq, Sk, False, None, **terms), dout=dout)
            within(lse, ref.lse, ref.t_lse, "lse")
            for name, x in zip(("out", "dq", "dk", "dv"), (out, *grads)):
                within(x, getattr(ref, name), getattr(ref, "t_" + name), name)
        del graph


def test_workspace_contents_do_not_matter(cuda_ok):
    """Workspaces full of NaN patterns, or left by a call of another mask, give the same bits."""
    import torch
    q, k, v, dout = tensors(2, 150, 450, 4, 2, seed=18)
    ids = documents(2, 450, (200, 249))
    terms = dict(doc_q=ids[:, 300:], doc_k=ids)
    want = run(q, k, v, dout=dout, **terms)
    attn = vsa.MaskedAttention(vsa.make_mask(), 2, 150, 450, 4, 2)
    for fill in (0xFF, 0x7F):
        out, lse = attn.forward(q, k, v, **terms)
        grads = attn.backward(q, k, v, out, lse, dout, **terms)
        assert all(torch.equal(a, b) for a, b in zip((out, lse, *grads), want))
        for held in (attn.ws_fwd, attn.ws_bwd):
            for ws in held.values():
                ws.fill_(fill)


@pytest.mark.parametrize("shape", [(4, 128, 8000, 48, 48), (4, 64, 20000, 24, 24), (1, 700, 3000, 40, 40)],
                         ids=lambda s: "x".join(map(str, s)))
def test_many_blocks_agree_with_themselves(cuda_ok, shape):
    """Hundreds of blocks whose two slots share a ring of key tiles, twenty times: always the same bits. (A slot that
    took a stage's parity for a phase that it had not seen read a tile before it had landed, about once in fifteen
    calls of the first shape.)"""
    import torch
    B, Sq, Sk, Hq, Hk = shape
    q, k, v, _ = tensors(*shape, seed=19)
    attn = vsa.MaskedAttention(vsa.make_mask(), *shape)
    first, lse = attn.forward(q, k, v)
    for _ in range(20):
        again, _ = attn.forward(q, k, v)
        assert torch.equal(first, again)
    ref = Reference(q[:1, :, :1], k[:1, :, :1], v[:1, :, :1], visible(1, Sq, Sk))
    within(first[:1, :, :1], ref.out, ref.t_out, "out")


@pytest.mark.parametrize("parity", [0, 1])
@pytest.mark.parametrize("shape", [(1, 300, 20000, 8, 8), (2, 120, 6000, 6, 6)], ids=lambda s: "x".join(map(str, s)))
def test_slots_far_apart(cuda_ok, shape, parity):
    """Every second key tile lies so far above the one before that its slot raises the reference each time and falls
    behind the other slot of the block: the shared ring must not move on by more than a stage that a slot has seen
    (its parity would come round again, and the slot would wait for good)."""
    import torch
    B, Sq, Sk, Hq, Hk = shape
    q, k, v, _ = tensors(*shape, seed=23)
    tile = torch.arange(Sk, device="cuda") // 128
    up = 23.0 * ((int(tile[-1]) - tile) // 2 % 13) * (tile % 2 == parity)
    q[..., 0] = 1.0
    k[..., 0] = (up * math.sqrt(128)).to(k.dtype)[None, :, None]
    attn = vsa.MaskedAttention(vsa.make_mask(causal=True), *shape)
    first, lse = attn.forward(q, k, v)
    assert vsa.masked_attn_status(attn.ws_fwd[0]) == vsa.OK
    for _ in range(10):
        again, _ = attn.forward(q, k, v)
        assert torch.equal(first, again)
    assert vsa.masked_attn_status(attn.ws_fwd[0]) == vsa.OK
    ref = Reference(q[:, :, :2], k[:, :, :2], v[:, :, :2], visible(B, Sq, Sk, causal=True))
    within(first[:, :, :2], ref.out, ref.t_out, "out")
    within(lse[:, :2], ref.lse, ref.t_lse, "lse")


def test_prefixes_of_every_size(cuda_ok):
    """The smallest and largest 32-bit prefixes: none, and all keys."""
    import torch
    case = (3, 200, 333, 2, 1, True, (-2 ** 31, 2 ** 31 - 1, -1), 0.0, False, None)
    q, k, v, dout = tensors(*case[:5], seed=29)
    terms = terms_of(case)
    out, lse, dq, dk, dv = run(q, k, v, causal=True, dout=dout, **terms)
    ref = reference(case, q, k, v, {"prefix": terms["prefix"].double()}, dout)
    for name, got in (("lse", lse), ("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(got, getattr(ref, name), getattr(ref, "t_" + name), name)


@pytest.mark.parametrize("cap", [1e6, 1e30, 3e38])
@pytest.mark.parametrize("bias", [False, True])
def test_caps_far_above_the_scores(cuda_ok, cap, bias):
    """A cap c far above the scores is none: s - c tanh(s / c) <= s^3 / (3 c^2) < 2^-24 |s| for |s| < 400. The bounds
    are those without a cap, and 2^-23 |s| for the polynomial, below their 64 u."""
    case = (1, 300, 300, 2, 1, True, None, 0.0, bias, None)
    q, k, v, dout = tensors(*case[:5], seed=31)
    terms = terms_of(case)
    out, lse, dq, dk, dv = run(q, k, v, causal=True, cap=cap, dout=dout, **terms)
    ref = reference(case, q, k, v, terms, dout)
    for name, got in (("lse", lse), ("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(got, getattr(ref, name), getattr(ref, "t_" + name), name)


@pytest.mark.parametrize("cap", [1e-3, 1e-30, 1e-40])
def test_caps_far_below_the_scores(cuda_ok, cap):
    """Every score at the cap (or 0 for a query of zeros): nearly equal weights, no gradient of q and k."""
    case = (1, 150, 270, 2, 2, True, None, cap, False, None)
    q, k, v, dout = tensors(*case[:5], seed=37)
    q[:, 5] = 0
    out, lse, dq, dk, dv = run(q, k, v, causal=True, cap=cap, dout=dout)
    ref = reference(case, q, k, v, {}, dout)
    for name, got in (("lse", lse), ("out", out), ("dv", dv)):
        within(got, getattr(ref, name), getattr(ref, "t_" + name), name)
    assert dq.isfinite().all() and dk.isfinite().all()


@pytest.mark.parametrize("cap", [3.0, 30.0, 1e6])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("loud", [float("inf"), float("nan"), 3e38, 4e4])
def test_masked_places_change_nothing_under_a_cap(cuda_ok, cap, bias, loud):
    """Padding rows that hold infinities, NaN or numbers far beyond the cap: the same bits as with zeros there, in the
    other rows of their tiles too."""
    import torch
    case, clean, terms, pad = with_padding()
    if bias:
        terms["slopes"] = slopes_of(case[3])
    for t in clean:
        t[pad] = 0
    want = run(*clean[:3], causal=True, cap=cap, dout=clean[3], **terms)
    dirty = [t.clone() for t in clean]
    for t in dirty:
        t[pad] = torch.where(torch.rand(t[pad].shape, device="cuda") < 0.5, loud, -loud).to(t.dtype)
    got = run(*dirty[:3], causal=True, cap=cap, dout=dirty[3], **terms)
    for name, a, b in zip(("out", "lse", "dq", "dk", "dv"), got, want):
        assert torch.equal(a, b), name


def later_keys(Sq, Sk, H, cap, bias, at):
    """A key that only later queries see reaches no earlier one, whatever it holds: the same bits."""
    import torch
    q, k, v, dout = tensors(1, Sq, Sk, H, H, seed=41)
    terms = {"slopes": slopes_of(H)} if bias else {}
    want = run(q, k, v, causal=True, cap=cap, dout=dout, **terms)
    for j in at:
        for loud in (float("nan"), float("inf"), 1e6):
            k2, v2 = k.clone(), v.clone()
            k2[:, j] = loud
            v2[:, j, :, 9] = float("inf")
            got = run(q, k2, v2, causal=True, cap=cap, dout=dout, **terms)
            before = max(0, j - (Sk - Sq))                   # queries that do not see it
            assert torch.equal(got[0][:, :before], want[0][:, :before]), ("out", j, loud)
            assert torch.equal(got[1][..., :before], want[1][..., :before]), ("lse", j, loud)
            assert torch.equal(got[2][:, :before], want[2][:, :before]), ("dq", j, loud)


@pytest.mark.parametrize("bias", [False, True])
def test_first_visible_key_of_a_warps_last_row(cuda_ok, bias):
    """Keys at multiples of 64 that only the last row of 32 sees in their half of a tile: the others of the warp meet
    their own first keys in the half before, where that row has found a maximum or not."""
    later_keys(700, 765, 8, 0.0, bias, range(128, 765, 64))


@pytest.mark.parametrize("cap", [3.0, 30.0, 1e6])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("Sq,Sk", [(1, 500), (40, 500), (333, 500), (200, 265), (700, 765)])
def test_later_keys_may_hold_anything_under_a_cap(cuda_ok, cap, bias, Sq, Sk):
    later_keys(Sq, Sk, 4, cap, bias, {Sk - Sq // 2 - 1, 128 if Sk - Sq < 128 else Sk - 1, (Sk - 1) // 64 * 64})


@pytest.mark.parametrize("bias", [False, True])
def test_scores_beside_others_far_beyond_the_cap(cuda_ok, bias):
    """Under a cap of 10^6, rows of ordinary scores beside one in sixteen whose scores reach the cap: s - c tanh(s / c)
    is below 2^-24 |s| for the ordinary ones, so that they keep the bounds of a call without a cap."""
    import torch
    case = (1, 300, 300, 2, 1, True, None, 0.0, bias, None)
    q, k, v, dout = tensors(*case[:5], seed=43)
    terms = terms_of(case)
    loud = torch.arange(300, device="cuda") % 16 == 5
    ref = reference(case, q, k, v, terms, dout)
    q = torch.where(loud[None, :, None, None], q * 1e6, q)
    out, lse, dq, dk, dv = run(q, k, v, causal=True, cap=1e6, dout=dout, **terms)
    assert torch.isfinite(lse).all()
    within(lse[..., ~loud], ref.lse[..., ~loud], ref.t_lse[..., ~loud], "lse")
    for name, got in (("out", out), ("dq", dq)):
        within(got[:, ~loud], getattr(ref, name)[:, ~loud], getattr(ref, "t_" + name)[:, ~loud], name)


def test_cache_of_more_than_65535_tiles(cuda_ok):
    """Two queries at the end of a cache of 8,388,900 positions. The bias leaves weight to the last keys only (e^-8000
    is 0), so that the formula over the last 8,000 is the formula over all; an infinity at the last key, which the
    first query does not see, is found where its tile lies."""
    import torch
    Sk, near = 8388900, 8000
    g = torch.Generator(device="cuda").manual_seed(61)
    q, dout = (torch.randn((1, 2, 1, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn((1, Sk, 1, 128), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    slopes = torch.ones(1, device="cuda")
    attn = vsa.MaskedAttention(vsa.make_mask(causal=True), 1, 2, Sk, 1, 1)
    out, lse = attn.forward(q, k, v, slopes=slopes)
    dq, dk, dv = attn.backward(q, k, v, out, lse, dout, slopes=slopes)
    assert all(vsa.masked_attn_status(ws) == vsa.OK for ws in (*attn.ws_fwd.values(), *attn.ws_bwd.values()))
    kn, vn = k[:, -near:], v[:, -near:]
    ref = Reference(q, kn, vn, visible(1, 2, near, True), slopes=slopes, dout=dout)
    for name, got in (("lse", lse), ("out", out), ("dq", dq), ("dk", dk[:, -near:]), ("dv", dv[:, -near:])):
        within(got, getattr(ref, name), getattr(ref, "t_" + name), name)
    assert not dk[:, :-near].any() and not dv[:, :-near].any()
    v[:, -1, :, 3] = float("inf")
    again, lse2 = attn.forward(q, k, v, slopes=slopes)
    assert torch.equal(again[:, 0], out[:, 0]) and again[:, 1].isnan().all() and torch.equal(lse2[..., 0], lse[..., 0])


def test_queries_of_more_than_65535_tiles(cuda_ok):
    """8,388,900 queries over five keys, without a mask; only the first and last queries have a gradient."""
    import torch
    Sq, Sk, ends = 8388900, 5, 300
    g = torch.Generator(device="cuda").manual_seed(62)
    q = torch.randn((1, Sq, 1, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn((1, Sk, 1, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    dout = torch.zeros_like(q)
    at = torch.cat([torch.arange(ends), torch.arange(Sq - ends, Sq)]).cuda()
    dout[:, at] = torch.randn((1, 2 * ends, 1, 128), generator=g, device="cuda").bfloat16()
    attn = vsa.MaskedAttention(vsa.make_mask(), 1, Sq, Sk, 1, 1)
    out, lse = attn.forward(q, k, v)
    dq, dk, dv = attn.backward(q, k, v, out, lse, dout)
    assert all(vsa.masked_attn_status(ws) == vsa.OK for ws in (*attn.ws_fwd.values(), *attn.ws_bwd.values()))
    ref = Reference(q[:, at], k, v, torch.ones((1, 2 * ends, Sk), dtype=torch.bool, device="cuda"), dout=dout[:, at])
    for name, got in (("lse", lse[..., at]), ("out", out[:, at]), ("dq", dq[:, at]), ("dk", dk), ("dv", dv)):
        within(got, getattr(ref, name), getattr(ref, "t_" + name), name)
    dq[:, at] = 0
    assert not dq.any()


@pytest.mark.parametrize("case", [(2, 2300, 2300, 12, 4, True, (700,), 0.0, False, None),
                                  (1, 3000, 3000, 24, 24, False, None, 0.0, False, (700, 1500, 90, 600)),
                                  (2, 2300, 2300, 12, 4, True, None, 20.0, True, None)], ids=ident)
def test_gradients_over_many_waves_of_blocks(cuda_ok, case):
    """Several blocks after one another on each SM: equal bits every time, and within the formula's bounds in the
    first and last heads."""
    import torch
    B, Sq, Sk, Hq, Hk, causal, prefix, cap, bias, docs = case
    q, k, v, dout = tensors(B, Sq, Sk, Hq, Hk, seed=63)
    terms = terms_of(case)
    first = run(q, k, v, causal=causal, cap=cap, dout=dout, **terms)
    attn = vsa.MaskedAttention(vsa.make_mask(causal=causal, softcap=cap), B, Sq, Sk, Hq, Hk)
    for _ in range(10):
        out, lse = attn.forward(q, k, v, **terms)
        grads = attn.backward(q, k, v, out, lse, dout, **terms)
        assert all(torch.equal(a, b) for a, b in zip((out, lse, *grads), first))
    n = Hq // Hk
    for h in (0, Hk - 1):
        rows = slice(h * n, (h + 1) * n)
        part = dict(terms, slopes=terms["slopes"][rows]) if bias else terms
        ref = Reference(q[:, :, rows], k[:, :, h:h + 1], v[:, :, h:h + 1],
                        visible(B, Sq, Sk, causal, terms.get("prefix"), terms.get("doc_q"), terms.get("doc_k")), cap,
                        part.get("slopes"), dout=dout[:, :, rows])
        for name, got in zip(("out", "lse", "dq", "dk", "dv"),
                             (first[0][:, :, rows], first[1][:, rows], first[2][:, :, rows],
                              first[3][:, :, h:h + 1], first[4][:, :, h:h + 1])):
            within(got, getattr(ref, name), getattr(ref, "t_" + name), name)


def test_status_of_the_latest_calls(cuda_ok):
    """A status word that a call left behind is read through the object (written here by the host), and cleared by the
    next call on that workspace."""
    import torch
    q, k, v, dout = tensors(1, 200, 200, 2, 2, seed=67)
    attn = vsa.MaskedAttention(vsa.make_mask(), 1, 200, 200, 2, 2)
    assert attn.status() == vsa.OK
    out, lse = attn.forward(q, k, v)
    attn.backward(q, k, v, out, lse, dout)
    assert attn.status() == vsa.OK
    for held, again in ((attn.ws_fwd, lambda: attn.forward(q, k, v)),
                        (attn.ws_bwd, lambda: attn.backward(q, k, v, out, lse, dout))):
        held[0][:4].view(torch.int32).fill_(vsa.ERR_TIMEOUT)
        assert attn.status() == vsa.ERR_TIMEOUT
        again()
        assert attn.status() == vsa.OK


@pytest.mark.parametrize("case", [
    (2, 1, 3001, 6, 2, True, None, 0.0, False, None),
    (1, 1, 33, 2, 2, False, None, 0.0, False, None),
    (1, 7, 900, 8, 2, True, None, 25.0, True, None),
    (1, 64, 1500, 4, 2, True, (1200,), 0.0, True, None),
    (2, 128, 700, 2, 2, False, None, 30.0, False, None),
    (1, 100, 520, 4, 4, True, None, 0.0, False, (100, 1, 130, 200)),
    (1, 3, 5000, 24, 1, False, None, 0.0, False, (3, 2000, 2997)),
    (1, 128, 128, 1, 1, True, None, 0.0, True, None),
], ids=ident)
@pytest.mark.parametrize("size", [1.3, 8.0])
def test_rows_of_one_tile_keep_two_terms_of_each_probability(cuda_ok, case, size):
    """Queries that fit one tile of 128 rows: a probability enters the second product as two bf16 terms, whose sum is
    within 2^-16 of it (each rounds by 2^-8, the second what the first left), so that in the bound of the output
    2^-16 stands for 2^-8."""
    import torch
    B, Sq, Sk, Hq, Hk, causal, prefix, cap, bias, docs = case
    q, k, v, _ = tensors(*case[:5], seed=71, size=size)
    terms = terms_of(case)
    out, lse = run(q, k, v, causal=causal, cap=cap, **terms)
    ref = reference(case, q, k, v, terms)
    within(lse, ref.lse, ref.t_lse, "lse")
    see = visible(B, Sq, Sk, causal, terms.get("prefix"), terms.get("doc_q"), terms.get("doc_k"))
    size_of = reference(case, q, k, v.abs(), terms).out                  # sum p |v|
    was = (ref.t_out - E * ref.out.abs()) / (1 + E)                      # the bound before the output's rounding
    now = was - (E - 2.0 ** -16) * size_of
    assert see.any() and (now >= 0).all()
    within(out, ref.out, now + E * (ref.out.abs() + now), "out")


@pytest.mark.parametrize("Sq", [1, 128, 129])
def test_visible_infinities_without_a_mask(cuda_ok, Sq):
    """An infinity in a visible v reaches its own channel only, of every query that sees it: the infinity, or for up to
    128 queries (whose two terms of a probability take it with both signs) NaN."""
    import torch
    q, k, v, _ = tensors(1, Sq, 300, 2, 1, seed=73)
    want, lse = run(q, k, v)
    v[0, 250, 0, 3] = float("inf")
    got, lse2 = run(q, k, v)
    rest = torch.arange(128, device="cuda") != 3
    assert torch.equal(got[..., rest], want[..., rest]) and torch.equal(lse, lse2)
    assert not torch.isfinite(got[..., 3]).any()
    if Sq > 128:
        assert (got[..., 3] == float("inf")).all()
