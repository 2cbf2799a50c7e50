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
