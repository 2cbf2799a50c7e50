"""The operators around the sparse attention call as measured cases: three-axis
rotary positions, layer norm, and dense attention with capped scores, a distance
bias, document and prefix masks; each in a plain form (elementary torch
operations) and through this package's own calls.

Head dim 128 and the 24 heads, prefix lengths and latent grids are those of this
repository's workloads; hidden widths and cache lengths are generic.
"""

import math

import torch

own = False

D = 128
FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # rotary positions of one new token per sequence: a streaming step of four sequences
        dict(name="rope_token", op="rope", B=4, S=1, Hq=24, Hk=24, dims="44,42,42", pairing="adjacent",
             dtype="bf16", out="bf16", grid="1,1,1", cond=0, start=900000, inverse=False, shared=False),
        # the packed [conditioning | video] sequence of the 5 s, 1344x768 workload
        dict(name="rope_5s", op="rope", B=1, S=133696, Hq=24, Hk=24, dims="44,42,42", pairing="adjacent",
             dtype="bf16", out="bf16", grid="32,48,84", cond=4672, start=0, inverse=False, shared=True),
        # the gradients that the sparse attention's backward leaves in fp32, shared key heads, 17k tokens
        dict(name="rope_grad", op="rope", B=1, S=17408, Hq=24, Hk=8, dims="16,56,56", pairing="halves",
             dtype="f32", out="bf16", grid="16,32,32", cond=1024, start=0, inverse=True, shared=True),
        # few rows of a hidden state, as in a streaming step
        dict(name="norm_rows", op="norm", B=1, S=4, H=1, N=4096, dtype="bf16", wtype="bf16", affine=True),
        # query and key heads in front of the rotation, 17k tokens x 24 heads
        dict(name="norm_heads", op="norm", B=1, S=17408, H=24, N=128, dtype="bf16", wtype="f32", affine=True),
        # hidden rows of a transformer block, forward and backward with the weight's gradient
        dict(name="norm_train", op="norm_train", B=1, S=17408, H=1, N=5120, dtype="bf16", wtype="f32", affine=True),
        # the same in fp32 at an odd width and an odd number of rows
        dict(name="norm_train_odd", op="norm_train", B=3, S=1231, H=1, N=1153, dtype="f32", wtype="f32", affine=True),
        # one new token per sequence over a long cache of shared key heads, causal
        dict(name="attn_token", op="attn", B=4, Sq=1, Sk=33001, Hq=24, Hk=8, causal=True, prefix=0, cap=0.0,
             bias=False, docs=""),
        # dense attention of a 24-head sequence, no mask: what a refused sparse case runs
        dict(name="attn_dense", op="attn", B=1, Sq=8192, Sk=8192, Hq=24, Hk=24, causal=False, prefix=0, cap=0.0,
             bias=False, docs=""),
        # a chunk of a causal video behind a bidirectional conditioning prefix, capped scores and a distance bias
        dict(name="attn_stream", op="attn", B=2, Sq=1111, Sk=5003, Hq=24, Hk=8, causal=True, prefix=700, cap=30.0,
             bias=True, docs=""),
        # several clips packed into one training sequence with padding at its end: forward and backward
        dict(name="attn_packed", op="attn_train", B=1, Sq=8192, Sk=8192, Hq=24, Hk=24, causal=False, prefix=0,
             cap=0.0, bias=False, docs="2048,1000,3100,64,1700,1"),
        # causal training with a cap and a bias at an odd length, shared key heads
        dict(name="attn_causal", op="attn_train", B=2, Sq=1555, Sk=1555, Hq=8, Hk=4, causal=True, prefix=131,
             cap=20.0, bias=True, docs=""),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "norm", "norm_train", "attn", "attn_train"])
    if op == "rope":
        T, h, w = _log(rng, 1, 32), _log(rng, 1, 48), _log(rng, 1, 84)
        cond = rng.choice([0, _log(rng, 1, 4672)])
        S = T * h * w + cond
        Hk = rng.choice([1, 2, 8, 24])
        Hq = Hk * rng.choice([1, 1, 3]) if Hk < 24 else 24
        dims = rng.choice(["44,42,42", "16,56,56", "64,32,32", "32,32,32", "0,64,64", "128,0,0", "2,62,60"])
        inverse = rng.random() < 0.5
        dtype = rng.choice(["bf16", "f16", "f32"]) if S < 60000 else rng.choice(["bf16", "f16"])
        B = 1 if S > 20000 else rng.choice([1, 2, 3])
        return dict(op=op, B=B, S=S, Hq=Hq, Hk=Hk, dims=dims, pairing=rng.choice(["adjacent", "halves"]),
                    dtype=dtype, out=rng.choice([dtype, dtype, "bf16"]), grid="%d,%d,%d" % (T, h, w), cond=cond,
                    start=rng.choice([0, rng.randrange(0, 1000000)]), inverse=inverse, shared=rng.random() < 0.5)
    if op in ("norm", "norm_train"):
        heads = rng.random() < 0.4
        N = 128 if heads else rng.choice([_log(rng, 1, 16384), 8 * _log(rng, 16, 1024)])
        H = rng.choice([1, 3, 8, 24]) if heads else 1
        rows = _log(rng, 1, max(2, min(40000, 17408 * 5120 // (N * H))))
        B = rng.choice([1, 2]) if rows > 1 else 1
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        return dict(op=op, B=B, S=max(1, rows // B), H=H, N=N, dtype=dtype, wtype=rng.choice([dtype, "f32"]),
                    affine=op == "norm_train" or rng.random() < 0.8)
    Hk = rng.choice([1, 2, 3, 8, 24])
    Hq = Hk * rng.choice([1, 1, 2, 3]) if Hk < 24 else 24
    cap = rng.choice([0.0, 0.0, 15.0, 50.0])
    bias = rng.random() < 0.4
    kind = rng.choice(["full", "causal", "prefix", "docs", "docs_causal"])
    if op == "attn" and rng.random() < 0.5:      # a cache and few new tokens
        Sk = _log(rng, 64, 40000)
        Sq = min(Sk, rng.choice([1, 1, 2, 7, 64, 300]))
        B = rng.choice([1, 2, 4])
        kind = rng.choice(["full", "causal", "prefix"])
    else:
        B = rng.choice([1, 1, 2])
        Sk = _log(rng, 17 if op == "attn_train" else 1, 6000 if B == 1 else 4000)
        Sq = Sk if kind in ("docs", "docs_causal") or op == "attn_train" or rng.random() < 0.5 else _log(rng, 1, Sk)
    docs = ""
    if kind in ("docs", "docs_causal"):
        left, parts = Sk, []
        while left > 0 and len(parts) < 12 and rng.random() < 0.9:
            parts.append(_log(rng, 1 if parts else min(17, left), left))
            left -= parts[-1]
        docs = ",".join(str(n) for n in (parts or [Sk]))
    return dict(op=op, B=B, Sq=Sq, Sk=Sk, Hq=Hq, Hk=Hk, causal=kind in ("causal", "prefix", "docs_causal"),
                prefix=rng.randrange(0, Sk + 1) if kind == "prefix" else 0, cap=cap, bias=bias, docs=docs)


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


# ------------------------------------------------------------------ inputs
def _positions(case, gen, device):
    """int32 [S, 3], or [B, S, 3] where sequences stand at positions of their own."""
    T, h, w = _ints(case["grid"])
    cond = torch.arange(case["cond"], device=device)[:, None].expand(-1, 3)
    n = torch.arange(T * h * w, device=device)
    video = torch.stack([n // (h * w), n // w % h, n % w], 1) + case["cond"]
    pos = torch.cat([cond, video]) + case["start"]
    if not case["shared"]:
        step = torch.randint(0, 1000, (case["B"], 1, 3), generator=gen, device=device)
        pos = pos[None] + step
    return pos.to(torch.int32).contiguous()


def _documents(case, device):
    """int32 [B, S] document of each token, -1 behind the last one."""
    ids = torch.full((case["Sk"],), -1, dtype=torch.int32, device=device)
    at = 0
    for i, n in enumerate(_ints(case["docs"])):
        ids[at:at + n] = i
        at += n
    return ids.expand(case["B"], -1).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(1000003 * seed + 17)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    st = {"case": case}
    if case["op"] == "rope":
        dt, out = FLOATS[case["dtype"]], FLOATS[case["out"]]
        B, S, Hq, Hk = case["B"], case["S"], case["Hq"], case["Hk"]
        st["q"], st["k"] = normal(B, S, Hq, D).to(dt), normal(B, S, Hk, D).to(dt)
        st["q_out"], st["k_out"] = (torch.empty(x.shape, dtype=out, device=dev) for x in (st["q"], st["k"]))
        st["pos"] = _positions(case, gen, dev)
    elif case["op"] in ("norm", "norm_train"):
        dt, wt = FLOATS[case["dtype"]], FLOATS[case["wtype"]]
        shape = (case["B"], case["S"], case["H"], case["N"])
        # a residual stream: rows of different size, a common offset and a few loud channels
        size = torch.exp(normal(*shape[:3], 1))
        loud = torch.exp(normal(case["N"]))
        st["x"] = (size * (normal(*shape) * loud + 0.5)).to(dt)
        st["y"] = torch.empty_like(st["x"])
        rows = shape[:3]
        st["mean"], st["rstd"] = (torch.empty(rows, dtype=torch.float32, device=dev) for _ in range(2))
        st["w"] = (1 + 0.2 * normal(case["N"])).to(wt) if case["affine"] else None
        st["b"] = (0.2 * normal(case["N"])).to(wt) if case["affine"] else None
        if case["op"] == "norm_train":
            st["dy"] = normal(*shape).to(dt)
            st["dx"] = torch.empty_like(st["dy"])
            st["dw"], st["db"] = (torch.empty(case["N"], dtype=torch.float32, device=dev) for _ in range(2))
    else:
        B, Sq, Sk, Hq, Hk = (case[n] for n in ("B", "Sq", "Sk", "Hq", "Hk"))
        bf = torch.bfloat16
        st["q"], st["k"], st["v"] = ((1.3 * normal(B, S, H, D)).to(bf) for S, H in ((Sq, Hq), (Sk, Hk), (Sk, Hk)))
        st["doc"] = _documents(case, dev) if case["docs"] else None
        st["prefix"] = torch.full((B,), case["prefix"], dtype=torch.int32, device=dev) if case["prefix"] else None
        st["slopes"] = (2.0 ** (-2.0 - 6.0 * torch.arange(Hq, device=dev) / Hq)).float() if case["bias"] else None
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((B, Hq, Sq), dtype=torch.float32, device=dev)
        if case["op"] == "attn_train":
            st["dout"] = normal(B, Sq, Hq, D).to(bf)
            st["dq"], st["dk"], st["dv"] = (torch.empty_like(st[n]) for n in ("q", "k", "v"))
    return st


# ------------------------------------------------------------------ plain forms
THETA = 10000.0
EPS = 1e-6


def _pairs(dims, pairing, device):
    """Channels (a, b) of each rotated pair, its axis and its frequency."""
    a, b, axis, freq = [], [], [], []
    at = 0
    for ax, d in enumerate(_ints(dims)):
        i = torch.arange(d // 2, device=device)
        a.append(at + (2 * i if pairing == "adjacent" else i))
        b.append(at + (2 * i + 1 if pairing == "adjacent" else i + d // 2))
        axis.append(torch.full_like(i, ax))
        freq.append(THETA ** (-2.0 * i.double() / max(d, 1)))
        at += d
    return torch.cat(a), torch.cat(b), torch.cat(axis), torch.cat(freq)


def _plain_rope(st):
    case = st["case"]
    a, b, axis, freq = _pairs(case["dims"], case["pairing"], st["q"].device)
    angle = st["pos"].double()[..., axis] * freq
    cos, sin = angle.cos().float().unsqueeze(-2), angle.sin().float().unsqueeze(-2)
    if case["inverse"]:
        sin = -sin

    def turned(x):
        x = x.float()
        y = x.clone()
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., a] * sin + x[..., b] * cos
        return y.to(FLOATS[case["out"]])
    return {"q": turned(st["q"]), "k": turned(st["k"])}


def _plain_norm(st):
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + EPS)
    xh = xc * rstd
    y = xh
    if st["w"] is not None:
        y = y * st["w"].float() + st["b"].float()
    out = {"y": y.to(st["x"].dtype), "mean": mean.squeeze(-1), "rstd": rstd.squeeze(-1)}
    if "dy" in st:
        dy = st["dy"].float()
        g = dy * st["w"].float()
        dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
        out.update(dx=dx.to(st["dy"].dtype), dw=(dy * xh).sum((0, 1, 2)), db=dy.sum((0, 1, 2)))
    return out


def _visible(case, st):
    """bool [B, 1, Sq, Sk]: the pairs that take part."""
    Sq, Sk = case["Sq"], case["Sk"]
    dev = st["q"].device
    i = torch.arange(Sq, device=dev)[:, None] + (Sk - Sq)
    j = torch.arange(Sk, device=dev)[None, :]
    see = torch.ones((1, 1, Sq, Sk), dtype=torch.bool, device=dev)
    if case["causal"]:
        see = see & ((j <= i) | (j < case["prefix"]))
    if st["doc"] is not None:
        dk = st["doc"]
        dq = dk[:, Sk - Sq:]
        see = see & ((dq[:, :, None] == dk[:, None, :]) & (dq[:, :, None] >= 0))[:, None]
    return see


def _scores(case, st, q, k):
    """q, k [B, H, S, D] of one type -> masked scores and the tanh of the cap (or None)."""
    s = (q @ k.transpose(-1, -2)) / math.sqrt(D)
    t = None
    if case["cap"]:
        t = torch.tanh(s / case["cap"])
        s = case["cap"] * t
    if st["slopes"] is not None:
        i = torch.arange(case["Sq"], device=q.device)[:, None] + (case["Sk"] - case["Sq"])
        j = torch.arange(case["Sk"], device=q.device)[None, :]
        s = s - st["slopes"].to(q.dtype)[:, None, None] * (i - j).abs()
    return s.masked_fill(~_visible(case, st), -math.inf), t


def _heads(x, group):
    """[B, S, H, D] -> [B, H * group, S, D]"""
    return x.transpose(1, 2).repeat_interleave(group, 1)


def _plain_attn(st):
    case = st["case"]
    g = case["Hq"] // case["Hk"]
    B, Hk = case["B"], case["Hk"]
    q, k, v = _heads(st["q"].float(), 1), _heads(st["k"].float(), g), _heads(st["v"].float(), g)
    s, t = _scores(case, st, q, k)
    top = s.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    p = p / total.clamp_min(1e-37)
    o = p @ v
    out = {"out": o.transpose(1, 2).to(torch.bfloat16).contiguous(), "lse": lse}
    if "dout" in st:
        do = _heads(st["dout"].float(), 1)
        ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
        if t is not None:
            ds = ds * (1 - t * t)
        ds = ds / math.sqrt(D)
        grads = {"dq": ds @ k, "dk": ds.transpose(-1, -2) @ q, "dv": p.transpose(-1, -2) @ do}
        grads["dk"], grads["dv"] = (grads[n].view(B, Hk, g, -1, D).sum(2) for n in ("dk", "dv"))
        out.update({n: x.transpose(1, 2).to(torch.bfloat16).contiguous() for n, x in grads.items()})
    return out


# ------------------------------------------------------------------ this package's calls
def _own_rope(st):
    from block_sparse_video_geometry_b200 import vsa
    case = st["case"]
    rope = vsa.make_rope(dims=tuple(_ints(case["dims"])), theta=THETA,
                         pairing=vsa.ROPE_HALVES if case["pairing"] == "halves" else vsa.ROPE_ADJACENT)
    call = vsa.rope_bwd if case["inverse"] else vsa.rope_fwd
    call(rope, st["pos"], st["q"], st["k"], st["q_out"], st["k_out"])
    return {"q": st["q_out"], "k": st["k_out"]}


def _own_norm(st):
    from block_sparse_video_geometry_b200 import vsa
    vsa.layer_norm_fwd(st["x"], st["w"], st["b"], EPS, st["y"], st["mean"], st["rstd"])
    out = {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}
    if "dy" in st:
        if "ws" not in st:
            n = vsa.layer_norm_bwd_workspace_size(st["x"])
            st["ws"] = torch.empty(n, dtype=torch.uint8, device=st["x"].device)
        vsa.layer_norm_bwd(st["dy"], st["x"], st["w"], st["mean"], st["rstd"], st["dx"], st["dw"], st["db"], st["ws"])
        out.update(dx=st["dx"], dw=st["dw"], db=st["db"])
    return out


def _own_attn(st):
    from block_sparse_video_geometry_b200 import vsa
    case = st["case"]
    if "attn" not in st:
        mask = vsa.make_mask(causal=case["causal"], softcap=case["cap"])
        st["attn"] = vsa.MaskedAttention(mask, case["B"], case["Sq"], case["Sk"], case["Hq"], case["Hk"])
    terms = dict(prefix=st["prefix"], slopes=st["slopes"])
    if st["doc"] is not None:
        terms.update(doc_q=st["doc"][:, case["Sk"] - case["Sq"]:], doc_k=st["doc"])
    st["attn"].forward(st["q"], st["k"], st["v"], st["out"], st["lse"], **terms)
    out = {"out": st["out"], "lse": st["lse"]}
    if "dout" in st:
        st["attn"].backward(st["q"], st["k"], st["v"], st["out"], st["lse"], st["dout"], st["dq"], st["dk"], st["dv"],
                            **terms)
        out.update(dq=st["dq"], dk=st["dk"], dv=st["dv"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_rope(state) if op == "rope" else _own_norm(state) if op.startswith("norm") else _own_attn(state)
    return _plain_rope(state) if op == "rope" else _plain_norm(state) if op.startswith("norm") else _plain_attn(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _visible_pairs(case):
    """Visible (query, key) pairs of one batch entry and head."""
    Sq, Sk, at, pairs = case["Sq"], case["Sk"], 0, 0
    spans = _ints(case["docs"]) or [Sk]
    for n in spans:
        lo, hi = max(at, Sk - Sq), at + n           # the queries of this document, as key positions
        if case["causal"] and hi > lo:
            p = min(max(case["prefix"] - at, 0), n)   # keys of it that every query sees
            first, last = lo - at + 1, hi - at        # visible keys of its first and last query, by order alone
            count = last - first + 1
            below = max(0, min(count, p - first + 1))
            pairs += below * p + (first + below + last) * (count - below) // 2
        else:
            pairs += max(0, hi - lo) * n
        at += n
    return pairs


def work(case):
    if case["op"] == "rope":
        n = case["B"] * case["S"] * (case["Hq"] + case["Hk"]) * D
        pos = case["S"] * 12 * (1 if case["shared"] else case["B"])
        rotated = sum(_ints(case["dims"])) / D
        return {"bytes": n * (SIZE[case["dtype"]] + SIZE[case["out"]]) + pos, "flops": int(3 * n * rotated)}
    if case["op"] in ("norm", "norm_train"):
        rows = case["B"] * case["S"] * case["H"]
        n, size, w = rows * case["N"], SIZE[case["dtype"]], SIZE[case["wtype"]] * case["N"]
        fwd = 2 * n * size + 8 * rows + (2 * w if case["affine"] else 0)
        if case["op"] == "norm":
            return {"bytes": fwd, "flops": 7 * n}
        return {"bytes": fwd + 2 * n * size + 8 * case["N"], "flops": 18 * n}
    B, Sq, Sk, Hq, Hk = (case[n] for n in ("B", "Sq", "Sk", "Hq", "Hk"))
    q, kv = B * Sq * Hq * D * 2, B * Sk * Hk * D * 2
    pairs = B * Hq * _visible_pairs(case)
    if case["op"] == "attn":
        return {"bytes": 2 * q + 2 * kv + 4 * B * Hq * Sq, "flops": 4 * D * pairs}
    return {"bytes": 4 * q + 4 * kv + 4 * B * Hq * Sq, "flops": 14 * D * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rope(st):
    case = st["case"]
    dims, T = _ints(case["dims"]), st["pos"].double()
    out = {}
    for name in ("q", "k"):
        x = st[name].double()
        parts, at = [], 0
        for ax, d in enumerate(dims):
            blk = x[..., at:at + d]
            z = torch.complex(blk[..., 0::2], blk[..., 1::2]) if case["pairing"] == "adjacent" else \
                torch.complex(blk[..., :d // 2], blk[..., d // 2:])
            w = torch.exp(-math.log(THETA) * torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / max(d, 1))
            a = T[..., ax, None] * w
            a = (-a if case["inverse"] else a).unsqueeze(-2)
            z = z * torch.complex(torch.cos(a), torch.sin(a))
            parts.append(torch.stack([z.real, z.imag], -1).flatten(-2) if case["pairing"] == "adjacent" else
                         torch.cat([z.real, z.imag], -1))
            at += d
        out[name] = torch.cat(parts + [x[..., at:]], -1)
    return out


def _exact_norm(st):
    x = st["x"].double().flatten(0, 2)
    var, mean = torch.var_mean(x, -1, unbiased=False)
    rstd = 1.0 / torch.sqrt(var + EPS)
    w = st["w"].double() if st["w"] is not None else torch.ones_like(x[0])
    b = st["b"].double() if st["b"] is not None else torch.zeros_like(x[0])
    xh = (x - mean[:, None]) * rstd[:, None]
    shape = st["x"].shape
    out = {"y": (xh * w + b).view(shape), "mean": mean.view(shape[:3]), "rstd": rstd.view(shape[:3])}
    if "dy" in st:
        dy = st["dy"].double().flatten(0, 2)
        g, N = dy * w, x.shape[1]
        c1, c2 = g.sum(1) / N, torch.einsum("rn,rn->r", g, xh) / N
        dx = (g - c1[:, None] - xh * c2[:, None]) * rstd[:, None]
        out.update(dx=dx.view(shape), dw=torch.einsum("rn,rn->n", dy, xh), db=dy.sum(0))
    return out


def _exact_attn(st):
    case = st["case"]
    B, Sq, Sk, Hq, Hk = (case[n] for n in ("B", "Sq", "Sk", "Hq", "Hk"))
    g, dev = Hq // Hk, st["q"].device
    train = "dout" in st
    shapes = {"out": (B, Sq, Hq, D), "lse": (B, Hq, Sq)}
    if train:
        shapes.update(dq=(B, Sq, Hq, D), dk=(B, Sk, Hk, D), dv=(B, Sk, Hk, D))
    out = {n: torch.zeros(s, dtype=torch.float64, device=dev) for n, s in shapes.items()}
    at_q = torch.arange(Sk - Sq, Sk, device=dev)
    at_k = torch.arange(Sk, device=dev)
    for b in range(B):
        hidden = torch.zeros((Sq, Sk), dtype=torch.bool, device=dev)
        if case["causal"]:
            hidden |= (at_k[None] > at_q[:, None]) & (at_k[None] >= case["prefix"])
        if st["doc"] is not None:
            d = st["doc"][b]
            hidden |= (d[at_q][:, None] != d[None]) | (d[at_q][:, None] < 0)
        for h in range(Hq):
            q, k, v = st["q"][b, :, h].double(), st["k"][b, :, h // g].double(), st["v"][b, :, h // g].double()
            s = torch.mm(q, k.t()) * D ** -0.5
            slope = torch.ones_like(s[:1, :1])
            if case["cap"]:
                slope = 1 / torch.cosh(s / case["cap"]) ** 2
                s = case["cap"] * torch.tanh(s / case["cap"])
            if st["slopes"] is not None:
                s -= st["slopes"][h].double() * (at_q[:, None] - at_k[None]).abs().double()
            s[hidden] = -math.inf
            lse = torch.logsumexp(s, 1)
            p = torch.exp(s - lse.clamp_min(-1e300)[:, None])
            o = p @ v
            out["out"][b, :, h], out["lse"][b, h] = o, lse
            if train:
                do = st["dout"][b, :, h].double()
                dp = torch.mm(do, v.t())
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) * slope * D ** -0.5
                out["dq"][b, :, h] = ds @ k
                out["dk"][b, :, h // g] += ds.t() @ q
                out["dv"][b, :, h // g] += p.t() @ do
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    return _exact_rope(st) if op == "rope" else _exact_norm(st) if op.startswith("norm") else _exact_attn(st)
