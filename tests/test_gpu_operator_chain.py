"""The operators around the sparse call as they are used together: layer norm of
the query and key heads, three-axis rotation by the layout's positions, sparse
attention (or, for what it refuses, dense attention over the same tensors), and
the gradients back through all of them.

Every call is compared with its formula in 64 bits on the tensors that the call
before it left, with the tolerances of that call's own tests."""

import numpy as np
import pytest

from block_sparse_video_geometry_b200 import vsa, workloads as W
from oracle import vsa_oracle as O

import test_gpu_masked as M
import test_gpu_norm as N
import test_gpu_rope as R
import vsa_cases as C
from test_gpu_backward import check_grad, oracle_grads

pytestmark = pytest.mark.gpu
WL = W.Workload("chain", B=1, H=2, cond=((W.SEG_TEXT, 40), (W.SEG_REF_IMAGE, 33)), grid=(6, 8, 9), keep=0.4, seed=31)


def bits(t):
    return t.contiguous().view(__import__("torch").int16).cpu().numpy().view(np.uint16)


@pytest.fixture(scope="module")
def chain():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    wl, dev = WL, torch.device("cuda:0")
    S, H = wl.seq_len, wl.H
    g = torch.Generator(device=dev).manual_seed(5)
    n = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    qkv = (n(1, S, 3, H, 128) * 2 + 0.3).bfloat16()             # a fused projection
    c = {"x": [qkv[:, :, i] for i in range(2)], "v": qkv[:, :, 2].contiguous(),
         "w": [1 + 0.2 * n(128) for _ in range(2)], "g": torch.rand((1, S, H), generator=g, device=dev).bfloat16()}
    layout = vsa.Layout(wl.segments(), S)
    pos = torch.empty((S, 3), dtype=torch.int32, device=dev)
    vsa.rope_positions(layout, pos)
    rope = vsa.make_rope((44, 42, 42), pairing=vsa.ROPE_HALVES)
    c["normed"], c["stats"] = [], []
    for x, w in zip(c["x"], c["w"]):
        y = torch.empty((1, S, H, 128), dtype=torch.bfloat16, device=dev)
        mean, rstd = (torch.empty((1, S, H), device=dev) for _ in range(2))
        vsa.layer_norm_fwd(x, w, None, 1e-6, y, mean, rstd)
        c["normed"].append(y)
        c["stats"].append((mean, rstd))
    c["turned"] = [torch.empty_like(y) for y in c["normed"]]
    vsa.rope_fwd(rope, pos, *c["normed"], *c["turned"])
    c["dout"] = n(1, S, H, 128).bfloat16()
    c.update(layout=layout, pos=pos, rope=rope)
    return c


def back_through(c, grads):
    """The gradients of q and k taken back through the rotation and the norm, each checked."""
    import torch
    S, H = WL.seq_len, WL.H
    for i, dt in enumerate(grads):
        dn = torch.empty((1, S, H, 128), device="cuda")
        vsa.rope_bwd(c["rope"], c["pos"], dt, None, dn, None)
        R.check(dn, *R.reference(dt, c["pos"], (44, 42, 42), vsa.ROPE_HALVES, sign=-1.0))
        dx = torch.empty((1, S, H, 128), dtype=torch.bfloat16, device="cuda")
        dw, db = torch.empty(128, device="cuda"), torch.empty(128, device="cuda")
        ws = torch.empty(vsa.layer_norm_bwd_workspace_size(c["x"][i]), dtype=torch.uint8, device="cuda")
        vsa.layer_norm_bwd(dn, c["x"][i], c["w"][i], *c["stats"][i], dx, dw, db, ws)
        N.check_step(c["x"][i].contiguous(), c["w"][i], None, dn, (c["normed"][i], *c["stats"][i], dx, dw, db))


def test_norm_and_rotation(chain):
    for i in range(2):
        ref = N.Reference(chain["x"][i].contiguous(), chain["w"][i], None, 1e-6)
        N.within(chain["normed"][i], ref.y, ref.tol_y(chain["normed"][i].dtype), "normed")
        R.check(chain["turned"][i], *R.reference(chain["normed"][i], chain["pos"], (44, 42, 42), vsa.ROPE_HALVES))


def test_sparse_attention_and_its_gradients(chain):
    import torch
    q, k, v, g, dout = *chain["turned"], chain["v"], chain["g"], chain["dout"]
    lay = C.oracle_layout(WL)
    prm = C.params_of(WL)
    p = vsa.make_params(**prm)
    fwd = vsa.Forward(chain["layout"], p, 1, WL.H)
    out = fwd(q, k, v, g)
    assert vsa.sparse_attn_status(fwd.ws_attn) == vsa.OK
    grads = [torch.empty(q.shape, device="cuda") for _ in range(3)]
    dg = torch.empty(g.shape, device="cuda")
    ws = torch.empty(chain["layout"].sparse_attn_bwd_workspace_size(1, WL.H, p), dtype=torch.uint8, device="cuda")
    vsa.sparse_attn_bwd(chain["layout"], p, q, k, v, g, fwd.idx, fwd.cnt, fwd.kmax, fwd.o_coarse, dout, *grads, dg, ws)
    assert vsa.sparse_attn_bwd_status(ws) == vsa.OK
    host = [bits(t) for t in (q, k, v, g)]
    res = dict(out=out.cpu().numpy())
    idx, cnt = fwd.idx.cpu().numpy(), fwd.cnt.cpu().numpy()
    f = O.bf16_bits_to_f64
    for h in range(WL.H):
        ho = C.HeadOracle(WL, lay, host, 0, h, prm)
        near = C.compare_selection(ho, idx[0, h], cnt[0, h])
        C.note_near_ties(len(near))
        C.compare_outputs(ho, res, 0, h, range(chain["layout"].info.n_tiles), near_tie=near)
        sel = [near.get(qt, s) for qt, s in enumerate(ho.sel)]
        want = oracle_grads(*(f(x[0, :, h]) for x in host), f(bits(dout)[0, :, h]), lay, ho.p, sel)
        for name, got, w in zip(("dq", "dk", "dv", "dg"), (*grads, dg), want):
            check_grad(got[0, :, h].cpu().numpy(), w, "%s h%d" % (name, h))
    back_through(chain, grads[:2])


def test_dense_attention_and_its_gradients(chain):
    """The same tensors through the dense call, conditioning and video as two documents with a capped score, its
    bf16 gradients back through the same rotation and norm."""
    import torch
    q, k, v, dout = *chain["turned"], chain["v"], chain["dout"]
    S = WL.seq_len
    ids = (torch.arange(S, device="cuda")[None] >= 73).to(torch.int32)
    attn = vsa.MaskedAttention(vsa.make_mask(softcap=30.0), 1, S, S, WL.H, WL.H)
    terms = dict(doc_q=ids, doc_k=ids)
    out, lse = attn.forward(q, k, v, **terms)
    dq, dk, dv = attn.backward(q, k, v, out, lse, dout, **terms)
    ref = M.Reference(q, k, v, M.visible(1, S, S, False, None, ids, ids), 30.0, dout=dout)
    for name, got in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        M.within(got, getattr(ref, name), getattr(ref, "t_" + name), name)
    back_through(chain, [dq, dk])


def test_full_keep_sparse_equals_dense(chain):
    """The sparse call that keeps every tile, its gate at 0, and the dense call answer the same question: each within
    its own bound of the formula, so within their sum of each other (the sparse call's is 2e-2)."""
    import torch
    q, k, v = *chain["turned"], chain["v"]
    S = WL.seq_len
    fwd = vsa.Forward(chain["layout"], vsa.make_params(keep=1.0), 1, WL.H)
    sparse = fwd(q, k, v, torch.zeros_like(chain["g"]))
    attn = vsa.MaskedAttention(vsa.make_mask(), 1, S, S, WL.H, WL.H)
    dense, _ = attn.forward(q, k, v)
    ref = M.Reference(q, k, v, M.visible(1, S, S))
    assert ((dense.double() - sparse.double()).abs() - ref.t_out).max().item() <= C.OUT_MAX_ABS
