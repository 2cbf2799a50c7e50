"""The operators on streams: in order with the torch operations of the current
stream."""

import pytest

from block_sparse_video_geometry_b200 import vsa, workloads as W

import test_gpu_masked as M
import test_gpu_rope as R

pytestmark = pytest.mark.gpu
DELAY = 40_000_000                     # cycles: some 20 ms, far longer than the calls


def late(x, value):
    """x receives `value` on the current stream, behind a delay."""
    import torch
    torch.cuda._sleep(DELAY)
    x.copy_(value)


def test_calls_follow_the_current_stream(cuda_ok):
    """Inside a block of a side stream every call reads what torch wrote on it before, late, and is read by torch
    behind it."""
    import torch
    wl = W.Workload("streams", B=1, H=2, cond=((W.SEG_TEXT, 40),), grid=(4, 8, 8), keep=0.5, seed=3)
    S, H = wl.seq_len, wl.H
    layout = vsa.Layout(wl.segments(), S)
    rope, mask = vsa.make_rope(), vsa.make_mask(causal=True)
    x = [R.draw((1, S, H, 128), "bf16", 50 + i) for i in range(4)]
    w = torch.randn(128, device="cuda")
    gate = torch.rand((1, S, H), device="cuda").bfloat16()
    f32 = lambda *s: torch.zeros(s, device="cuda")                                    # noqa: E731
    fwd = vsa.Forward(layout, vsa.make_params(keep=0.5), 1, H)
    attn = vsa.MaskedAttention(mask, 1, S, S, H, H)
    pos = torch.empty((S, 3), dtype=torch.int32, device="cuda")

    def chain(q, k, v, dout):
        vsa.rope_positions(layout, pos)
        y, dx = torch.empty_like(q), torch.empty_like(q)
        mean, rstd, dw, db = f32(1, S, H), f32(1, S, H), f32(128), f32(128)
        ws = torch.empty(vsa.layer_norm_bwd_workspace_size(q), dtype=torch.uint8, device="cuda")
        vsa.layer_norm_fwd(q, w, None, 1e-6, y, mean, rstd)
        turned, kt = torch.empty_like(y), torch.empty_like(k)
        vsa.rope_fwd(rope, pos, y, k, turned, kt)
        sparse = fwd(turned, kt, v, gate)
        out, lse = attn.forward(turned, kt, v)
        dq, dk, dv = attn.backward(turned, kt, v, out, lse, dout)
        back = torch.empty_like(dq)
        vsa.rope_bwd(rope, pos, dq, None, back, None)
        vsa.layer_norm_bwd(back, q, w, mean, rstd, dx, dw, db, ws)
        return [t * 1 for t in (y, turned, kt, sparse, out, lse, dq, dk, dv, dx, dw, db)]

    want = chain(*x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        given = [torch.zeros_like(t) for t in x]
        for a, b in zip(given, x):
            late(a, b)
        got = chain(*given)
        late(given[0], torch.zeros_like(given[0]))
        for ws in (*attn.ws_fwd.values(), *attn.ws_bwd.values()):
            assert vsa.masked_attn_status(ws) == vsa.OK
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


def test_calls_are_captured_on_the_current_stream(cuda_ok):
    """Without a stream of their own the calls go into the graph that torch is capturing."""
    import torch
    q, k, v, dout = M.tensors(1, 200, 200, 2, 2, seed=51)
    attn = vsa.MaskedAttention(vsa.make_mask(causal=True), 1, 200, 200, 2, 2)
    out, lse = attn.forward(q, k, v)
    grads = attn.backward(q, k, v, out, lse, dout)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.forward(q, k, v, out, lse)
        attn.backward(q, k, v, out, lse, dout, *grads)
    for a, b in zip((q, k, v, dout), M.tensors(1, 200, 200, 2, 2, seed=52)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    want = M.run(q, k, v, causal=True, dout=dout)
    assert all(torch.equal(a, b) for a, b in zip((out, lse, *grads), want))
    del graph
