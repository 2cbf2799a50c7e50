"""The operators on streams: in order with the torch operations of the current
stream, and memory that their calls allocate on another one."""

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


def test_allocating_calls_on_another_stream(cuda_ok):
    """Memory that was freed on the current stream, whose queued work still reads it, is not what a call on another
    stream writes; nor does that stream's next call get the outputs that the current stream still reads."""
    import torch
    shape = (1, 300, 300, 4, 2)
    q, k, v, dout = M.tensors(*shape, seed=53)
    want = M.run(q, k, v, causal=True, dout=dout)
    side = torch.cuda.Stream()
    attn = vsa.MaskedAttention(vsa.make_mask(causal=True), *shape)
    torch.cuda.synchronize()
    for _ in range(3):
        pending = [torch.full_like(t, 7) for t in want for _ in range(4)]
        torch.cuda._sleep(DELAY)
        seen = [t.clone() for t in pending]
        del pending                                                  # free on the current stream, read late
        out, lse = attn.forward(q, k, v, stream=side)
        grads = attn.backward(q, k, v, out, lse, dout, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(DELAY)
        mine = [t.clone() for t in (out, lse, *grads)]
        del out, lse, grads                                          # read late by the current stream
        attn.forward(k.repeat(1, 1, 2, 1), k, k, stream=side)        # other outputs of the same sizes
        torch.cuda.synchronize()
        assert all(bool((t == 7).all()) for t in seen)
        assert all(torch.equal(a, b) for a, b in zip(mine, want))


def test_one_workspace_on_several_streams(cuda_ok):
    """An object used on one stream after another, each waiting for the one before, and dropped while the last still
    runs."""
    import torch
    shape = (1, 300, 300, 4, 2)
    q, k, v, dout = M.tensors(*shape, seed=54)
    want = M.run(q, k, v, causal=True, dout=dout)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(3):
        attn = vsa.MaskedAttention(vsa.make_mask(causal=True), *shape)
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                if i:
                    s.wait_stream(streams[i - 1])
                torch.cuda._sleep(DELAY // 4)
                out, lse = attn.forward(q, k, v)
                grads = attn.backward(q, k, v, out, lse, dout)
        sizes = [ws.numel() for ws in (*attn.ws_fwd.values(), *attn.ws_bwd.values())]
        del attn
        with torch.cuda.stream(streams[0]):                          # whose memory the workspaces were
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, lse, *grads), want))
        del junk
