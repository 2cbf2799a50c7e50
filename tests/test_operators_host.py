"""Refusals of the operators around the sparse call, without a GPU: malformed
arguments return a status before any GPU work (the pointers here are never
followed)."""

import contextlib
import ctypes

import pytest

from block_sparse_video_geometry_b200 import vsa

FAKE = 1 << 20          # aligned, never dereferenced


def view(heads=2, dtype=vsa.DTYPE_BF16, data=FAKE, sb=1 << 14, ss=256, sh=128):
    return vsa.view_bytes(data or 0, sb, ss, sh, heads, dtype)


def rope_call(rope=None, B=2, S=8, pos=FAKE, pos_sb=24, q=None, k=None, qo=None, ko=None, name="vsa_rope_fwd"):
    rope = vsa.make_rope() if rope is None else rope
    return getattr(vsa.lib(), name)(ctypes.byref(rope), B, S, pos, pos_sb, q or view(), k, qo or view(), ko, None)


@pytest.mark.parametrize("rope", [
    vsa.make_rope((43, 42, 42)), vsa.make_rope((-2, 64, 64)), vsa.make_rope((64, 64, 2)), vsa.make_rope(theta=0.0),
    vsa.make_rope(theta=-1.0), vsa.make_rope(theta=float("inf")), vsa.make_rope(theta=float("nan")),
    vsa.make_rope(scale=(1.0, float("nan"), 1.0)), vsa.make_rope(pairing=2),
    vsa.make_rope((126, 0, 0), theta=1e-320, scale=(1e300, 1.0, 1.0)),
])
def test_rope_refuses_malformed_parameters(rope):
    assert rope_call(rope) == vsa.ERR_INVALID_ARG
    assert rope_call(rope, name="vsa_rope_bwd") == vsa.ERR_INVALID_ARG


def test_rope_refuses_malformed_arguments():
    bad = vsa.ERR_INVALID_ARG
    assert rope_call(B=-1) == bad and rope_call(S=-1) == bad and rope_call(pos=None) == bad
    assert rope_call(pos_sb=23) == bad and rope_call(pos_sb=-24) == bad and rope_call(pos=FAKE + 2) == bad
    assert rope_call(k=view()) == bad and rope_call(ko=view()) == bad            # k without its output and back
    assert rope_call(q=view(heads=3)) == bad and rope_call(q=view(heads=0)) == bad
    for v in (view(dtype=3), view(dtype=-1), view(data=None), view(data=FAKE + 8), view(ss=-256), view(ss=252)):
        assert rope_call(q=v) == bad and rope_call(qo=v) == bad
    for v in (view(sb=0), view(ss=0), view(sh=64)):                               # overlapping output rows
        assert rope_call(qo=v) == bad
    assert rope_call(S=1 << 31, pos_sb=0) == vsa.ERR_UNSUPPORTED
    assert rope_call(q=view(heads=5000), qo=view(heads=5000)) == vsa.ERR_UNSUPPORTED
    assert rope_call(S=0) == vsa.OK and rope_call(B=0, pos=None) == vsa.OK         # nothing to do
    L = vsa.lib()
    lay = vsa.Layout([(vsa.SEG_VIDEO, 0, 8, (2, 2, 2))], 8)
    assert L.vsa_rope_positions(None, 0, 0, 0, FAKE, None) == bad
    assert L.vsa_rope_positions(lay.handle, 0, 0, 0, None, None) == bad


def norm_fwd(B=2, S=8, width=64, x=None, w=FAKE, b=FAKE, wt=vsa.DTYPE_F32, eps=1e-6, y=None, mean=FAKE, rstd=FAKE):
    x, y = x or view(), y or view()
    return vsa.lib().vsa_layer_norm_fwd(B, S, width, x, w, b, wt, eps, y, mean, rstd, None)


def norm_bwd(B=2, S=8, width=64, dy=None, x=None, w=FAKE, wt=vsa.DTYPE_F32, mean=FAKE, rstd=FAKE, dx=None, dw=FAKE,
             db=FAKE, ws=FAKE, nbytes=1 << 30):
    dy, x, dx = dy or view(), x or view(), dx or view()
    return vsa.lib().vsa_layer_norm_bwd(B, S, width, dy, x, w, wt, mean, rstd, dx, dw, db, ws, nbytes, None)


def test_layer_norm_refuses_malformed_arguments():
    bad = vsa.ERR_INVALID_ARG
    for call in (norm_fwd, norm_bwd):
        assert call(B=-1) == bad and call(S=-1) == bad and call(width=0) == bad and call(width=-4) == bad
        assert call(width=vsa.MAX_NORM_WIDTH + 1) == vsa.ERR_UNSUPPORTED
        assert call(S=1 << 31) == vsa.ERR_UNSUPPORTED and call(S=1 << 29) == vsa.ERR_UNSUPPORTED
        assert call(wt=vsa.DTYPE_F16) == bad and call(wt=7) == bad and call(w=FAKE + 2) == bad
        for v in (view(heads=0), view(heads=3), view(dtype=5), view(data=None), view(data=FAKE + 1), view(sb=-1)):
            assert call(x=v) == bad
    for v in (view(dtype=vsa.DTYPE_F32), view(heads=1), view(ss=0), view(sh=63)):
        assert norm_fwd(y=v) == bad
    assert norm_fwd(eps=-1e-6) == bad and norm_fwd(eps=float("nan")) == bad and norm_fwd(eps=float("inf")) == bad
    assert norm_fwd(mean=None) == bad and norm_fwd(rstd=None) == bad and norm_fwd(rstd=FAKE + 1) == bad
    for v in (view(dtype=vsa.DTYPE_F16), view(heads=1)):
        assert norm_bwd(dy=v) == bad and norm_bwd(dx=v) == bad
    assert norm_bwd(mean=None) == bad and norm_bwd(rstd=None) == bad and norm_bwd(dw=FAKE + 2) == bad
    assert norm_bwd(ws=None) == bad and norm_bwd(ws=FAKE + 128) == bad
    n = ctypes.c_size_t()
    assert vsa.lib().vsa_layer_norm_bwd_workspace_size(2, 8, 2, 64, ctypes.byref(n)) == vsa.OK and n.value >= 512
    assert norm_bwd(nbytes=n.value - 1) == vsa.ERR_WORKSPACE_TOO_SMALL
    assert vsa.lib().vsa_layer_norm_bwd_workspace_size(2, 8, 0, 64, ctypes.byref(n)) == bad
    assert vsa.lib().vsa_layer_norm_bwd_workspace_size(2, 8, 2, 64, None) == bad
    assert norm_fwd(S=0) == vsa.OK


def test_binding_refuses_what_it_cannot_pass_on():
    import torch
    cpu = torch.zeros((1, 4, 2, 128))
    pos = torch.zeros((4, 3), dtype=torch.int32)
    rope = vsa.make_rope()
    with pytest.raises(ValueError, match="CUDA device"):
        vsa.rope_fwd(rope, pos, cpu, None, cpu.clone(), None)
    with pytest.raises(ValueError, match="128"):
        vsa.rope_fwd(rope, pos, cpu[..., :64], None, cpu[..., :64], None)
    with pytest.raises(ValueError, match="pos"):
        vsa.rope_fwd(rope, pos.long(), cpu, None, cpu, None)
    with pytest.raises(ValueError, match="pos"):
        vsa.rope_fwd(rope, pos[:3], cpu, None, cpu, None)
    with pytest.raises(ValueError, match="together"):
        vsa.rope_fwd(rope, pos, cpu, cpu, cpu, None)
    with pytest.raises(ValueError, match="dims"):
        vsa.make_rope((64, 64))
    x = torch.zeros((4, 128))
    with pytest.raises(ValueError, match="CUDA device"):
        vsa.layer_norm_fwd(x, None, None, 1e-6, x.clone())
    with pytest.raises(ValueError, match="shape"):
        vsa.layer_norm_fwd(x, None, None, 1e-6, x[:2])
    with pytest.raises(ValueError, match="one type"):
        vsa.layer_norm_fwd(x, torch.zeros(128), torch.zeros(128).half(), 1e-6, x.clone())
    with pytest.raises(ValueError, match=r"\[S, width\]"):
        vsa.layer_norm_fwd(x[0], None, None, 1e-6, x[0])


def attn_call(name="fwd", mask=None, B=1, Sq=8, Sk=8, q=None, k=None, v=None, out=None, lse=FAKE, dout=None, dq=None,
              dk=None, dv=None, ws=FAKE, nbytes=1 << 40, **terms):
    t = vsa.MaskTerms(**terms)
    mask = mask if mask is not None else vsa.make_mask()
    q, k, v, out, dout, dq, dk, dv = (x or view() for x in (q, k, v, out, dout, dq, dk, dv))
    L = vsa.lib()
    if name == "fwd":
        return L.vsa_masked_attn_fwd(ctypes.byref(mask), ctypes.byref(t), B, Sq, Sk, q, k, v, out, lse, ws, nbytes, None)
    return L.vsa_masked_attn_bwd(ctypes.byref(mask), ctypes.byref(t), B, Sq, Sk, q, k, v, out, lse, dout, dq, dk, dv, ws,
                                 nbytes, None)


@pytest.mark.parametrize("name", ["fwd", "bwd"])
def test_masked_attention_refuses_malformed_arguments(name):
    bad, no = vsa.ERR_INVALID_ARG, vsa.ERR_UNSUPPORTED
    call = lambda **kw: attn_call(name, **kw)  # noqa: E731
    for m in (vsa.Mask(2, 0, 0.0, 0.0), vsa.Mask(0, 2, 0.0, 0.0), vsa.make_mask(scale=float("nan")),
              vsa.make_mask(softcap=-1.0), vsa.make_mask(softcap=float("inf"))):
        assert call(mask=m) == bad
    assert call(B=-1) == bad and call(Sq=-1) == bad and call(Sk=-1) == bad
    assert call(q=view(heads=3)) == bad and call(k=view(heads=0)) == bad       # 3 is no multiple of 2
    assert call(v=view(heads=1)) == bad and call(out=view(heads=4)) == bad
    for v in (view(dtype=vsa.DTYPE_F16), view(dtype=vsa.DTYPE_F32), view(data=None), view(data=FAKE + 8), view(ss=252),
              view(ss=-256)):
        assert call(q=v) == bad and call(k=v) == bad and call(v=v) == bad and call(out=v) == bad
    assert call(lse=FAKE + 2) == bad and call(ws=None) == bad and call(ws=FAKE + 128) == bad
    assert call(q=view(ss=0)) == no and call(v=view(ss=0)) == no
    assert call(Sk=(1 << 24) + 1) == no and call(B=70000) == no
    assert call(k=view(ss=1 << 40)) == no
    # documents: both or neither, as the mask says; a prefix needs a causal mask
    doc = vsa.make_mask(documents=True)
    assert call(mask=doc) == bad and call(mask=doc, doc_q=FAKE) == bad and call(doc_q=FAKE, doc_k=FAKE) == bad
    assert call(mask=doc, doc_q=FAKE, doc_k=FAKE + 2) == bad
    assert call(prefix=FAKE) == bad and call(slopes=FAKE + 1) == bad
    n = ctypes.c_size_t()
    size = getattr(vsa.lib(), "vsa_masked_attn_%sworkspace_size" % ("bwd_" if name == "bwd" else ""))
    causal = vsa.make_mask(causal=True)
    assert size(ctypes.byref(causal), 1, 8, 8, 2, 2, ctypes.byref(n)) == vsa.OK and n.value > 256
    assert call(mask=causal, nbytes=n.value - 1) == vsa.ERR_WORKSPACE_TOO_SMALL
    assert size(None, 1, 8, 8, 2, 2, ctypes.byref(n)) == bad and size(ctypes.byref(causal), 1, 8, 8, 2, 2, None) == bad
    assert size(ctypes.byref(causal), 1, 8, 8, 3, 2, ctypes.byref(n)) == bad
    assert vsa.lib().vsa_masked_attn_status(None, None) == bad
    if name == "bwd":
        for x in (view(sb=0), view(ss=0), view(sh=64), view(heads=1)):
            assert call(dk=x, B=2) == bad and call(dq=x, B=2) == bad and call(dv=x, B=2) == bad
        assert call(dout=view(heads=1)) == bad
    else:
        assert call(out=view(ss=0)) == bad and call(out=view(sh=64)) == bad


def test_masked_attention_binding_refusals():
    import torch
    mask = vsa.make_mask()
    q = torch.zeros((1, 8, 4, 128)).bfloat16()
    k = torch.zeros((1, 9, 2, 128)).bfloat16()
    lse = torch.zeros((1, 4, 8))
    ws = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA device"):
        vsa.masked_attn_fwd(mask, q, k, k, q.clone(), lse, ws)
    with pytest.raises(ValueError, match="multiple"):
        vsa.masked_attn_fwd(mask, q[:, :, :3], k, k, q, lse, ws)
    with pytest.raises(ValueError, match="lse"):
        vsa.masked_attn_fwd(mask, q, k, k, q.clone(), lse[:, :2], ws)
    ids = torch.zeros((1, 9), dtype=torch.int32)
    with pytest.raises(ValueError, match="come together"):
        vsa.masked_attn_fwd(mask, q, k, k, q.clone(), lse, ws, doc_q=ids[:, :8], doc_k=ids)
    with pytest.raises(ValueError, match="doc_q"):
        vsa.masked_attn_fwd(vsa.make_mask(documents=True), q, k, k, q.clone(), lse, ws, doc_q=ids, doc_k=ids)
    with pytest.raises(ValueError, match="slopes"):
        vsa.masked_attn_fwd(mask, q, k, k, q.clone(), lse, ws, slopes=torch.zeros(3))
    with pytest.raises(vsa.VSAError):
        vsa.MaskedAttention(mask, 1, 8, 8, 3, 2)
    attn = vsa.MaskedAttention(mask, 1, 8, 8, 4, 2)
    with pytest.raises(ValueError, match="made for"):
        attn.forward(q, k, k)


@pytest.mark.parametrize("name", ["rope_fwd", "rope_bwd"])
def test_positions_at_foreign_strides_are_refused(name):
    """One token's positions read at strides that the tensor does not have would be other tokens' (or lie behind it):
    refused like those of several tokens. Views whose last two dimensions are contiguous reach the device check."""
    import torch
    call = getattr(vsa, name)
    table = torch.arange(3 * 10, dtype=torch.int32).view(3, 10)          # axis-major
    tables = table.expand(2, 3, 10).contiguous()
    wide = torch.zeros((5, 6), dtype=torch.int32)
    x = lambda B, S: torch.zeros((B, S, 2, 128))                          # noqa: E731
    for pos, B in ((table[:, 4:5].t(), 1), (table[0, 4:5].expand(1, 3), 1), (wide[:1, ::2], 1),
                   (tables[:, :, 4:5].transpose(1, 2), 2), (tables[:1, :, 4:5].transpose(1, 2), 1),
                   (table[0, 4:5].expand(2, 1, 3), 2)):
        with pytest.raises(ValueError, match="pos must"):
            call(vsa.make_rope(), pos, x(B, 1), None, x(B, 1), None)
    for pos, B, S in ((table.t(), 1, 10), (wide[:4, :3], 1, 4), (tables.transpose(1, 2), 2, 10)):
        with pytest.raises(ValueError, match="pos must"):
            call(vsa.make_rope(), pos, x(B, S), None, x(B, S), None)
    rows = torch.zeros((2, 10, 3), dtype=torch.int32)
    for pos, B, S in ((rows[0, 4:5], 1, 1), (rows[:, 4:5], 2, 1), (rows[:1, 4:5], 1, 1), (rows[0, 4].expand(2, 1, 3), 2, 1),
                      (wide[2:3, :3], 1, 1), (wide[2:3, 1:4].t().t(), 1, 1), (rows[:, 2:9], 2, 7), (rows[:, :0], 2, 0)):
        with pytest.raises(ValueError, match="CUDA device"):
            call(vsa.make_rope(), pos, x(B, S), None, x(B, S), None)


@pytest.fixture
def fake_cuda(monkeypatch):
    """Tensors that say they are on cuda:1 while cuda:0 is current, torch streams that are numbers, and a library that
    notes the stream (its last argument) of each call."""
    import torch

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream = handle

    class Fake(torch.Tensor):
        device = torch.device("cuda", 1)
        kept = ()

        def get_device(self):
            return 1

        def record_stream(self, s):
            self.kept = (*self.kept, s.cuda_stream)

    class Library:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: setattr(a[-1]._obj, "value", 1024) or vsa.OK
            return lambda *a: calls.append((name, a[-1], here[-1])) or vsa.OK

    calls, here, memory = [], ["cuda:0"], []
    current = {None: Stream(70), 0: Stream(70), 1: Stream(71)}
    state = {"stream": None}

    @contextlib.contextmanager
    def on_device(index):
        here.append("cuda:%d" % getattr(index, "index", index))
        yield
        here.pop()

    @contextlib.contextmanager
    def on_stream(s):
        before, state["stream"] = state["stream"], s
        yield
        state["stream"] = before

    def current_stream(device=None):
        return state["stream"] or current[getattr(device, "index", device)]

    make = torch.empty

    def empty(shape, dtype=None, device=None):
        memory.append(current_stream(device).cuda_stream)
        return make(shape, dtype=dtype).as_subclass(Fake)

    for name, x in (("current_device", lambda: 0), ("current_stream", current_stream), ("is_initialized", lambda: True),
                    ("device", on_device), ("stream", on_stream), ("ExternalStream", Stream),
                    ("default_stream", lambda device=None: Stream(0))):
        monkeypatch.setattr(torch.cuda, name, x)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: current_stream(i).cuda_stream)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(vsa, "lib", Library)
    tensor = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype).as_subclass(Fake)   # noqa: E731
    return tensor, calls, memory, on_stream, Stream


def test_none_is_the_current_stream_of_the_tensors_device(fake_cuda):
    """Every call stands in order with the torch operations around it: on the current stream of its tensors' device,
    with that device current; on a given stream otherwise."""
    import torch
    tensor, calls, _, on_stream, Stream = fake_cuda
    q, x, f = tensor(1, 4, 2, 128), tensor(4, 64), tensor(4, dtype=torch.float32)
    pos, ws = tensor(4, 3, dtype=torch.int32), tensor(1024, dtype=torch.uint8)
    w = tensor(64, dtype=torch.float32)
    lse, mask = tensor(1, 2, 4, dtype=torch.float32), vsa.make_mask()
    attn = vsa.MaskedAttention(mask, 1, 4, 4, 2, 2)
    layout = type("L", (), {"info": type("I", (), {"seq_len": 4}), "handle": 0})
    every = [lambda **kw: vsa.rope_positions(layout, pos, **kw),
             lambda **kw: vsa.rope_fwd(vsa.make_rope(), pos, q, q, q, q, **kw),
             lambda **kw: vsa.rope_bwd(vsa.make_rope(), pos, q, None, q, None, **kw),
             lambda **kw: vsa.layer_norm_fwd(x, w, None, 1e-6, x, f, f, **kw),
             lambda **kw: vsa.layer_norm_bwd(x, x, w, f, f, x, w, w, ws, **kw),
             lambda **kw: vsa.masked_attn_fwd(mask, q, q, q, q, lse, ws, **kw),
             lambda **kw: vsa.masked_attn_bwd(mask, q, q, q, q, lse, q, q, q, q, ws, **kw),
             lambda **kw: vsa.masked_attn_status(ws, **kw),
             lambda **kw: attn.forward(q, q, q, q, lse, **kw),
             lambda **kw: attn.backward(q, q, q, q, lse, q, q, q, q, **kw)]
    for call in every:
        for kw, side, want in (({}, None, 71), ({}, Stream(5), 5), (dict(stream=Stream(9)), None, 9),
                               (dict(stream=9), Stream(5), 9), (dict(stream=0), None, 0)):
            calls.clear()
            with on_stream(side) if side else contextlib.nullcontext():
                call(**kw)
            assert [c[1:] for c in calls] == [(want, "cuda:1")], (calls, kw)


def test_older_calls_take_the_current_stream_too(fake_cuda):
    """The sparse calls beside them, on the same stream without being given one."""
    import torch
    tensor, calls, _, on_stream, Stream = fake_cuda
    q, g, i = tensor(1, 64, 2, 128), tensor(1, 64, 2), tensor(1, 2, 1, 1, dtype=torch.int32)
    layout = type("L", (), {"handle": 0})
    for side, want in ((None, 70), (Stream(5), 5)):
        calls.clear()
        with on_stream(side) if side else contextlib.nullcontext():
            vsa.coarse_select(layout, vsa.make_params(), q, q, q, i, i, g, g)
            vsa.coarse_select_status(g)
        assert [c[1] for c in calls] == [want, want]
    assert vsa._stream_handle(0) == 0


def test_tensors_that_a_call_allocates_belong_to_its_stream(fake_cuda):
    """Outputs and workspaces of a call on a side stream come out of that stream's memory and stay while the caller's
    stream uses them; a workspace stays for every stream that has used it."""
    import torch
    tensor, calls, memory, on_stream, Stream = fake_cuda
    q, lse = tensor(1, 4, 2, 128), tensor(1, 2, 4, dtype=torch.float32)
    attn = vsa.MaskedAttention(vsa.make_mask(), 1, 4, 4, 2, 2)
    outs = attn.forward(q, q, q, stream=Stream(9)) + attn.backward(q, q, q, q, lse, q, stream=Stream(9))
    assert memory == [9] * 7 and all(t.kept == (71,) for t in outs)          # five outputs, two workspaces
    memory.clear()
    ws = attn.ws_fwd[0]
    attn.forward(q, q, q, q, lse, stream=9)
    attn.forward(q, q, q, q, lse)
    attn.forward(q, q, q, q, lse)
    assert not memory and ws.kept == (71, 71)              # as allocated for another stream, and once as used on this
    with on_stream(Stream(5)):
        out, _ = attn.forward(q, q, q)
    assert memory == [5, 5] and out.kept == () and ws.kept == (71, 71, 5)
    with pytest.raises(ValueError, match="made for device"):
        vsa.MaskedAttention(vsa.make_mask(), 1, 4, 4, 2, 2, device="cuda:0").forward(q, q, q)


def test_status_of_an_attention_object(fake_cuda, monkeypatch):
    """The first error among the workspaces of its calls."""
    tensor, calls, _, _, _ = fake_cuda
    import torch
    q, lse = tensor(1, 4, 2, 128), tensor(1, 2, 4, dtype=torch.float32)
    attn = vsa.MaskedAttention(vsa.make_mask(), 1, 4, 4, 2, 2)
    assert attn.status() == vsa.OK                         # nothing ran
    attn.forward(q, q, q, q, lse)
    attn.backward(q, q, q, q, lse, q, q, q, q)
    calls.clear()
    assert attn.status(stream=9) == vsa.OK and calls == [("vsa_masked_attn_status", 9, "cuda:1")] * 2
    monkeypatch.setattr(vsa, "masked_attn_status",
                        lambda ws, stream=None: vsa.ERR_TIMEOUT if ws is attn.ws_bwd[0] else vsa.OK)
    assert attn.status() == vsa.ERR_TIMEOUT


@pytest.mark.parametrize("rows,width,blocks", [(17408, 5120, 320), (148, 16384, 148), (100000, 16384, 160), (40, 16384, 40),
                                               (3693, 1153, 640), (1 << 20, 128, 640), (300, 128, 38), (1, 1, 1),
                                               (1 << 20, 2048, 800), (100, 2048, 100)])
def test_layer_norm_workspace_holds_the_blocks_that_run(rows, width, blocks):
    """A partial row of two sums for each block that can run: on 160 SMs, as many blocks per SM as make 640 threads
    (long rows) or 1024 (short ones, 8 rows or more a block), and no more blocks than rows."""
    n = ctypes.c_size_t()
    assert vsa.lib().vsa_layer_norm_bwd_workspace_size(1, rows, 1, width, ctypes.byref(n)) == vsa.OK
    assert n.value == (blocks * 2 * width * 4 + 255) // 256 * 256
