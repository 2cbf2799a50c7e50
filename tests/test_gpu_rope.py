"""Three-axis rotary positions (vsa_rope_fwd, vsa_rope_bwd, vsa_rope_positions)
against the formula in 64 bits.

Tolerance per element of a pair (a, b). The angle is formed in 64 bits on both
sides: the kernel's rate (a power within one step, a product, a quotient by a
rounded 2 pi) and its product with the position are off by at most 6 * 2^-53 of
the angle, the reference's (a power, two products) by at most 4 * 2^-53, so the
two differ by up to 10 * 2^-53 |angle| (7 * 10^-6 at the end of the 32-bit
positions with a scale of 3, where 2^31 * 3 radians leave no more bits; 10^-9 at
10^6). The rounding of the fraction of a turn to 32 bits, at most 2^-25 for a value up to
1/2, is an angle error of 2 pi 2^-25 < 3.2 * 2^-24; the sine and cosine are
within 4 * 2^-24 of their argument's (2 ulp of a value up to 1); the two
products and their sum round three times. So the rotation is off by at most
(3.2 + 4 + 3) 2^-24 < 11 * 2^-24, and the angle's share, times (|a| + |b|), and the stored result by half
a step of its type more (fp16 below 2^-14: 2^-25).
"""

import math

import pytest

from block_sparse_video_geometry_b200 import vsa

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def types():
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def reference(x, pos, dims, pairing, theta=10000.0, scale=(1.0, 1.0, 1.0), sign=1.0):
    """x [B, S, H, 128] and pos [S, 3] or [B, S, 3] -> rotated x in float64 and the bound of the rotation per element."""
    import torch
    x = x.double()
    y, size = x.clone(), 0.0 * torch.nan_to_num(x)
    p = pos.double() if pos.dim() == 3 else pos.double()[None]
    at = 0
    for ax, d in enumerate(dims):
        for i in range(d // 2):
            a, b = (at + 2 * i, at + 2 * i + 1) if pairing == vsa.ROPE_ADJACENT else (at + i, at + i + d // 2)
            ang = (sign * p[..., ax] * scale[ax] * theta ** (-2.0 * i / d))[..., None]
            c, s = torch.cos(ang), torch.sin(ang)
            y[..., a] = x[..., a] * c - x[..., b] * s
            y[..., b] = x[..., a] * s + x[..., b] * c
            size[..., a] = size[..., b] = (11 * U + 10 * 2.0 ** -53 * ang.abs()) * (x[..., a].abs() + x[..., b].abs())
        at += d
    return y, size


def check(got, want, size):
    import torch
    half_step = torch.finfo(got.dtype).eps / 2
    tol = size + (want.abs() + size) * half_step
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (got.double() - want).abs()
    worst = (err - tol).max().item()
    assert worst <= 0, "beyond its bound by %.3g (error %.3g)" % (worst, err.max().item())


def draw(shape, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (3 * torch.randn(shape, generator=g, device="cuda")).to(types()[dtype])


CASES = [
    # B, S, Hq, Hk, dims, pairing, in, out, far, per-batch positions
    (1, 1, 1, 1, (44, 42, 42), 0, "bf16", "bf16", 0, False),
    (3, 1, 24, 8, (44, 42, 42), 1, "bf16", "bf16", 900000, True),
    (2, 67, 3, 1, (16, 56, 56), 1, "f32", "bf16", 0, True),
    (2, 67, 3, 1, (16, 56, 56), 0, "f32", "f32", 2 ** 31 - 200, False),
    (1, 515, 5, 5, (32, 32, 32), 1, "f16", "f16", 10 ** 6, False),
    (1, 515, 5, 5, (2, 62, 60), 1, "f16", "f32", -2 ** 31, False),
    (1, 130, 7, 2, (0, 64, 64), 0, "bf16", "f16", 4096, False),
    (2, 2100, 2, 1, (128, 0, 0), 1, "bf16", "bf16", 31, True),      # several tokens per block, the last one partial
    (1, 4099, 1, 3, (6, 0, 2), 0, "f32", "bf16", 5, False),
    (1, 33, 2, 2, (0, 0, 0), 1, "bf16", "bf16", 5, False),          # nothing turns
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%dx%d-%s-%s" % (c[0], c[1], c[2], c[6], c[7]))
@pytest.mark.parametrize("backward", [False, True])
def test_matches_the_formula(cuda_ok, case, backward):
    import torch
    B, S, Hq, Hk, dims, pairing, ti, to, far, own = case
    q, k = draw((B, S, Hq, 128), ti, 1), draw((B, S, Hk, 128), ti, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(0, 199, ((B, S, 3) if own else (S, 3)), generator=g, device="cuda").add(far).to(torch.int32)
    qo, ko = (torch.full(x.shape, float("nan"), dtype=types()[to], device="cuda") for x in (q, k))
    scale = (1.0, 0.25, 3.0)
    rope = vsa.make_rope(dims, theta=10000.0, scale=scale, pairing=pairing)
    (vsa.rope_bwd if backward else vsa.rope_fwd)(rope, pos, q, k, qo, ko)
    for x, y in ((q, qo), (k, ko)):
        check(y, *reference(x, pos, dims, pairing, scale=scale, sign=-1.0 if backward else 1.0))


def test_gradient_is_the_transpose_and_differences_agree(cuda_ok):
    """<rope(x), y> = <x, rope_bwd(y)> for random x, y; and the difference quotient of <rope(x), y> along a
    direction equals <direction, rope_bwd(y)> (the map is linear: any step gives it). Both sides are sums of n
    products whose factors are off by 11 * 2^-24 (|a| + |b|)."""
    import torch
    B, S, H = 2, 37, 3
    x, y, e = (draw((B, S, H, 128), "f32", n) for n in (4, 5, 6))
    pos = torch.arange(S, device="cuda", dtype=torch.int32)[:, None].repeat(1, 3) * 1000
    rope = vsa.make_rope((44, 42, 42), pairing=vsa.ROPE_HALVES)
    outs = {n: torch.empty_like(t) for n, t in (("x", x), ("e", x + e), ("g", y))}
    vsa.rope_fwd(rope, pos, x, None, outs["x"], None)
    vsa.rope_fwd(rope, pos, x + e, None, outs["e"], None)
    vsa.rope_bwd(rope, pos, y, None, outs["g"], None)
    dot = lambda a, b: (a.double() * b.double()).sum().item()  # noqa: E731
    size = 11 * U * 2 * (x.abs().max() + e.abs().max()).item() * y.abs().double().sum().item() * 2
    assert abs(dot(outs["x"], y) - dot(x, outs["g"])) <= size
    assert abs((dot(outs["e"], y) - dot(outs["x"], y)) - dot(e, outs["g"])) <= 2 * size


@pytest.mark.parametrize("pairing", [vsa.ROPE_ADJACENT, vsa.ROPE_HALVES])
def test_strides_in_place_and_broadcast(cuda_ok, pairing):
    import torch
    B, S, H = 2, 53, 3
    dims = (44, 42, 42)
    rope = vsa.make_rope(dims, pairing=pairing)
    pos = torch.randint(0, 50, (B, S, 3), device="cuda").to(torch.int32)
    qkv = draw((B, S, 3, H, 128), "bf16", 7)                       # slices of a fused projection
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    want_q, size_q = reference(q, pos, dims, pairing)
    want_k, size_k = reference(k, pos, dims, pairing)
    heads_first = torch.full((B, H, S, 128), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    ko = torch.empty_like(k)
    vsa.rope_fwd(rope, pos, q, k, heads_first, ko)
    check(heads_first, want_q, size_q)
    check(ko, want_k, size_k)
    v = qkv[:, :, 2].clone()
    vsa.rope_fwd(rope, pos, q, k, q, k)                            # in place
    check(q, want_q, size_q)
    check(k, want_k, size_k)
    assert torch.equal(qkv[:, :, 2], v)
    one = draw((B, S, 1, 128), "bf16", 8).expand(B, S, H, 128)     # one head broadcast
    out = torch.empty((B, S, H, 128), dtype=torch.bfloat16, device="cuda")
    vsa.rope_fwd(rope, pos, one, None, out, None)
    check(out, *reference(one, pos, dims, pairing))


def test_channels_behind_the_blocks_pass_through(cuda_ok):
    """Infinities, NaN and negative zero behind the rotated channels come out as they are, and stay there."""
    import torch
    x = draw((1, 9, 2, 128), "bf16", 9)
    x[..., 96::2] = float("inf")
    x[..., 97::4] = float("nan")
    x[..., 99::4] = -0.0
    pos = torch.arange(9, device="cuda", dtype=torch.int32)[:, None].repeat(1, 3)
    for pairing in (vsa.ROPE_ADJACENT, vsa.ROPE_HALVES):
        y = torch.empty_like(x)
        vsa.rope_fwd(vsa.make_rope((32, 32, 32), pairing=pairing), pos, x, None, y, None)
        bits = lambda t: t[..., 96:].contiguous().view(torch.int16)  # noqa: E731
        nan = torch.isnan(x[..., 96:].float())            # a NaN's payload is not kept
        assert torch.equal(torch.isnan(y[..., 96:].float()), nan) and torch.equal(bits(y)[~nan], bits(x)[~nan])
        check(y[..., :96], *(t[..., :96] for t in reference(x, pos, (32, 32, 32), pairing)))


def test_empty_and_mixed_types(cuda_ok):
    import torch
    rope = vsa.make_rope()
    none = torch.empty((2, 0, 3, 128), dtype=torch.bfloat16, device="cuda")
    vsa.rope_fwd(rope, torch.empty((0, 3), dtype=torch.int32, device="cuda"), none, none, none.clone(), none.clone())
    q, k = draw((1, 20, 2, 128), "f32", 10), draw((1, 20, 1, 128), "bf16", 11)
    pos = torch.arange(20, device="cuda", dtype=torch.int32)[:, None].repeat(1, 3)
    qo, ko = torch.empty_like(q), torch.empty(k.shape, dtype=torch.float16, device="cuda")
    vsa.rope_fwd(rope, pos, q, k, qo, ko)                           # q and k of different types
    for x, y in ((q, qo), (k, ko)):
        check(y, *reference(x, pos, (44, 42, 42), 0))


def test_captured_call_replays_on_new_inputs(cuda_ok):
    import torch
    rope = vsa.make_rope()
    q = draw((1, 70, 2, 128), "bf16", 12)
    pos = torch.arange(70, device="cuda", dtype=torch.int32)[:, None].repeat(1, 3)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        vsa.rope_fwd(rope, pos, q, None, out, None, stream=s)
    for seed in (13, 14):
        q.copy_(draw(q.shape, "bf16", seed))
        pos.add_(12345)
        graph.replay()
        torch.cuda.synchronize()
        check(out, *reference(q, pos, (44, 42, 42), 0))


@pytest.mark.parametrize("cond,grid,after", [
    (((0, 70),), (5, 6, 7), ((2, 3),)),
    ((), (3, 1, 9), ()),
    (((0, 5), (1, 300)), (9, 4, 13), ((2, 100),)),
])
def test_layout_positions(cuda_ok, cond, grid, after):
    import torch
    segs, at, want, n = [], 0, [], 0
    for kind, length in cond:
        segs.append((kind, at, length, None))
        at += length
    n_video = math.prod(grid)
    before = at
    segs.append((vsa.SEG_VIDEO, at, n_video, grid))
    at += n_video
    for kind, length in after:
        segs.append((kind, at, length, None))
        at += length
    for i in range(at):
        j = i - before
        if 0 <= j < n_video:
            t, h, w = j // (grid[1] * grid[2]), j // grid[2] % grid[1], j % grid[2]
            want.append((t + 100, h - 3, w + 7))
        else:
            want.append((n, n, n))
            n += 1
    pos = torch.empty((at, 3), dtype=torch.int32, device="cuda")
    vsa.rope_positions(vsa.Layout(segs, at), pos, origin=(100, -3, 7))
    assert pos.tolist() == [list(p) for p in want]


@pytest.mark.parametrize("dims", [(34, 30, 30), (16, 24, 8), (44, 42, 42), (16, 56, 56)], ids=lambda d: "%d-%d-%d" % d)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_halves_in_place_at_every_alignment(cuda_ok, dims, dtype):
    """Halves whose partners lie at multiples of four channels or not, in place, with infinities and NaN behind the
    rotated channels and rows of views with space between them."""
    import torch
    end = sum(dims)
    wide = draw((2, 83, 5, 160), dtype, 21)
    x = wide[:, :, 1:4, :128]
    x[..., end:] = float("inf")
    x[..., end + 1::3] = float("nan")
    pos = torch.arange(83, device="cuda", dtype=torch.int32)[:, None].repeat(1, 3) * 77
    want = reference(x, pos, dims, vsa.ROPE_HALVES)
    before = wide.clone()
    vsa.rope_fwd(vsa.make_rope(dims, pairing=vsa.ROPE_HALVES), pos, x, None, x, None)
    check(x[..., :end], *(t[..., :end] for t in want))
    tail, old = x[..., end:].float(), before[:, :, 1:4, end:128].float()
    assert torch.equal(tail.isnan(), old.isnan()) and torch.equal(tail.isinf(), old.isinf())
    assert torch.equal(wide[..., 128:], before[..., 128:]) and torch.equal(wide[:, :, 0], before[:, :, 0])
    assert torch.equal(wide[:, :, 4], before[:, :, 4])


@pytest.mark.parametrize("pairing", [vsa.ROPE_ADJACENT, vsa.ROPE_HALVES])
def test_one_token_of_a_table_of_positions(cuda_ok, pairing):
    """A streaming step takes its token's row out of a longer table, shared or of each batch entry."""
    import torch
    dims = (44, 42, 42)
    rope = vsa.make_rope(dims, pairing=pairing)
    table = torch.randint(0, 5000, (3, 30, 3), device="cuda").to(torch.int32)
    q = draw((3, 1, 5, 128), "bf16", 41)
    for pos in (table[0, 17:18], table[:, 17:18], table[0, 17].expand(3, 1, 3)):
        out = torch.full_like(q, float("nan"))
        vsa.rope_fwd(rope, pos, q, None, out, None)
        check(out, *reference(q, pos, dims, pairing))
