"""Layer norm (vsa_layer_norm_fwd, vsa_layer_norm_bwd) against the formula in
64 bits.

Tolerances, u = 2^-24. A row sum is at most 16 values in sequence per thread,
then at most 10 pairwise levels and the product with 1/n: a sum of terms t_i is
off by at most 32 u sum|t_i|. So
  mean : dm <= 33 u mean|x|
  x - mean rounds once and carries dm; the variance about a mean that is off by
  dm grows by dm^2, its sum rounds as above: relative dv <= 36 u + (dm r)^2 (u
  for the addition of eps; r = rstd); the reciprocal square root is within 2 steps
  of 2^-23 (its documented bound):
  rstd : dr <= dv / 2 + 4 u (relative)
  xh   : dxh <= dm r + |xh| (dr + 3 u)
  y    : |w| dxh + 2 u (|xh w| + |b|) + half a step of y's type
  dx   : c1 = mean(g), c2 = mean(g xh): dc1 <= 34 u mean|g|,
         dc2 <= 35 u mean|g xh| + mean(|g| dxh);
         dx <= r (dc1 + |xh| dc2 + |c2| dxh + 4 u (|g| + |c1| + |xh c2|)) + |dx| (dr + u) + half a step
  dw, db: at most R terms in sequence over all blocks and their joining:
         (R + 16) u sum|dy xh| + sum |dy| dxh, and (R + 16) u sum|dy|.
The backward's statistics come from its inputs mean and rstd, whose own error
the bounds above include.
"""

import pytest

from block_sparse_video_geometry_b200 import vsa

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def types():
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


class Reference:
    """The formula in float64 on x [rows, N] with the error bounds of the module's docstring."""

    def __init__(self, x, w, b, eps):
        x = x.double().reshape(-1, x.shape[-1])
        n = x.shape[1]
        self.w = w.double() if w is not None else x.new_ones(n)
        self.b = b.double() if b is not None else x.new_zeros(n)
        self.mean = x.mean(1, keepdim=True)
        var = ((x - self.mean) ** 2).mean(1, keepdim=True)
        self.r = (var + eps) ** -0.5
        self.xh = (x - self.mean) * self.r
        self.y = self.xh * self.w + self.b
        self.dm = 33 * U * x.abs().mean(1, keepdim=True)
        self.dr = (36 * U + (self.dm * self.r) ** 2) / 2 + 4 * U
        self.dxh = self.dm * self.r + self.xh.abs() * (self.dr + 3 * U)

    def tol_y(self, dtype):
        return (self.w.abs() * self.dxh + 2 * U * ((self.xh * self.w).abs() + self.b.abs())
                + half_step(dtype) * self.y.abs() * 1.001 + (2.0 ** -25 if half_step(dtype) == 2.0 ** -11 else 0))

    def backward(self, dy):
        dy = dy.double().reshape(self.xh.shape)
        g = dy * self.w
        c1, c2 = g.mean(1, keepdim=True), (g * self.xh).mean(1, keepdim=True)
        dx = self.r * (g - c1 - self.xh * c2)
        dc1 = 34 * U * g.abs().mean(1, keepdim=True)
        dc2 = 35 * U * (g * self.xh).abs().mean(1, keepdim=True) + (g.abs() * self.dxh).mean(1, keepdim=True)
        tol = self.r * (dc1 + self.xh.abs() * dc2 + c2.abs() * self.dxh
                        + 4 * U * (g.abs() + c1.abs() + (self.xh * c2).abs())) + dx.abs() * (self.dr + U)
        rows = dy.shape[0]
        dw, db = (dy * self.xh).sum(0), dy.sum(0)
        tw = (rows + 16) * U * (dy * self.xh).abs().sum(0) + (dy.abs() * self.dxh).sum(0)
        tb = (rows + 16) * U * dy.abs().sum(0)
        return dx, tol, dw, tw, db, tb


def within(got, want, tol, what):
    err = (got.double().reshape(want.shape) - want).abs()
    worst = (err - tol).max().item() if err.numel() else 0.0
    assert worst <= 0, "%s: beyond its bound by %.3g (error %.3g)" % (what, worst, err.max().item())


def rows_of(shape, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return (torch.exp(n(*shape[:-1], 1)) * (n(*shape) * torch.exp(n(shape[-1])) + 0.5)).to(types()[dtype])


def step(x, w, b, dy, eps=1e-6, dx_dtype=None, stream=None):
    """Forward and backward; checks every output; returns them."""
    import torch
    y = torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda")
    mean, rstd = (torch.full(x.shape[:-1], float("nan"), dtype=torch.float32, device="cuda") for _ in range(2))
    vsa.layer_norm_fwd(x, w, b, eps, y, mean, rstd, stream)
    dx = torch.full(x.shape, float("nan"), dtype=dx_dtype or dy.dtype, device="cuda")
    dw, db = (torch.full((x.shape[-1],), float("nan"), dtype=torch.float32, device="cuda") for _ in range(2))
    ws = torch.full((vsa.layer_norm_bwd_workspace_size(x),), 255, dtype=torch.uint8, device="cuda")   # NaN sums
    vsa.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db, ws, stream)
    return y, mean, rstd, dx, dw, db


def check_step(x, w, b, dy, outs, eps=1e-6):
    y, mean, rstd, dx, dw, db = outs
    ref = Reference(x, w, b, eps)
    within(mean, ref.mean, ref.dm, "mean")
    within(rstd, ref.r, ref.r * ref.dr, "rstd")
    within(y, ref.y, ref.tol_y(y.dtype), "y")
    want, tol, wdw, tw, wdb, tb = ref.backward(dy)
    tiny = 2.0 ** -25 if half_step(dx.dtype) == 2.0 ** -11 else 0.0
    within(dx, want, tol + (want.abs() + tol) * half_step(dx.dtype) + tiny, "dx")
    within(dw, wdw, tw, "dweight")
    within(db, wdb, tb, "dbias")


CASES = [
    # shape, x, weight, dy, dx
    ((1, 1), "f32", "f32", "f32", "f32"),
    ((5, 1), "bf16", "f32", "f32", "bf16"),
    ((7, 3), "bf16", "bf16", "bf16", "bf16"),
    ((33, 31), "f16", "f16", "f16", "f16"),
    ((2, 300, 3, 128), "bf16", "f32", "bf16", "bf16"),       # heads
    ((2, 301, 5, 128), "f16", "f16", "f32", "f16"),
    ((1, 67, 24, 128), "f32", "f32", "f32", "f32"),
    ((1027, 256), "bf16", "bf16", "f32", "f32"),             # one warp per row
    ((1026, 257), "bf16", "bf16", "bf16", "f32"),            # odd width: single elements
    ((3, 111, 264), "f16", "f32", "f16", "f16"),             # the narrowest row of a block
    ((4, 4096), "bf16", "bf16", "bf16", "bf16"),
    ((311, 79), "bf16", "bf16", "bf16", "bf16"),            # odd widths: lanes of a warp, then blocks
    ((65, 511), "f16", "f32", "f32", "f16"),
    ((65, 513), "bf16", "f32", "f32", "bf16"),
    ((600, 4097), "bf16", "f32", "bf16", "f32"),
    ((1300, 9009), "bf16", "bf16", "bf16", "bf16"),
    ((700, 1153), "f32", "f32", "f32", "f32"),
    ((171, 5120), "bf16", "f32", "bf16", "bf16"),
    ((171, 5128), "bf16", "f32", "f32", "bf16"),             # the next kernel variant
    ((600, 6144), "bf16", "f32", "bf16", "bf16"),            # just 48 KB of rows in flight
    ((6, 3000), "bf16", "f32", "bf16", "bf16"),
    ((9, 8192), "f16", "f16", "f16", "f16"),
    ((9, 8193), "bf16", "bf16", "bf16", "bf16"),
    ((3, 8200), "bf16", "f32", "f32", "f32"),
    ((2, 16384), "f32", "f32", "f32", "f32"),
    ((2, 16381), "f32", "f32", "f32", "f32"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[0])) + "-" + "-".join(c[1:]))
def test_matches_the_formula(cuda_ok, case):
    import torch
    shape, tx, tw, tg, td = case
    x = rows_of(shape, tx, 1)
    w = (1 + 0.3 * torch.randn(shape[-1], device="cuda")).to(types()[tw])
    b = (0.3 * torch.randn(shape[-1], device="cuda")).to(types()[tw])
    dy = torch.randn(shape, device="cuda").to(types()[tg])
    check_step(x, w, b, dy, step(x, w, b, dy, dx_dtype=types()[td]))


@pytest.mark.parametrize("N", [128, 130, 1000])
def test_without_weight_bias_or_statistics(cuda_ok, N):
    import torch
    x = rows_of((2, 9, 3, N), "bf16", 2)
    dy = torch.randn(x.shape, device="cuda").bfloat16()
    check_step(x, None, None, dy, step(x, None, None, dy))
    b = torch.randn(N, device="cuda")
    y = torch.empty_like(x)
    vsa.layer_norm_fwd(x, None, b, 1e-6, y)
    ref = Reference(x, None, b, 1e-6)
    within(y, ref.y, ref.tol_y(y.dtype), "y")
    _, mean, rstd, dx, dw, db = step(x, None, None, dy)
    only = torch.empty_like(dy)
    ws = torch.empty(vsa.layer_norm_bwd_workspace_size(x), dtype=torch.uint8, device="cuda")
    vsa.layer_norm_bwd(dy, x, None, mean, rstd, only, None, None, ws)
    assert torch.equal(only, dx)
    for which in (0, 1):
        got = torch.empty(N, device="cuda")
        vsa.layer_norm_bwd(dy, x, None, mean, rstd, only, got if which == 0 else None, got if which else None, ws)
        assert torch.equal(got, (dw, db)[which])


def test_large_offsets_and_constant_rows(cuda_ok):
    """A common offset of 1000 deviations, and rows of one value (variance 0: y is the bias)."""
    import torch
    x = torch.randn((50, 640), device="cuda") + 1000.0
    x[7] = 3.25
    w, b = torch.randn(640, device="cuda"), torch.randn(640, device="cuda")
    dy = torch.randn((50, 640), device="cuda")
    out = step(x, w, b, dy)
    check_step(x, w, b, dy, out)
    assert torch.equal(out[0][7], b)


@pytest.mark.parametrize("N", [128, 768])
def test_infinities_stay_in_their_row(cuda_ok, N):
    import torch
    x = rows_of((40, N), "bf16", 3)
    dy = torch.randn((40, N), device="cuda").bfloat16()
    clean = step(x, None, None, dy)
    x[5, 3] = float("inf")
    x[6, 0] = float("nan")
    y, mean, rstd, dx, dw, db = step(x, None, None, dy)
    keep = [i for i in range(40) if i not in (5, 6)]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(dx[keep], clean[3][keep])
    assert torch.isnan(y[6].float()).all() and torch.isnan(y[5, 3])


def test_strides_in_place_and_alignment(cuda_ok):
    import torch
    big = rows_of((2, 30, 3, 4, 128), "bf16", 4)
    x = big[:, :, 1]                                      # heads of a fused projection
    w, b = torch.randn(128, device="cuda"), torch.randn(128, device="cuda")
    dy = torch.randn((2, 4, 30, 128), device="cuda").bfloat16().transpose(1, 2)
    check_step(x, w, b, dy, step(x, w, b, dy))
    other = big[:, :, 2].clone()
    ref = Reference(x.clone(), w, b, 1e-6)
    vsa.layer_norm_fwd(x, w, b, 1e-6, x)                  # in place
    within(x, ref.y, ref.tol_y(x.dtype), "y")
    assert torch.equal(big[:, :, 2], other)
    flat = rows_of((31 * 520 + 1,), "bf16", 5)
    shifted = flat[1:].view(31, 520)                      # rows off by one element
    dy = torch.randn((31, 520), device="cuda").bfloat16()
    w, b = torch.randn(520, device="cuda"), torch.randn(520, device="cuda")
    check_step(shifted, w, b, dy, step(shifted, w, b, dy))
    padded = rows_of((31, 523), "bf16", 6)[:, :520]       # a row stride that is no multiple of 16 bytes
    check_step(padded, w, b, dy, step(padded, w, b, dy))
    one = torch.randn((1, 1, 520), device="cuda").bfloat16().expand(2, 5, 520)      # a broadcast gradient
    x = rows_of((2, 5, 520), "bf16", 7)
    check_step(x, w, b, one, step(x, w, b, one))
    mean, rstd = (torch.empty((2, 5), device="cuda") for _ in range(2))
    y = torch.empty_like(x)
    vsa.layer_norm_fwd(x, w, b, 1e-6, y, mean, rstd)
    g = torch.randn((2, 5, 520), device="cuda")
    want = step(x, w, b, g)
    ws = torch.empty(vsa.layer_norm_bwd_workspace_size(x), dtype=torch.uint8, device="cuda")
    dw, db = torch.empty(520, device="cuda"), torch.empty(520, device="cuda")
    vsa.layer_norm_bwd(g, x, w, mean, rstd, g, dw, db, ws)          # dx over dy
    assert torch.equal(g, want[3]) and torch.equal(dw, want[4])


@pytest.mark.parametrize("N", [1, 2])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_one_and_two_elements(cuda_ok, N, dtype):
    """One element: y is the bias and dx is 0. Two: xh is +-1 up to eps, dx cancels to rounding, whose every step is
    the formula's own in 32 bits."""
    import torch
    x = rows_of((500, N), dtype, 11)
    w, b = 1 + 0.3 * torch.randn(N, device="cuda"), torch.randn(N, device="cuda")
    dy = torch.randn((500, N), device="cuda").to(x.dtype)
    outs = step(x, w, b, dy)
    check_step(x, w, b, dy, outs)
    if N == 1:
        assert torch.equal(outs[0], b.to(x.dtype).expand(500, 1)) and not outs[3].float().any()
    else:
        xf, g = x.float(), dy.float() * w
        xh = (xf - outs[1][:, None]) * outs[2][:, None]
        dx = outs[2][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        assert torch.equal(outs[3], dx.to(x.dtype))


def test_no_rows(cuda_ok):
    import torch
    x = torch.empty((2, 0, 128), device="cuda")
    y, mean, rstd, dx, dw, db = step(x, torch.ones(128, device="cuda"), None, x.clone())
    assert not dw.any() and not db.any()


def test_differences_agree(cuda_ok):
    """The gradient against central differences of sum(y * dy) in float64 on the formula: the kernel's dx, dweight
    and dbias along a random direction e, against (L(+h) - L(-h)) / 2h, whose error is h^2 / 6 |L'''|; h = 1e-4 and
    third derivatives of order |L'| leave 1e-8 relative, far below the kernel's 32-bit bounds used here."""
    import torch
    x = rows_of((13, 96), "f32", 8)
    w, b = 1 + 0.3 * torch.randn(96, device="cuda"), torch.randn(96, device="cuda")
    dy = torch.randn((13, 96), device="cuda")
    _, _, _, dx, dw, db = step(x, w, b, dy)
    ref = Reference(x, w, b, 1e-6)
    _, tol, _, tw, _, tb = ref.backward(dy)
    loss = lambda x, w, b: (Reference(x, w, b, 1e-6).y * dy.double()).sum()  # noqa: E731
    h = 1e-4
    for i, (grad, bound) in enumerate(((dx, tol), (dw, tw), (db, tb))):
        at = [x.double(), w.double(), b.double()]
        e = torch.randn(at[i].shape, device="cuda", dtype=torch.float64) * (ref.r ** -1 if i == 0 else 1.0)
        e = e / e.abs().max()
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * e, at[i] - h * e
        diff = ((loss(*up) - loss(*down)) / (2 * h)).item()
        got = (grad.double() * e).sum().item()
        slack = (e.abs() * (bound + U * grad.abs())).sum().item() + 1e-6 * (grad.abs().double() * e.abs()).sum().item()
        assert abs(got - diff) <= slack, (i, got, diff, slack)


def test_same_bits_and_captured_replay(cuda_ok):
    import torch
    x = rows_of((900, 1024), "bf16", 9)
    w = torch.randn(1024, device="cuda")
    dy = torch.randn((900, 1024), device="cuda").bfloat16()
    first, second = step(x, w, None, dy), step(x, w, None, dy)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, dx = torch.empty_like(x), torch.empty_like(dy)
    mean, rstd = torch.empty(900, device="cuda"), torch.empty(900, device="cuda")
    dw, db = torch.empty(1024, device="cuda"), torch.empty(1024, device="cuda")
    ws = torch.empty(vsa.layer_norm_bwd_workspace_size(x), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        vsa.layer_norm_fwd(x, w, None, 1e-6, y, mean, rstd, s)
        vsa.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db, ws, s)
    x.copy_(rows_of((900, 1024), "bf16", 10))
    dy.copy_(torch.randn((900, 1024), device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    check_step(x, w, None, dy, (y, mean, rstd, dx, dw, db))


@pytest.mark.parametrize("shape", [(17408, 5120), (40, 16384), (3000, 9009), (1, 4096), (2, 300, 24, 128), (5000, 257),
                                   (700, 1153), (1500, 2048)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("shift", [0, 1])
def test_nothing_is_written_behind_the_workspace(cuda_ok, shape, shift):
    """Exactly the bytes that were asked for, marked ones behind them, rows aligned or not."""
    import torch
    n = 1
    for s in shape:
        n *= s
    flat = torch.randn(n + shift, device="cuda").bfloat16()
    x = flat[shift:].view(shape)
    dy = torch.randn(shape, device="cuda")
    y = torch.empty_like(x)
    mean, rstd = (torch.empty(shape[:-1], device="cuda") for _ in range(2))
    vsa.layer_norm_fwd(x, None, None, 1e-6, y, mean, rstd)
    size = vsa.layer_norm_bwd_workspace_size(x)
    ws = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    dx = torch.empty(shape, device="cuda")
    dw, db = (torch.empty(shape[-1], device="cuda") for _ in range(2))
    vsa.layer_norm_bwd(dy, x, None, mean, rstd, dx, dw, db, ws[:size])
    assert bool((ws[size:] == 0x5A).all())
    ref = Reference(x, None, None, 1e-6)
    _, _, wdw, tw, wdb, tb = ref.backward(dy)
    within(dw, wdw, tw, "dweight")
    within(db, wdb, tb, "dbias")
