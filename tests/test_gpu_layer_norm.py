"""moe_layer_norm_fwd / moe_layer_norm_bwd against the formulas in 64 bits.

Tolerances. u = eps(fp32) / 2 = 2^-24, r = eps(type) / 2 the rounding of a result.
  Row sums of H terms: a thread adds at most 16 of them one after the other, then
  at most 5 + 16 more, so a sum is off by at most 37 u times the sum of the
  terms' magnitudes; with the few operations around it, C = 40 u bounds every sum.
  mean: C * mean|x|.  rstd: the variance is a sum of squares of deviations that are
  off by (mean's error + u |x|) each; relative to the deviation's own size D = rms
  that is kappa = C * (mean|x| + max|x|) / D, so rstd is off by at most
  (C + 2 kappa) relative (first order, doubled below). y: each factor's error,
  |n| (C + 2 kappa) + kappa on n, times gamma, and the final rounding r.
  dx and the parameter gradients follow the same way from n and the given statistics.
"""
import numpy as np
import pytest
import torch

from bwd_route_b200 import ops
from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
C = 40 * U
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _tiny(dtype):
    """Half of the smallest step near zero."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


class Out(Guarded):
    """A guarded output of any element type: whole 32-bit words of guard around it."""

    def __init__(self, *shape, dtype=F32):
        n = int(np.prod(shape))
        size = torch.empty(0, dtype=dtype).element_size()
        words = (n * size + 3) // 4
        super().__init__(words, torch.int32)
        self.t = self.buf.view(torch.uint8)[256:256 + n * size].view(dtype).view(*shape)


def _inputs(T, H, dtype, pdtype, seed=0, ld=None, offset=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + H)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = torch.empty(T, ld or H, dtype=dtype, device="cuda")[:, :H]
    x.copy_(r(T, H) * (0.5 + r(H).abs()) + offset * r(H))
    return x, (1 + 0.2 * r(H)).to(pdtype), (0.3 * r(H)).to(pdtype), r(T, H).to(dtype)


def _reference(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = 1 / (var + eps).sqrt()
    n = (x - mean) * rstd
    g = 1.0 if gamma is None else gamma.double()
    b = 0.0 if beta is None else beta.double()
    kappa = C * (x.abs().mean(1, keepdim=True) + x.abs().amax(1, keepdim=True)) / (var + eps).sqrt()
    return mean[:, 0], rstd[:, 0], n * g + b, n, kappa


def _within(name, got, want, tol):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {(err / tol).max().item():.3g} tolerances"


def _check_y(y, x, gamma, beta, eps):
    _, _, want, n, kappa = _reference(x, gamma, beta, eps)
    rel = (C + 2 * kappa) * 2
    fp32 = gamma.double().abs() * (n.abs() * rel + 2 * kappa) + 4 * U * (want.abs() + beta.double().abs())
    _within("y", y, want, fp32 + _half(y.dtype) * (want.abs() + fp32) + _tiny(y.dtype))


SHAPES = [(1, 1), (3, 2), (5, 7), (1, 8), (2, 31), (9, 32), (8, 33), (17, 64), (7, 100), (33, 127), (4, 128), (1000, 256),
          (5, 512), (3, 513), (6, 1000), (7, 1001), (2, 1024), (3, 2048), (2, 4096), (2, 4097), (3, 5000), (2, 8191),
          (2, 8192), (4099, 40),
          # rows of 4 to 32 threads, odd numbers of them, and widths that allow two values at a time
          (1001, 16), (30001, 3), (777, 50), (333, 58), (130, 258), (65, 500), (67, 1002), (9, 2050), (5, 7970), (20000, 64)]


@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, BF16), (F16, F32), (F16, F16), (BF16, F32)], ids=str)
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H, dtype, pdtype):
    x, gamma, beta, _ = _inputs(T, H, dtype, pdtype)
    eps = 1e-5
    y, mean, rstd = Out(T, H, dtype=dtype), Out(T), Out(T)
    ops.moe_layer_norm_fwd(x, gamma, beta, eps, y.t, mean.t, rstd.t)
    torch.cuda.synchronize()
    assert y.guards_intact() and mean.guards_intact() and rstd.guards_intact()
    m, r, want, n, kappa = _reference(x, gamma, beta, eps)
    _within("mean", mean.t, m, C * x.double().abs().mean(1) + 1e-38)
    _within("rstd", rstd.t, r, ((C + 2 * kappa) * 2)[:, 0] * r)
    _check_y(y.t, x, gamma, beta, eps)


@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, BF16), (F16, F32), (F16, F16), (BF16, F32)], ids=str)
@pytest.mark.parametrize("T,H", SHAPES)
def test_backward(T, H, dtype, pdtype):
    x, gamma, beta, dy = _inputs(T, H, dtype, pdtype)
    _backward(x, gamma, dy, 1e-5)


def _backward(x, gamma, dy, eps, want=("dx", "dgamma", "dbeta"), dx_over_dy=False):
    T, H = x.shape
    dtype = x.dtype
    pdtype = dtype if gamma is None else gamma.dtype
    mean, rstd, _, _, _ = _reference(x, gamma, None, eps)
    mean, rstd = mean.float(), rstd.float()
    ws = ops.new_layer_norm_workspace(T, H, "cuda")
    out = {"dx": Out(T, H, dtype=dtype), "dgamma": Out(H, dtype=pdtype), "dbeta": Out(H, dtype=pdtype)}
    dy0 = dy.clone()
    if dx_over_dy:
        out["dx"].t.copy_(dy)
        dy = out["dx"].t
    ops.moe_layer_norm_bwd(x, dy, gamma, mean, rstd, *(out[k].t if k in want else None for k in out), ws)
    torch.cuda.synchronize()
    assert all(o.guards_intact() for o in out.values())
    # the formula, from the statistics given
    m, r, d = mean.double()[:, None], rstd.double()[:, None], dy0.double()
    g = torch.ones(H, dtype=torch.float64, device="cuda") if gamma is None else gamma.double()
    xd = x.double()
    n = (xd - m) * r
    dn = 2 * U * (xd.abs() + m.abs()) * r + U * n.abs()  # how far the kernel's n may be
    u = d * g
    s1, s2 = u.mean(1, keepdim=True), (u * n).mean(1, keepdim=True)
    e1 = C * u.abs().mean(1, keepdim=True)
    e2 = (C * (u * n).abs() + u.abs() * dn).mean(1, keepdim=True)
    if "dx" in want:
        ref = r * (u - s1 - n * s2)
        tol = r * (4 * U * (u.abs() + s1.abs() + (n * s2).abs()) + e1 + n.abs() * e2 + dn * s2.abs()) * 1.01
        _within("dx", out["dx"].t, ref, tol + _half(dtype) * (ref.abs() + tol) + _tiny(dtype))
    # Sums over tokens: at most 64 rows in a register, ceil(T / 64) flushes, 64 row teams (256 threads,
    # 4 of them a row at least), 32 + 32 blocks.
    chain = (64 + -(-T // 64) + 64 + 64) * U
    for k, ref, mag in (("dgamma", (d * n).sum(0), (d.abs() * (n.abs() * chain + dn)).sum(0)),
                        ("dbeta", d.sum(0), d.abs().sum(0) * chain)):
        if k in want:
            _within(k, out[k].t, ref, mag + _half(pdtype) * (ref.abs() + mag) + _tiny(pdtype))
    return out


@pytest.mark.parametrize("want", [("dx",), ("dgamma",), ("dbeta",), ("dgamma", "dbeta"), ("dx", "dbeta")], ids="+".join)
def test_backward_of_some_outputs(want):
    x, gamma, _, dy = _inputs(37, 96, F32, F32)
    out = _backward(x, gamma, dy, 1e-5, want)
    for k in ("dx", "dgamma", "dbeta"):
        if k not in want:  # left as it was
            assert bool((out[k].buf == out[k].buf[0]).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_backward_over_many_rows(dtype):
    """Every block adds more rows than one flush of its column sums."""
    x, gamma, _, dy = _inputs(300001, 24, dtype, dtype)
    _backward(x, gamma, dy, 1e-5)


@pytest.mark.parametrize("H,ld", [(64, 96), (64, 67), (100, 104), (1001, 1003)])
def test_strided_rows_and_no_parameters(H, ld):
    T = 41
    for dtype in (F32, BF16):
        x, _, _, dy = _inputs(T, H, dtype, dtype, ld=ld)
        assert x.stride(0) == ld
        y, y2 = Out(T, H, dtype=dtype), Out(T, H, dtype=dtype)
        ops.moe_layer_norm_fwd(x, None, None, 0.0, y.t)
        one, zero = torch.ones(H, dtype=dtype, device="cuda"), torch.zeros(H, dtype=dtype, device="cuda")
        ops.moe_layer_norm_fwd(x, one, zero, 0.0, y2.t)
        assert torch.equal(y.t, y2.t) and y.guards_intact()
        # rows a dense copy would start elsewhere may be summed in another order: the same bound, not the same bits
        _check_y(y.t, x, one, zero, 0.0)
        _backward(x, None, dy, 1e-5)


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_rows_that_start_off_sixteen_bytes(shift):
    T, H = 9, 128
    for dtype in (F32, F16):
        x, gamma, beta, dy = _inputs(T, H, dtype, dtype)
        off = torch.empty(T * H + shift, dtype=dtype, device="cuda")[shift:].view(T, H)
        off.copy_(x)
        a, b = torch.empty_like(x), torch.empty_like(x)
        ops.moe_layer_norm_fwd(x, gamma, beta, 1e-5, a)
        ops.moe_layer_norm_fwd(off, gamma, beta, 1e-5, b)
        # another thread layout, so another order of the sums: each is within the test's bound of the other
        _check_y(b, x, gamma, beta, 1e-5)
        _backward(off, gamma, dy, 1e-5)


def test_in_place():
    x, gamma, beta, dy = _inputs(77, 640, F32, F32)
    want = torch.empty_like(x)
    ops.moe_layer_norm_fwd(x, gamma, beta, 1e-5, want)
    over = x.clone()
    ops.moe_layer_norm_fwd(over, gamma, beta, 1e-5, over)
    assert torch.equal(over, want)
    _backward(x, gamma, dy, 1e-5, dx_over_dy=True)


def test_far_from_zero():
    """Deviations much smaller than the mean: the variance comes from the deviations themselves."""
    T, H = 6, 384
    x = (1000 + torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda"))
    y = torch.empty_like(x)
    ops.moe_layer_norm_fwd(x, None, None, 0.0, y)
    _, _, want, n, kappa = _reference(x, None, None, 0.0)
    _within("y", y, want, (n.abs() * (C + 2 * kappa) + kappa) * 2 + U * want.abs())


def test_rows_with_infinities_and_nan_leave_the_others_alone():
    x, gamma, beta, dy = _inputs(16, 200, F32, F32)
    want = torch.empty_like(x)
    ops.moe_layer_norm_fwd(x, gamma, beta, 1e-5, want)
    bad = x.clone()
    bad[3, 5], bad[7, 199], bad[8, 0] = float("nan"), float("inf"), -float("inf")
    y = torch.empty_like(x)
    ops.moe_layer_norm_fwd(bad, gamma, beta, 1e-5, y)
    rows = torch.tensor([r not in (3, 7, 8) for r in range(16)], device="cuda")
    assert torch.equal(y[rows], want[rows])
    assert torch.isnan(y[~rows]).all()


def test_constant_rows():
    x = torch.full((2, 48), 3.25, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    ops.moe_layer_norm_fwd(x, None, None, 1e-5, y, mean, rstd)
    assert (y == 0).all() and (mean == 3.25).all()
    ops.moe_layer_norm_fwd(x, None, None, 0.0, y, mean, rstd)
    assert torch.isinf(rstd).all() and torch.isnan(y).all()


def test_no_rows():
    H = 40
    e = torch.empty(0, H, device="cuda")
    ops.moe_layer_norm_fwd(e, None, None, 1e-5, e)
    dg, db = torch.full((H,), 7.0, device="cuda"), torch.full((H,), 7.0, device="cuda")
    s = torch.empty(0, device="cuda")
    ops.moe_layer_norm_bwd(e, e, None, s, s, None, dg, db, None)
    assert (dg == 0).all() and (db == 0).all()


def test_gradient_against_differences():
    """Central differences of L = sum(c * y) in x, gamma and beta, through the forward kernel in fp32.

    L is a sum of H terms of size ~1 per row, each within ~1e-6 of the formula, so a difference over
    2h with h = 1/32 is off by at most ~ 2 * 40 * 1e-6 / (1/16) = 1.3e-3 plus the third-derivative term
    h^2 / 6 * |L'''|, below 1e-2 at unit scale; 2e-2 covers both."""
    T, H, h = 2, 40, 1.0 / 32
    x, gamma, beta, _ = _inputs(T, H, F32, F32, offset=0.2)
    c = torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")

    def loss(x, gamma, beta):
        out = torch.empty_like(x)
        ops.moe_layer_norm_fwd(x, gamma, beta, 1e-5, out)
        return (out.double() * c.double()).sum().item()

    ops.moe_layer_norm_fwd(x, gamma, beta, 1e-5, y, mean, rstd)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    ops.moe_layer_norm_bwd(x, c, gamma, mean, rstd, dx, dg, db, ops.new_layer_norm_workspace(T, H, "cuda"))
    for k, (t, grad) in enumerate(((x, dx), (gamma, dg), (beta, db))):
        for i in range(0, t.numel(), 7):
            at = []
            for s in (h, -h):
                moved = t.clone()
                moved.view(-1)[i] += s
                at.append(loss(*(moved if j == k else v for j, v in enumerate((x, gamma, beta)))))
            num = (at[0] - at[1]) / (2 * h)
            assert abs(num - grad.view(-1)[i].item()) <= 2e-2 * max(1.0, abs(num)), (k, i, num, grad.view(-1)[i].item())


def test_repeats_bit_for_bit_and_on_another_stream_and_in_a_graph():
    T, H = 5000, 320
    x, gamma, beta, dy = _inputs(T, H, BF16, BF16)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    y = torch.empty_like(x)
    ws = ops.new_layer_norm_workspace(T, H, "cuda")
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)

    def both(stream=None):
        ops.moe_layer_norm_fwd(x, gamma, beta, 1e-5, y, mean, rstd, stream)
        ops.moe_layer_norm_bwd(x, dy, gamma, mean, rstd, dx, dg, db, ws, stream)

    outs = (y, mean, rstd, dx, dg, db)
    both()
    want = [t.clone() for t in outs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in outs:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
