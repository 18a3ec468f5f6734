"""moe_topk_fwd / moe_topk_bwd against the definition in 64 bits.

Tolerances. u = 2^-24, r = eps(type) / 2. A tensor-core sum over n terms adds 16 at a
time to an fp32 accumulator, each addition off by at most 2^-22 of the largest
magnitude in it: A(n) = (n / 16 + 8) 2^-22 of the sum of the terms' magnitudes.
  y, d_x: A(H) of the magnitudes; when K > 1 every row w W x (the bias is added after it,
  in fp32) is rounded to fp16 scaled to its block's largest value, 2^-11 of itself and
  2^-39 of that value; r of the result.
  d_weights: A(H) of the magnitudes for the inner sum, 2 H u of them for the outer.
  dW: the rows w g are rounded to the type, independent errors of at most r of each
  term, so beyond 8 r sqrt(sum of squares) with probability below 2 exp(-32) per
  element (Hoeffding); A(n) of the magnitudes for n pairs, r of the result.
  db: n u of the magnitudes, r of the result.
The 16-bit rows of y and d_x and the rounded terms of dW are an allowance: the tests of rows
added in fp32 and of fp32 terms, further down, hold the calls to bounds without it.
"""
import numpy as np
import pytest
import torch

from bwd_route_b200 import ops
from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F16 = torch.bfloat16, torch.float16


def _acc(n):
    return (n / 16 + 8) * 2.0 ** -22


class Out(Guarded):
    def __init__(self, *shape, dtype=BF16):
        n = int(np.prod(shape))
        size = torch.empty(0, dtype=dtype).element_size()
        super().__init__((n * size + 3) // 4, torch.int32)
        self.t = self.buf.view(torch.uint8)[256:256 + n * size].view(dtype).view(*shape)


def _routing(T, E, K, seed=0, skew=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(T, E, generator=g, device="cuda") + skew * torch.randn(E, generator=g, device="cuda")
    r = ops.Routing.empty(T * K, E, "cuda")
    w = torch.empty(T, K, device="cuda")
    ops.moe_topk_route(logits, ops.TopKRule(E, K, ops.MOE_SCORE_SIGMOID), None, r, w, ops.new_topk_workspace(T, E, K, 0, "cuda"))
    return r, w


def _data(T, E, K, H, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (rand(T, H).to(dtype), (rand(E, H, H) / H ** 0.5).to(dtype), (rand(E, H) * 0.3).to(dtype), rand(T, H).to(dtype))


def _reference(x, W, b, g, idx, w):
    """Values and the magnitudes (sums of |terms|) their errors are measured by."""
    T, H = x.shape
    E, K = W.shape[0], w.shape[1]
    d = torch.float64
    x, W, w = x.to(d), W.to(d), w.to(d)
    b = torch.zeros(E, H, dtype=d, device=x.device) if b is None else b.to(d)
    idx = idx.view(T, K).long()
    z = lambda *s: torch.zeros(*s, dtype=d, device=x.device)  # noqa: E731
    o = {"y": z(T, H), "y_acc": z(T, H), "y_rows": z(T, H)}
    if g is not None:
        g = g.to(d)
        o |= {"d_x": z(T, H), "d_x_acc": z(T, H), "d_x_rows": z(T, H), "dW": z(E, H, H), "dW_abs": z(E, H, H),
              "dW_sq": z(E, H, H), "db": z(E, H), "db_abs": z(E, H), "d_weights": z(T, K), "dw_abs": z(T, K)}
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        wt = w[t, k][:, None]
        plain = x[t] @ W[e].T
        row = plain + b[e]
        o["y"].index_add_(0, t, wt * row)
        o["y_rows"].index_add_(0, t, (wt * plain).abs())
        o["y_acc"].index_add_(0, t, wt.abs() * (x[t].abs() @ W[e].abs().T + b[e].abs()))
        if g is None:
            continue
        back, mag = g[t] @ W[e], g[t].abs() @ W[e].abs()
        o["d_x"].index_add_(0, t, wt * back)
        o["d_x_rows"].index_add_(0, t, (wt * back).abs())
        o["d_x_acc"].index_add_(0, t, wt.abs() * mag)
        wg = wt * g[t]
        o["dW"][e] = wg.T @ x[t]
        o["dW_abs"][e] = wg.abs().T @ x[t].abs()
        o["dW_sq"][e] = (wg ** 2).T @ (x[t] ** 2)
        o["db"][e], o["db_abs"][e] = wg.sum(0), wg.abs().sum(0)
        o["d_weights"][t, k] = (g[t] * row).sum(1)
        o["dw_abs"][t, k] = (x[t].abs() * mag).sum(1) + (g[t].abs() * b[e].abs()).sum(1)
    return o


def _within(name, got, want, tol):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {(err / tol).max().item():.3g} tolerances"


def _check_rows(name, got, o, K, H):
    f = torch.finfo(got.dtype)
    r = f.eps / 2
    rows = o[name + "_rows"]
    fp32 = 2 * _acc(H) * o[name + "_acc"] + (2.0 ** -11 * rows * 1.01 + 2.0 ** -38 * rows.amax(1, True) if K > 1 else 0)
    _within(name, got, o[name], fp32 + r * (o[name].abs() + fp32) + f.smallest_normal * f.eps * K)


def _fwd(x, W, b, routing, w, ws=None):
    T, H = x.shape
    E, K = W.shape[0], w.shape[1]
    ws = ops.new_topk_workspace(T, E, K, H, "cuda") if ws is None else ws
    y = Out(T, H, dtype=x.dtype)
    ops.moe_topk_fwd(x, W, b, routing, w, y.t, ws)
    torch.cuda.synchronize()
    assert ops.moe_top1_device_flags(ws) == 0 and y.guards_intact()
    return y.t


OUTS = ("d_x", "dW", "db", "d_weights")


def _bwd(x, W, b, g, routing, w, want=OUTS, ws=None):
    T, H = x.shape
    E, K = W.shape[0], w.shape[1]
    ws = ops.new_topk_workspace(T, E, K, H, "cuda") if ws is None else ws
    out = {"d_x": Out(T, H, dtype=x.dtype), "dW": Out(E, H, H, dtype=x.dtype), "db": Out(E, H, dtype=x.dtype),
           "d_weights": Out(T, K, dtype=torch.float32)}
    ops.moe_topk_bwd(x, W, b, g, routing, w, *(out[k].t if k in want else None for k in OUTS), ws)
    torch.cuda.synchronize()
    assert ops.moe_top1_device_flags(ws) == 0
    assert all(v.guards_intact() for v in out.values())
    for k in OUTS:
        if k not in want:
            assert bool((out[k].buf == out[k].buf[0]).all()), k
    return {k: v.t for k, v in out.items()}


def _check_bwd(got, o, routing, K, H, want=OUTS):
    f = torch.finfo(got["dW"].dtype)
    r = f.eps / 2
    n = int(routing.counts.max())
    if "d_x" in want:
        _check_rows("d_x", got["d_x"], o, K, H)
    if "d_weights" in want:
        _within("d_weights", got["d_weights"], o["d_weights"], (_acc(H) + 2 * H * U) * o["dw_abs"] + 1e-30)
    if "dW" in want:
        fp32 = 8 * r * o["dW_sq"].sqrt() + _acc(n) * 2 * o["dW_abs"]
        _within("dW", got["dW"], o["dW"], fp32 + r * (o["dW"].abs() + fp32) + f.smallest_normal * (1 + o["dW_abs"]))
    if "db" in want:
        fp32 = (n + 2) * U * o["db_abs"]
        _within("db", got["db"], o["db"], fp32 + r * (o["db"].abs() + fp32) + f.smallest_normal * f.eps)


SHAPES = [
    # T, E, K, H
    (1, 1, 1, 64), (1, 4, 2, 128), (2, 3, 3, 64), (5, 8, 1, 256), (127, 2, 2, 128), (128, 1, 1, 256), (129, 5, 3, 192),
    (300, 64, 8, 64), (40, 256, 16, 64), (1000, 4, 2, 256), (700, 8, 2, 320), (513, 7, 4, 512), (260, 6, 2, 1024),
    (5003, 4, 2, 128), (3000, 16, 4, 256), (20000, 8, 2, 64), (900, 3, 2, 448), (33, 8, 2, 2048),
]


@pytest.mark.parametrize("T,E,K,H", SHAPES)
def test_forward(T, E, K, H):
    for dtype in (BF16, F16):
        x, W, b, _ = _data(T, E, K, H, dtype)
        routing, w = _routing(T, E, K)
        for bias in (b, None):
            o = _reference(x, W, bias, None, routing.expert_idx, w)
            _check_rows("y", _fwd(x, W, bias, routing, w), o, K, H)


@pytest.mark.parametrize("T,E,K,H", SHAPES)
def test_backward(T, E, K, H):
    for dtype in (BF16, F16):
        x, W, b, g = _data(T, E, K, H, dtype)
        routing, w = _routing(T, E, K)
        for bias in (b, None):
            o = _reference(x, W, bias, g, routing.expert_idx, w)
            _check_bwd(_bwd(x, W, bias, g, routing, w), o, routing, K, H)


@pytest.mark.parametrize("T,E,K,H,skew", [(60000, 8, 2, 256, 1.0), (49151, 8, 2, 256, 0.5), (30000, 3, 2, 128, 0.3), (4000, 32, 4, 1024, 2.0),
                                          (20001, 60, 6, 64, 1.0), (6000, 2, 1, 512, 4.0),
                                          (50000, 4, 2, 192, 1.5), (49152, 2, 2, 256, 0.0), (70000, 9, 2, 128, 0.5),
                                          (60001, 12, 2, 64, 2.0), (9001, 13, 1, 640, 1.0), (5000, 8, 2, 1024, 1.0)])
def test_many_pairs_and_uneven_experts(T, E, K, H, skew):
    """Several tiles per block, experts cut into pieces and whole ones, experts without a pair."""
    x, W, b, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K, 3, skew)
    o = _reference(x, W, b, g, routing.expert_idx, w)
    _check_rows("y", _fwd(x, W, b, routing, w), o, K, H)
    _check_bwd(_bwd(x, W, b, g, routing, w), o, routing, K, H)


def _small_integers(T, E, K, H, seed):
    """Eight entries of +-1 per row and column of W, tokens of -1, 0, 1, weights 1/2 and 1: every sum
    is a multiple of 1/2 below 128, exact in both types."""
    g = torch.Generator().manual_seed(seed)
    W = torch.zeros(E, H, H)
    for e in range(E):
        for s in torch.randperm(H, generator=g)[:8].tolist():
            rows = torch.arange(H)
            W[e, rows, (rows + s) % H] = torch.randint(0, 2, (H,), generator=g).float() * 2 - 1
    tri = lambda *s: torch.randint(-1, 2, s, generator=g).float()  # noqa: E731
    w = torch.randint(1, 3, (T, K), generator=g).float() / 2
    return tri(T, H), W, tri(E, H), tri(T, H), w


@pytest.mark.parametrize("T,E,K,H", [(200, 4, 2, 128), (333, 6, 3, 256), (50, 5, 1, 64), (150, 3, 2, 320), (100, 4, 4, 1024),
                                     (50001, 3, 2, 192), (49152, 2, 2, 256), (52000, 4, 2, 64)])
def test_exact_on_small_integers(T, E, K, H):
    x, W, b, g, w = _small_integers(T, E, K, H, T)
    routing, _ = _routing(T, E, K, T)
    for dtype in (BF16, F16):
        X, WW, B, G = (v.to(dtype).cuda() for v in (x, W, b, g))
        ww = w.cuda()
        o = _reference(X, WW, B, G, routing.expert_idx, ww)
        assert torch.equal(_fwd(X, WW, B, routing, ww).double(), o["y"])
        got = _bwd(X, WW, B, G, routing, ww)
        for k in OUTS:  # dW and db: sums of at most T / 2 halves, below 128 or rounded once
            assert torch.equal(got[k], o[k].to(got[k].dtype)), k


@pytest.mark.parametrize("want", [("d_x",), ("d_weights",), ("dW",), ("db",), ("d_x", "dW"), ("db", "d_weights"),
                                  ("dW", "db"), ("d_x", "d_weights")], ids="+".join)
def test_some_outputs(want):
    T, E, K, H = 300, 5, 2, 192
    x, W, b, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    o = _reference(x, W, b, g, routing.expert_idx, w)
    _check_bwd(_bwd(x, W, b, g, routing, w, want), o, routing, K, H, want)


def _routing_of(idx, E):
    """A routing built on the host from given experts [T, K]."""
    flat = idx.reshape(-1).cuda()
    counts = torch.bincount(flat, minlength=E)
    i = torch.int32
    return ops.Routing(flat.to(i), counts.to(i), torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(i),
                       torch.sort(flat, stable=True)[1].to(i))


@pytest.mark.parametrize("T,E,H", [(400, 6, 64), (400, 6, 256), (50000, 6, 256), (49200, 7, 192)])
def test_everything_on_one_expert_and_the_same_expert_twice(T, E, H):
    """The larger ones group their tokens by pairs of experts."""
    K = 2
    x, W, b, g = _data(T, E, K, H, BF16)
    w = torch.rand(T, K, device="cuda")
    for idx in (torch.tensor([[2, 5]]).repeat(T, 1), torch.tensor([[3, 3]]).repeat(T, 1)):
        routing = _routing_of(idx, E)
        o = _reference(x, W, b, g, routing.expert_idx, w)
        _check_rows("y", _fwd(x, W, b, routing, w), o, K, H)
        got = _bwd(x, W, b, g, routing, w)
        _check_rows("d_x", got["d_x"], o, K, H)
        none = torch.bincount(idx.reshape(-1), minlength=E) == 0
        assert not got["dW"][none].any() and not got["db"][none].any()
        _check_bwd(got, o, routing, K, H)


def test_expert_indices_off_eight_bytes():
    """Pairs of indices are read together only where they start on 8 bytes."""
    T, E, K, H = 50000, 4, 2, 128
    x, W, b, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    off = torch.empty(T * K + 1, dtype=torch.int32, device="cuda")[1:]
    off.copy_(routing.expert_idx)
    moved = ops.Routing(off, routing.counts, routing.offsets, routing.perm)
    o = _reference(x, W, b, g, routing.expert_idx, w)
    _check_rows("y", _fwd(x, W, b, moved, w), o, K, H)
    _check_bwd(_bwd(x, W, b, g, moved, w), o, moved, K, H)


def test_weights_of_zero_and_negative_weights():
    T, E, K, H = 130, 4, 3, 128
    x, W, b, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    w = w - 0.4
    w[5] = 0
    o = _reference(x, W, b, g, routing.expert_idx, w)
    y = _fwd(x, W, b, routing, w)
    _check_rows("y", y, o, K, H)
    assert not y[5].any()
    _check_bwd(_bwd(x, W, b, g, routing, w), o, routing, K, H)


def test_a_token_with_nan_leaves_the_others_alone():
    T, E, K, H = 300, 4, 2, 256
    x, W, b, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    want = _fwd(x, W, b, routing, w)
    bad = x.clone()
    bad[17, 3], bad[200, 0] = float("nan"), float("inf")
    y = _fwd(bad, W, b, routing, w)
    rows = torch.tensor([t not in (17, 200) for t in range(T)], device="cuda")
    assert torch.equal(y[rows], want[rows])
    assert torch.isnan(y[17]).all() and not torch.isfinite(y[200]).any()


@pytest.mark.parametrize("K", [1, 2, 4])
def test_an_infinite_weight_of_the_product_leaves_other_columns_alone(K):
    T, E, H = 300, 4, 128
    x, W, b, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    o = _reference(x, W, b, g, routing.expert_idx, w)
    bad = W.clone()
    bad[2, 7, 5] = float("inf")
    chosen = (routing.expert_idx.view(T, K) == 2).any(1)
    assert chosen.any() and (x[:, 5] != 0).all() and (g[:, 7] != 0).all()
    for name, col, got in (("y", 7, _fwd(x, bad, b, routing, w)), ("d_x", 5, _bwd(x, bad, b, g, routing, w)["d_x"])):
        assert torch.equal(torch.isinf(got[:, col]), chosen), name
        got[:, col] = o[name][:, col].to(BF16)
        _check_rows(name, got, o, K, H)


@pytest.mark.parametrize("T,K", [(300, 1), (300, 2), (300, 5), (50000, 2)])
def test_weights_that_are_nan_or_infinite(T, K):
    E, H = 6, 128
    x, W, b, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    good = _fwd(x, W, b, routing, w), _bwd(x, W, b, g, routing, w, ("d_x",))["d_x"]
    bad = w.clone()
    bad[3, K - 1], bad[200, 0] = float("nan"), float("inf")
    rows = torch.tensor([t not in (3, 200) for t in range(T)], device="cuda")
    for want, got in zip(good, (_fwd(x, W, b, routing, bad), _bwd(x, W, b, g, routing, bad, ("d_x",))["d_x"])):
        assert torch.equal(got[rows], want[rows])
        assert torch.isnan(got[3]).all() and not torch.isfinite(got[200]).any()


def test_no_tokens():
    E, K, H = 4, 2, 128
    _, W, b, _ = _data(1, E, K, H, BF16)
    e = torch.empty(0, H, dtype=BF16, device="cuda")
    routing = ops.Routing.empty(0, E, "cuda")
    w = torch.empty(0, K, device="cuda")
    ws = ops.new_topk_workspace(0, E, K, H, "cuda")
    ops.moe_topk_fwd(e, W, b, routing, w, e.clone(), ws)
    dW, db = torch.ones_like(W), torch.ones_like(b)
    ops.moe_topk_bwd(e, W, b, e, routing, w, e.clone(), dW, db, w.clone(), ws)
    assert not dW.any() and not db.any()


@pytest.mark.parametrize("T,E,K,H", [(9000, 8, 3, 256), (50000, 5, 2, 256)])
def test_repeats_bit_for_bit_with_one_workspace(T, E, K, H):
    """Whatever the order in which a token's rows come in: the same bits, call after call, and with
    another size through the same workspace in between; on another stream; captured and replayed."""
    x, W, b, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    ws = ops.new_topk_workspace(T, E, K, H, "cuda")
    y0, g0 = _fwd(x, W, b, routing, w, ws), _bwd(x, W, b, g, routing, w, ws=ws)
    x1, W1, b1, g1 = _data(70, 4, 2, 64, BF16)
    r1, w1 = _routing(70, 4, 2)
    for _ in range(5):
        _fwd(x1, W1, b1, r1, w1, ws)
        assert torch.equal(_fwd(x, W, b, routing, w, ws), y0)
        got = _bwd(x, W, b, g, routing, w, ws=ws)
        assert all(torch.equal(got[k], g0[k]) for k in OUTS)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert torch.equal(_fwd(x, W, b, routing, w, ws), y0)
    torch.cuda.synchronize()
    y = torch.empty_like(x)
    out = [torch.empty_like(g0[k]) for k in OUTS]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_topk_fwd(x, W, b, routing, w, y, ws)
        ops.moe_topk_bwd(x, W, b, g, routing, w, *out, ws)
    for _ in range(3):
        y.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y0) and all(torch.equal(a, g0[k]) for a, k in zip(out, OUTS))


def test_gradient_against_differences():
    """Differences of L = sum(c * y) in fp64 of the reference, which the forward above is held to: the
    backward's d_x, d_weights, dW and db are the derivatives. y is linear in each argument, so a
    difference is exact up to fp64 rounding; the backward's own bounds apply."""
    T, E, K, H = 3, 3, 2, 64
    x, W, b, c = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    got = _bwd(x, W, b, c, routing, w)
    o = _reference(x, W, b, c, routing.expert_idx, w)
    _check_bwd(got, o, routing, K, H)
    loss = lambda *a: (_reference(*a[:3], None, routing.expert_idx, a[3])["y"] * c.double()).sum().item()  # noqa: E731
    args = [x.double(), W.double(), b.double(), w.double()]
    base = loss(*args)
    for j, k in enumerate(("d_x", "dW", "db", "d_weights")):
        for i in range(0, args[j].numel(), max(1, args[j].numel() // 40)):
            moved = [a.clone() for a in args]
            moved[j].view(-1)[i] += 0.5
            num = (loss(*moved) - base) * 2
            assert abs(num - o[k].view(-1)[i].item()) <= 1e-9 * (1 + abs(num)), (k, i)


@pytest.mark.parametrize("K", [1, 2, 5])
@pytest.mark.parametrize("want", [("d_x",), ("dW",), ("db",), ("d_x", "dW", "db")], ids="+".join)
def test_expert_indices_are_read_for_the_weights_gradient_only(want, K):
    """Without d_weights the bias plays no part, and the routing may come without expert_idx."""
    T, E, H = 300, 6, 128
    x, W, b, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    bare = ops.Routing(None, routing.counts, routing.offsets, routing.perm)
    o = _reference(x, W, b, g, routing.expert_idx, w)
    _check_bwd(_bwd(x, W, b, g, bare, w, want), o, routing, K, H, want)


@pytest.mark.parametrize("T,E,K,H", [(5, 8, 2, 256), (129, 5, 3, 192), (300, 64, 8, 64), (40, 256, 16, 64), (700, 8, 2, 320),
                                     (513, 7, 4, 512), (260, 6, 2, 1024), (5003, 4, 2, 128), (50000, 5, 2, 128)])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_a_tokens_rows_are_added_in_fp32(T, E, K, H, dtype):
    """y and d_x are rounded to 16 bits once, at the end: beside that rounding and the products' own bound
    there are K roundings of fp32 and those of the bias, K u and 2 u of the magnitudes."""
    x, W, b, g = _data(T, E, K, H, dtype)
    routing, w = _routing(T, E, K)
    o = _reference(x, W, b, g, routing.expert_idx, w)
    got = {"y": _fwd(x, W, b, routing, w), "d_x": _bwd(x, W, b, g, routing, w, ("d_x",))["d_x"]}
    f = torch.finfo(dtype)
    for k, v in got.items():
        fp32 = (2 * _acc(H) + (K + 2) * U) * o[k + "_acc"]
        _within(k, v, o[k], fp32 + f.eps / 2 * (o[k].abs() + fp32) + f.smallest_normal * f.eps)


@pytest.mark.parametrize("K", [1, 2, 4])
def test_large_weights_of_tiny_rows(K):
    """Rows of a few 2^-118 under weights of 2^119 and 2^120 are ordinary numbers."""
    T, E, H = 200, 5, 128
    x, W, _, g, w = _small_integers(T, E, K, H, 7)
    routing, _ = _routing(T, E, K, 7)
    X, WW, G = ((v * s).to(BF16).cuda() for v, s in ((x, 2.0 ** -60), (W, 2.0 ** -58), (g, 2.0 ** -60)))
    ww = (w * 2.0 ** 120).cuda()
    o = _reference(X, WW, None, G, routing.expert_idx, ww)
    assert torch.equal(_fwd(X, WW, None, routing, ww).double(), o["y"])
    assert torch.equal(_bwd(X, WW, None, G, routing, ww, ("d_x",))["d_x"].double(), o["d_x"])


@pytest.mark.parametrize("T,E,K,H", [(300, 4, 2, 128), (5003, 4, 2, 128), (700, 8, 3, 320), (3000, 2, 1, 512), (50000, 6, 2, 64)])
@pytest.mark.parametrize("w_to,g_rms,x_rms", [(16.0, 6000.0, 1e-3), (1000.0, 6000.0, 1e-5), (0.1, 1e-5, 1.0), (0.1, 1e-6, 30.0),
                                              (1e-6, 1.0, 3e3)])
def test_fp16_weight_gradient_whatever_the_terms_size(T, E, K, H, w_to, g_rms, x_rms):
    """w d_out leaves fp16's range above or below, dW itself does not. Beside the bounds at the top a term
    is off by 2^-39 of its expert's largest at most (half of fp16's last step, the largest brought to
    2^14), and the result by half of the type's last step."""
    x, W, b, g = _data(T, E, K, H, F16)
    x, g = (x.float() * x_rms).to(F16), (g.float() * g_rms).to(F16)
    assert torch.isfinite(g).all() and torch.isfinite(x).all()
    routing, _ = _routing(T, E, K)
    w = torch.rand(T, K, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") * w_to
    o = _reference(x, W, b, g, routing.expert_idx, w)
    got = _bwd(x, W, b, g, routing, w, ("dW", "db"))
    assert o["dW"].abs().max() < 6e4
    f = torch.finfo(F16)
    r, n = f.eps / 2, int(routing.counts.max())
    last = n * 2.0 ** -39 * (w.max() * g.abs().max().float() * x.abs().max().float()).double()
    fp32 = 8 * r * o["dW_sq"].sqrt() + _acc(n) * 2 * o["dW_abs"] + last
    _within("dW", got["dW"], o["dW"], fp32 + r * (o["dW"].abs() + fp32) + f.smallest_normal * r)
    fp32 = (n + 2) * U * o["db_abs"]
    in_range = o["db"].abs() < 6e4
    _within("db", got["db"][in_range], o["db"][in_range], (fp32 + r * (o["db"].abs() + fp32) + f.smallest_normal * r)[in_range])


def test_fp16_weight_gradient_of_rows_of_zeros_and_infinities():
    """A huge weight over a row of zeros adds nothing; an infinite d_out reaches its own experts only."""
    T, E, K, H = 300, 6, 2, 128
    x, W, b, g = _data(T, E, K, H, F16)
    routing, w = _routing(T, E, K)
    g[5] = 0
    want = _bwd(x, W, b, g, routing, w, ("dW", "db"))
    huge = w.clone()
    huge[5] = 3e38
    got = _bwd(x, W, b, g, routing, huge, ("dW", "db"))
    assert torch.equal(got["dW"], want["dW"]) and torch.equal(got["db"], want["db"])
    bad = g.clone()
    bad[7, 3] = float("inf")
    hit = torch.zeros(E, dtype=torch.bool, device="cuda")
    hit[routing.expert_idx.view(T, K)[7].long()] = True
    got = _bwd(x, W, b, bad, routing, w, ("dW", "db"))
    assert torch.equal(got["dW"][~hit], want["dW"][~hit]) and torch.equal(got["db"][~hit], want["db"][~hit])
    rows = torch.arange(H, device="cuda") != 3
    assert torch.isfinite(got["dW"][hit][:, rows]).all() and not torch.isfinite(got["dW"][hit][:, 3]).any()


def _check_dW(got, o, routing):
    """The rows w g are two 16-bit numbers each: the upper one leaves at most one of its steps, the lower
    one rounds that to half of its own, so a term is off by eps r of itself at most (2^-15 bf16, 2^-21
    fp16), independently of the others (Hoeffding, as above); their products are 2 n terms of a sum."""
    f = torch.finfo(got.dtype)
    r, n = f.eps / 2, int(routing.counts.max())
    fp32 = 8 * f.eps * r * o["dW_sq"].sqrt() + _acc(2 * n) * 2 * o["dW_abs"]
    _within("dW", got, o["dW"], fp32 + r * (o["dW"].abs() + fp32) + f.smallest_normal * r)


@pytest.mark.parametrize("T,E,K,H", [(1, 4, 2, 128), (5, 8, 1, 256), (129, 5, 3, 192), (300, 64, 8, 64), (700, 8, 2, 320),
                                     (513, 7, 4, 512), (260, 6, 2, 1024), (5003, 4, 2, 128), (9001, 13, 1, 640)])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_weight_gradient_is_that_of_fp32_terms(T, E, K, H, dtype):
    x, W, b, g = _data(T, E, K, H, dtype)
    routing, w = _routing(T, E, K)
    for v in (w, torch.ones_like(w), -w.round(decimals=1)):
        o = _reference(x, W, b, g, routing.expert_idx, v)
        _check_dW(_bwd(x, W, b, g, routing, v, ("dW",))["dW"], o, routing)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
@pytest.mark.parametrize("one", [False, True], ids=["weights", "ones"])
def test_infinities_in_the_weight_gradient_are_those_of_the_formula(one, dtype):
    """An infinite x or d_out makes its column or row of dW infinite, with the sign of the other factor,
    and leaves everything else as it was."""
    T, E, K, H = 300, 5, 2, 128
    x, W, b, g = _data(T, E, K, H, dtype)
    routing, w = _routing(T, E, K)
    w = torch.ones_like(w) if one else w
    hit = torch.zeros(E, dtype=torch.bool, device="cuda")
    hit[routing.expert_idx.view(T, K)[7].long()] = True
    assert (g[7] != 0).all() and (x[7] != 0).all() and hit.any() and not hit.all()
    want = _bwd(x, W, b, g, routing, w, ("dW",))["dW"]
    for name in ("x", "g"):
        bx, bg = x.clone(), g.clone()
        (bx if name == "x" else bg)[7, 3] = float("inf")
        got = _bwd(bx, W, b, bg, routing, w, ("dW",))["dW"]
        line = got[:, :, 3] if name == "x" else got[:, 3, :]
        signs = torch.sign((g if name == "x" else x)[7].float())
        assert torch.equal(line[hit].float(), (signs * float("inf")).expand(int(hit.sum()), H))
        line[hit] = (want[:, :, 3] if name == "x" else want[:, 3, :])[hit]
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [40000, 50000])
def test_two_experts_without_expert_indices(T):
    """Without a bias expert_idx may be left out: the tokens are then not grouped by it."""
    E, K, H = 5, 2, 128
    x, W, _, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    bare = ops.Routing(None, routing.counts, routing.offsets, routing.perm)
    o = _reference(x, W, None, g, routing.expert_idx, w)
    _check_rows("y", _fwd(x, W, None, bare, w), o, K, H)
    _check_bwd(_bwd(x, W, None, g, bare, w), o, bare, K, H)


@pytest.mark.parametrize("T,E,K,H,dtype", [(40, 3, 2, 4096, BF16), (300, 2, 1, 4096, F16), (130, 2, 2, 2048, F16),
                                           (100000, 8, 1, 256, BF16), (60000, 8, 2, 256, F16), (20001, 12, 8, 128, BF16),
                                           (9000, 20, 16, 64, F16), (100001, 3, 2, 64, BF16), (51001, 32, 2, 128, BF16)])
def test_the_ends_of_the_range(T, E, K, H, dtype):
    """The widest rows, one expert for many tokens, many experts a token, fp16 in the grouped path."""
    x, W, b, g = _data(T, E, K, H, dtype)
    routing, w = _routing(T, E, K, 5, 0.5)
    o = _reference(x, W, b, g, routing.expert_idx, w)
    _check_rows("y", _fwd(x, W, b, routing, w), o, K, H)
    got = _bwd(x, W, b, g, routing, w)
    _check_bwd(got, o, routing, K, H)
    _check_dW(got["dW"], o, routing)


@pytest.mark.parametrize("want", [("d_x",), ("d_weights",), ("dW",), ("db",), ("db", "d_weights")], ids="+".join)
def test_some_outputs_of_grouped_tokens(want):
    T, E, K, H = 50000, 5, 2, 192
    x, W, b, g = _data(T, E, K, H, BF16)
    routing, w = _routing(T, E, K)
    o = _reference(x, W, b, g, routing.expert_idx, w)
    _check_bwd(_bwd(x, W, b, g, routing, w, want), o, routing, K, H, want)


def test_a_captured_fp16_backward_follows_its_inputs():
    """The powers of two that the terms of dW are staged with come from each call's own inputs."""
    T, E, K, H = 700, 5, 2, 128
    x, W, b, g = _data(T, E, K, H, F16)
    routing, w = _routing(T, E, K)
    ws = ops.new_topk_workspace(T, E, K, H, "cuda")
    outs = {k: v.clone() for k, v in _bwd(x, W, b, g, routing, w, ws=ws).items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_topk_bwd(x, W, b, g, routing, w, *(outs[k] for k in OUTS), ws)
    first = g.clone()
    for scale in (2.0 ** -12, 2.0 ** 8, 1.0):
        g.copy_(first * scale)
        graph.replay()
        torch.cuda.synchronize()
        want = _bwd(x, W, b, g, routing, w)
        assert all(torch.equal(outs[k], want[k]) for k in OUTS)
        o = _reference(x, W, b, g, routing.expert_idx, w)
        _check_dW(outs["dW"], o, routing)
