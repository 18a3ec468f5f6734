"""moe_topk_route / moe_topk_route_bwd against the definition in 64 bits (numpy).

Choices, counts, offsets and perm are compared exactly. Tolerances of the weights and
gradients, in units of u = 2^-24: an exponential of (l - m) is off by 4 (its own
2 ulp) plus |l - m| (the rounding of its argument), relative; sums of at most 256
terms add at most 16 + 4 roundings, the few products and quotients around them 12. So
a weight is off by at most (2 D + 48) u of itself, D the row's largest |l - m| with a
finite l (once for the term, once for the sum), and a gradient by at most that share of
the sum of the magnitudes it is made of, twice (weight and inner sum), plus its own
rounding to the type of the logits.
"""
import numpy as np
import pytest
import torch

import oracle
from bwd_route_b200 import ops
from gpu_harness import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SOFT, SIG = ops.MOE_SCORE_SOFTMAX, ops.MOE_SCORE_SIGMOID
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _scores(l, score):
    with np.errstate(all="ignore"):
        if score == SIG:
            q = np.exp(-np.abs(l))
            return np.where(l >= 0, 1 / (1 + q), q / (1 + q))
        m = l.max(1, keepdims=True)
        p = np.exp(l - np.where(np.isneginf(m), 0, m))
        z = p.sum(1, keepdims=True)
        return p / np.where(z == 0, 1, z)


def _select(l, rule, bias):
    """The definition, one expert after the other."""
    T, E = l.shape
    S = E // rule.groups
    s = _scores(l, rule.score)
    v = s if bias is None else s + bias.astype(np.float64)
    order = l if bias is None else v
    masked = np.isnan(l) | np.isneginf(l) | np.isnan(order)
    order, v = np.where(masked, -np.inf, order), np.where(masked, -np.inf, v)
    rows = np.arange(T)
    inside = np.ones((T, E), bool)
    if rule.groups > 1:
        by = order if rule.group_best == 1 else v
        g = np.sort(by.reshape(T, rule.groups, S), 2)[:, :, S - rule.group_best:].sum(2)
        kept = np.argsort(-g, 1, kind="stable")[:, :rule.top_groups]
        inside = np.zeros((T, rule.groups), bool)
        np.put_along_axis(inside, kept, True, 1)
        inside = np.repeat(inside, S, 1)
    idx = np.empty((T, rule.K), np.int64)
    # order of preference: inside before outside, then the value, then the index
    for t in rows:
        c = np.flatnonzero(inside[t])
        idx[t] = c[np.argsort(-order[t, c], kind="stable")[:rule.K]]
    return idx


def _weights(l, idx, rule):
    k = np.take_along_axis(l, idx, 1)
    if rule.renorm:
        low = np.minimum(k, 0) if rule.score == SIG else k
        m = low.max(1, keepdims=True)
        with np.errstate(all="ignore"):
            p = np.exp(low - np.where(np.isneginf(m), 0, m))
            p = p / (1 + np.exp(-np.abs(k))) if rule.score == SIG else p
        z = p.sum(1, keepdims=True)
        return rule.scale * p / np.where(z == 0, 1, z)
    return rule.scale * np.take_along_axis(_scores(l, rule.score), idx, 1)


def _spread(l):
    f = np.where(np.isfinite(l), l, 0.0)
    return 2 * np.abs(f).max(1, keepdims=True)  # |l - m| and |l| of a row are at most this


def _run(logits, rule, bias=None, ws=None, stream=None):
    T, E, K = logits.shape[0], rule.E, rule.K
    i = torch.int32
    g = {"expert_idx": Guarded(T * K, i), "counts": Guarded(E, i), "offsets": Guarded(E + 1, i),
         "perm": Guarded(T * K, i), "weights": Guarded(T * K, F32, (T, K))}
    ws = ops.new_topk_workspace(T, E, K, 0, "cuda") if ws is None else ws
    r = ops.Routing(*(g[k].t for k in ("expert_idx", "counts", "offsets", "perm")))
    ops.moe_topk_route(logits, rule, bias, r, g["weights"].t, ws, stream)
    torch.cuda.synchronize()
    assert all(x.guards_intact() for x in g.values())
    return {k: x.host() for k, x in g.items()}, r


def _check(logits, rule, bias=None):
    got, routing = _run(logits, rule, bias)
    T, K, E = logits.shape[0], rule.K, rule.E
    l = logits.double().cpu().numpy()
    b = None if bias is None else bias.cpu().numpy()
    idx = _select(l, rule, b)
    np.testing.assert_array_equal(got["expert_idx"].reshape(T, K), idx)
    flat = idx.reshape(-1)
    counts = np.bincount(flat, minlength=E)
    np.testing.assert_array_equal(got["counts"], counts)
    np.testing.assert_array_equal(got["offsets"], np.concatenate([[0], np.cumsum(counts)]))
    np.testing.assert_array_equal(got["perm"], np.argsort(flat, kind="stable"))
    want = _weights(l, idx, rule)
    tol = (2 * _spread(l) + 48) * U * np.abs(want) + 2.0 ** -126
    w = got["weights"].astype(np.float64)
    assert np.array_equal(np.isnan(w), np.isnan(want))
    assert np.all((np.abs(w - want) <= tol) | np.isnan(want)), np.nanmax(np.abs(w - want) / tol)
    return got, routing


def _logits(T, E, dtype, seed, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, E, generator=g, device="cuda") * spread).to(dtype), \
        torch.randn(E, generator=g, device="cuda") * 0.1


R = ops.TopKRule
RULES = [
    R(1, 1), R(2, 2, SIG, True), R(4, 2), R(8, 1, SOFT, False, 0.5), R(8, 2, SOFT, True), R(8, 8, SIG, True, 2.5),
    R(7, 3, SIG), R(15, 15, SOFT, True), R(16, 4, SIG, True, 1.0, 4, 2, 2), R(16, 15, SOFT, False, 1.0, 16, 15, 1),
    R(17, 5, SOFT, True), R(32, 16, SIG, True), R(32, 6, SOFT, False, 16.0, 8, 3, 1), R(33, 4, SIG, True, 1.0, 11, 4, 2),
    R(60, 4, SOFT, True), R(60, 6, SIG, True, 2.5, 6, 3, 2), R(64, 8, SOFT, True), R(64, 6, SIG, True, 1.0, 8, 4, 1),
    R(65, 2, SIG), R(100, 10, SOFT, True, 1.0, 20, 6, 2), R(128, 8, SIG, True, 2.5, 8, 4, 2), R(128, 1), R(160, 6, SOFT, False, 16.0, 8, 3, 1),
    R(200, 16, SOFT, True), R(255, 8, SIG, True), R(256, 8, SIG, True, 2.5, 8, 4, 2), R(256, 8, SOFT, True, 1.0, 32, 5, 2),
    R(256, 16, SOFT), R(256, 4, SIG, False, 1.0, 2, 1, 1),
]


def _id(r):
    return f"E{r.E}K{r.K}{'sig' if r.score == SIG else 'soft'}{'n' if r.renorm else ''}G{r.groups}-{r.top_groups}-{r.group_best}"


@pytest.mark.parametrize("with_bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("rule", RULES, ids=_id)
def test_route(rule, with_bias):
    for T, dtype in ((1, F32), (2, BF16), (33, F16), (129, F32), (700, BF16), (3001, F32)):
        logits, bias = _logits(T, rule.E, dtype, T + rule.E)
        _check(logits, rule, bias if with_bias else None)


@pytest.mark.parametrize("E,K,T", [(8, 2, 100003), (64, 6, 20479), (256, 8, 9001), (16, 16, 4097)])
def test_route_many_tokens(E, K, T):
    logits, bias = _logits(T, E, F32, 5)
    _check(logits, R(E, K, SIG, True), bias)
    _check(logits, R(E, K, SOFT, True))


@pytest.mark.parametrize("E,K,groups,top", [(256, 8, 8, 2), (256, 8, 4, 1), (192, 8, 6, 2), (256, 16, 8, 2), (256, 16, 2, 1), (128, 8, 8, 1)])
@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
def test_few_groups_that_stay(E, K, groups, top, score):
    """As few lanes hold the experts that stay as a token chooses experts, or fewer."""
    for T, dtype in ((100, F32), (3000, BF16)):
        logits, bias = _logits(T, E, dtype, E + K)
        for best in (1, 2):
            _check(logits, R(E, K, score, True, 1.0, groups, top, best), bias)
            _check(logits, R(E, K, score, False, 1.0, groups, top, best))


@pytest.mark.parametrize("rule", [r for r in RULES if r.E >= 4], ids=_id)
def test_equal_values_go_to_the_lowest_index(rule):
    g = torch.Generator(device="cuda").manual_seed(1)
    for T in (50, 2000):
        logits = torch.randint(-1, 2, (T, rule.E), generator=g, device="cuda").float()
        logits[0] = 0.0
        logits[1] = -0.0
        logits[1, ::2] = 0.0  # -0 and +0 are equal
        _check(logits, rule)
        _check(logits, rule, torch.zeros(rule.E, device="cuda"))
        _check(logits, rule, (torch.arange(rule.E, device="cuda") % 3).float() * 0.25)


@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 48, 256])
def test_values_that_fp32_cannot_tell_apart(E, score):
    """The bias lifts every expert's v to the same level up to its own rounding, about 1e-8: the
    order is decided by what fp64 still sees."""
    logits, _ = _logits(1, E, F32, 9, 1.0)
    s = _scores(logits.double().cpu().numpy(), score)[0]
    bias = torch.tensor(1.25 - s, device="cuda", dtype=F32)
    v = np.sort(s + bias.double().cpu().numpy())
    assert np.diff(v).max() < 2.0 ** -22 and np.diff(v).min() > 1e-14
    logits = logits.expand(40, E).contiguous()
    for G, TG, best in ((1, 1, 1), (4, 2, 2), (2, 1, 1)):
        _check(logits, R(E, 4, score, True, 1.0, G, TG, best), bias)


@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [5, 200, 3000])
@pytest.mark.parametrize("E,K,groups", [(3, 1, 1), (3, 2, 1), (40, 6, 1), (64, 1, 1), (64, 6, 8), (65, 4, 1), (65, 1, 1), (256, 1, 1),
                                        (256, 8, 1), (256, 8, 8)])
def test_equal_values_at_the_border_beside_a_larger_one(E, K, groups, T, score):
    """Exact ties across place K, and experts behind them that fp32 cannot tell from the tie: the largest
    wins whatever its index. Sigmoid: bf16 steps near saturation under a bias of zero; softmax: logits a few
    2^-24 E apart under a bias of 4, whose last place is 2^-21."""
    g = torch.Generator(device="cuda").manual_seed(E + T)
    if score == SIG:
        logits = 10 + torch.randint(0, 96, (T, E), generator=g, device="cuda").float() / 16
        logits[0] = 14.0
        logits[0, E - 1] = 14.0625
        bias = torch.zeros(E, device="cuda")
    else:
        logits = torch.randint(0, 4, (T, E), generator=g, device="cuda").float() * (E * 2.0 ** -24)
        logits[0] = 0.0
        logits[0, E - 1] = E * 2.0 ** -24
        bias = torch.full((E,), 4.0, device="cuda")
    # every other row has K + 3 of them, the rest far below
    few = torch.rand(T, E, generator=g, device="cuda").argsort(1).argsort(1) < K + 3
    logits[1::2] -= 16.0 * ~few[1::2]
    logits = logits.to(BF16 if score == SIG else F32)
    rule = R(E, K, score, True, 1.0, groups, max(1, groups // 2), 1 if groups == 1 else 2)
    got, _ = _check(logits, rule, bias)
    if groups == 1:
        assert got["expert_idx"][0] == E - 1
        got, _ = _check(logits, rule, torch.where(torch.arange(E, device="cuda") % 3 == 0, bias, bias + 0.25))


@pytest.mark.parametrize("rule", [R(8, 3), R(8, 3, SOFT, True), R(40, 6, SIG, True), R(64, 6, SIG, True, 2.5, 8, 4, 2),
                                  R(256, 8, SOFT, True, 1.0, 8, 3, 1)], ids=_id)
@pytest.mark.parametrize("with_bias", [False, True], ids=["plain", "bias"])
def test_masked_experts(rule, with_bias):
    """-inf masks: some experts, all but one, all but K - 1, a whole group, and whole rows; and the
    type's lowest value, which is a number like any other."""
    E, K = rule.E, rule.K
    logits, bias = _logits(64, E, F32, 3)
    inf = float("inf")
    logits[1, ::2] = -inf
    logits[2, 1:] = -inf
    logits[3, :E - K + 1] = -inf
    logits[4] = -inf
    logits[5, :E // rule.groups] = -inf
    logits[6:20][torch.rand(14, E, generator=torch.Generator().manual_seed(2)).cuda() < 0.8] = -inf
    logits[21] = torch.finfo(F32).min
    logits[22, 3:] = torch.finfo(F32).min
    logits[63] = -inf
    _check(logits, rule, bias if with_bias else None)
    got, _ = _run(logits, rule, bias if with_bias else None)
    assert (got["weights"][4] == 0).all() and (got["weights"][63] == 0).all()


def test_nan_is_never_chosen_over_a_number():
    rule = R(8, 3, SIG, True)
    logits, _ = _logits(5, 8, F32, 3)
    logits[0, 2] = logits[1, :5] = logits[2, 1:] = float("nan")
    l = logits.double().cpu().numpy()
    got, _ = _run(logits, rule)
    idx = got["expert_idx"].reshape(5, 3)
    np.testing.assert_array_equal(idx, _select(l, rule, None))
    assert 2 not in idx[0] and set(idx[1]) == {5, 6, 7} and idx[2].tolist() == [0, 1, 2]
    assert np.isfinite(got["weights"][[0, 1, 3, 4]]).all() and np.isnan(got["weights"][2]).all()


@pytest.mark.parametrize("with_bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 40, 100, 256])
@pytest.mark.parametrize("T", [5, 400])
def test_rows_with_a_nan_or_an_infinity(T, E, score, renorm, with_bias):
    """Without a bias the logits alone are compared; with one, a softmax row with a NaN or +inf has only
    NaN to compare, and its experts come by index."""
    logits, bias = _logits(T, E, F32, 9)
    logits[0, 3], logits[1, 5], logits[3, E - 1] = float("nan"), float("inf"), float("inf")
    got, _ = _check(logits, R(E, 4, score, renorm), bias if with_bias else None)
    if with_bias and score == SOFT:
        assert (got["expert_idx"].reshape(T, 4)[[0, 1, 3]] == np.arange(4)).all()


@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 40, 100, 256])
@pytest.mark.parametrize("T", [5, 3000])
def test_a_nan_in_the_bias_masks_its_expert(T, E, score):
    logits, bias = _logits(T, E, F32, 9)
    bias[3] = float("nan")
    got, _ = _run(logits, R(E, E, score) if E == 8 else R(E, 4, score), bias)
    idx = got["expert_idx"].reshape(T, -1)
    if E == 8:  # all are chosen, the masked one last
        assert (idx[:, -1] == 3).all()
    else:
        assert (idx != 3).all()
    assert ((idx >= 0) & (idx < E)).all()


def test_weights_stay_finite_where_scores_underflow():
    logits = torch.full((3, 16), -300.0, device="cuda")
    logits[0, 3], logits[1, 5], logits[2, 0] = -250.0, -299.5, 900.0
    for score in (SOFT, SIG):
        _check(logits, R(16, 4, score, True))
    got, _ = _run(logits, R(16, 4, SIG, True))
    assert abs(got["weights"].sum(1) - 1).max() < 1e-6


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("E,ld,shift", [(64, 80, 0), (64, 65, 0), (60, 64, 0), (8, 8, 1), (256, 256, 2), (33, 40, 3)])
def test_strided_and_unaligned_rows(E, ld, shift, dtype):
    T = 300
    logits, bias = _logits(T, E, dtype, 4)
    buf = torch.zeros(T * ld + shift, dtype=dtype, device="cuda")[shift:].view(T, ld)
    buf[:, :E] = logits
    rule = R(E, 4, SIG, True)
    a, _ = _run(buf[:, :E], rule, bias)
    b, _ = _run(logits, rule, bias)
    for k in a:
        assert a[k].tobytes() == b[k].tobytes(), k


def test_one_expert_agrees_with_the_top_1_routing():
    T, E = 5000, 8
    logits, _ = _logits(T, E, F32, 11)
    got, routing = _run(logits, R(E, 1))
    ref = ops.Routing.empty(T, E, "cuda")
    ops.moe_top1_route(logits, T, 1, E, ref, ops.new_workspace(T, E, 0, "cuda"))
    for k in ("expert_idx", "counts", "offsets", "perm"):
        assert torch.equal(getattr(routing, k), getattr(ref, k)), k


def test_routing_passes_the_routing_check():
    for T, E, K in ((37, 8, 2), (9000, 32, 5)):
        logits, _ = _logits(T, E, F32, 12)
        _, routing = _run(logits, R(E, K))
        ws = ops.new_workspace(T * K, E, 0, "cuda")
        ops.moe_top1_check_routing(routing, T * K, E, ws)
        assert ops.moe_top1_device_flags(ws) == 0


def test_no_tokens():
    got, _ = _run(torch.empty(0, 12, device="cuda"), R(12, 3))
    assert not got["counts"].any() and not got["offsets"].any()


def test_repeats_streams_and_graphs():
    """One workspace, two sizes through it in turn; then a captured call replayed with new logits."""
    rule = R(64, 6, SIG, True, 2.5, 8, 4, 2)
    ws = ops.new_topk_workspace(4000, 64, 6, 0, "cuda")
    cases = [_logits(T, 64, F32, T) for T in (4000, 9, 4000, 257)]
    first = [_run(l, rule, b, ws)[0] for l, b in cases]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [_run(l, rule, b, ws)[0] for l, b in cases]
    for a, b in zip(first, again):
        assert all(a[k].tobytes() == b[k].tobytes() for k in a)
    logits, bias = cases[0][0].clone(), cases[0][1]
    r = ops.Routing.empty(4000 * 6, 64, "cuda")
    w = torch.empty(4000, 6, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_topk_route(logits, rule, bias, r, w, ws)
    for l, b in (cases[2], (cases[0][0].flip(0).contiguous(), bias)):
        logits.copy_(l)
        bias.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want, _ = _run(logits, rule, bias)
        assert w.cpu().numpy().tobytes() == want["weights"].tobytes()
        assert r.perm.cpu().numpy().tobytes() == want["perm"].tobytes()


# ---------------------------------------------------------------- gradient
def _grad(l, idx, g, rule):
    """(gradient, sum of the magnitudes it is made of) in 64 bits."""
    g = rule.scale * g
    out, mag = np.zeros_like(l), np.zeros_like(l)
    if rule.renorm:
        r = _weights(l, idx, R(rule.E, rule.K, rule.score, True))
        dot, adot = (g * r).sum(1, keepdims=True), (np.abs(g) * r).sum(1, keepdims=True)
        with np.errstate(all="ignore"):
            f = 1 / (1 + np.exp(np.take_along_axis(l, idx, 1))) if rule.score == SIG else 1.0
        np.put_along_axis(out, idx, r * (g - dot) * f, 1)
        np.put_along_axis(mag, idx, r * (np.abs(g) + adot) * f, 1)
        return out, mag
    s = _scores(l, rule.score)
    v = np.zeros_like(l)
    np.put_along_axis(v, idx, g, 1)
    if rule.score == SIG:
        with np.errstate(all="ignore"):
            one = 1 / (1 + np.exp(l))  # 1 - s
        return v * s * one, np.abs(v) * s * one
    return s * (v - (s * v).sum(1, keepdims=True)), s * (np.abs(v) + (s * np.abs(v)).sum(1, keepdims=True))


def _check_grad(logits, idx, d_weights, rule, old=None):
    T, E = logits.shape
    d = torch.full((T * E + 32,), 7.0, dtype=logits.dtype, device="cuda")
    out = d[16:16 + T * E].view(T, E)
    if old is not None:
        out.copy_(old)
    ops.moe_topk_route_bwd(logits, rule, idx, d_weights, out, old is not None)
    torch.cuda.synchronize()
    assert (d[:16] == 7).all() and (d[16 + T * E:] == 7).all()
    l = logits.double().cpu().numpy()
    want, mag = _grad(l, idx.view(T, rule.K).cpu().numpy().astype(np.int64), d_weights.double().cpu().numpy(), rule)
    tol = 2 * (2 * _spread(l) + 48) * U * mag
    if old is not None:
        o = old.double().cpu().numpy()
        want, tol = want + o, tol + U * (np.abs(o) + np.abs(want))
    fi = torch.finfo(logits.dtype)
    tol = tol + fi.eps / 2 * (np.abs(want) + tol) + fi.smallest_normal * fi.eps / 2 + 2.0 ** -126
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
    return got


@pytest.mark.parametrize("rule", RULES, ids=_id)
def test_gradient(rule):
    for T, dtype in ((1, F32), (3, F16), (37, BF16), (501, F32), (5000, BF16)):
        logits, bias = _logits(T, rule.E, dtype, T + rule.E)
        idx = torch.tensor(_select(logits.double().cpu().numpy(), rule, bias.cpu().numpy()), dtype=torch.int32,
                           device="cuda")
        dw = torch.randn(T, rule.K, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
        _check_grad(logits, idx, dw, rule)
        _check_grad(logits, idx.view(-1), dw, rule, torch.randn(T, rule.E, device="cuda").to(dtype))


@pytest.mark.parametrize("rule", [R(8, 3), R(8, 3, SOFT, True), R(8, 3, SIG), R(8, 3, SIG, True)], ids=_id)
def test_gradient_of_masked_rows_is_zero_there(rule):
    logits, _ = _logits(4, 8, F32, 3)
    logits[1, 2:] = -float("inf")
    logits[2] = -float("inf")
    idx = torch.tensor(_select(logits.double().cpu().numpy(), rule, None), dtype=torch.int32, device="cuda")
    got = _check_grad(logits, idx, torch.ones(4, 3, device="cuda") * torch.tensor([1.0, -2, 3], device="cuda"), rule)
    assert not got[2].any() and not got[1, 2:].any()


@pytest.mark.parametrize("rule", [R(12, 3, SOFT, False, 2.0), R(12, 3, SOFT, True, 2.0), R(12, 3, SIG, False, 2.0),
                                  R(12, 3, SIG, True, 2.0)], ids=_id)
def test_gradient_against_differences(rule):
    """Central differences of sum(c * weights) through the forward, h = 1/64, over logits whose choice a
    step of h does not change. The weights are within 2e-6 of the formula at this spread, so a difference
    is off by at most 3 * 2 * 2e-6 * 2 * |c| / (1/32) < 2e-3 and by h^2 / 6 * |third derivative| < 1e-3."""
    T, E, h = 4, 12, 1.0 / 64
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t)) for t in range(T)]).cuda().float() * 0.25
    c = torch.randn(T, 3, generator=g, device="cuda").clamp(-2, 2)
    base, routing = _run(logits, rule)
    d = torch.empty_like(logits)
    ops.moe_topk_route_bwd(logits, rule, routing.expert_idx, c, d)
    for t in range(T):
        for e in range(E):
            at = []
            for s in (h, -h):
                moved = logits.clone()
                moved[t, e] += s
                got, _ = _run(moved, rule)
                assert np.array_equal(got["expert_idx"], base["expert_idx"])
                at.append((got["weights"].astype(np.float64) * c.double().cpu().numpy()).sum())
            assert abs((at[0] - at[1]) / (2 * h) - d[t, e].item()) <= 3e-3


@pytest.mark.parametrize("score", [SOFT, SIG], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [1, 8, 40, 256])
def test_one_renormalised_expert_has_no_gradient(score, E):
    """Its weight is the scale whatever the logits: the gradient is exactly 0."""
    rule = R(E, 1, score, True, 2.5)
    logits, _ = _logits(500, E, F32, 8)
    got, routing = _run(logits, rule)
    assert (got["weights"] == 2.5).all()
    d = torch.ones_like(logits)
    ops.moe_topk_route_bwd(logits, rule, routing.expert_idx, torch.randn(500, 1, device="cuda"), d)
    assert not d.any()


def test_gradient_leaves_out_experts_outside_the_row():
    rule = R(8, 2, SOFT, True)
    logits, _ = _logits(3, 8, F32, 3)
    idx = torch.tensor([[0, 1], [-1, 8], [1 << 30, 2]], dtype=torch.int32, device="cuda")
    d = torch.empty_like(logits)
    ops.moe_topk_route_bwd(logits, rule, idx, torch.ones(3, 2, device="cuda"), d)
    assert not d[1].any() and torch.isfinite(d).all()


def test_gradient_of_strided_logits():
    rule = R(20, 4, SOFT)
    logits, _ = _logits(50, 20, F32, 3)
    buf = torch.zeros(50, 33, device="cuda")
    buf[:, :20] = logits
    idx = torch.tensor(_select(logits.double().cpu().numpy(), rule, None), dtype=torch.int32, device="cuda")
    _check_grad(buf[:, :20], idx, torch.randn(50, 4, device="cuda"), rule)
