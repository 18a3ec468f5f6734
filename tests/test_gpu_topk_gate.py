"""A step of the top-k block, all its calls together, against 64-bit autograd of the
same chain (the chosen experts held fixed).

Tolerances, 2-norm of the difference over 2-norm of the result. Every rounding to the
16-bit type moves its vector by at most r = eps / 2 of itself. The maps between the
roundings (W of entries N(0, 1/H), the norm's Jacobian, sums over tokens) are random and
keep a perturbation's share of the norm within a factor of 1.5. Roundings on the way:
y: normed, y. d_weights, d_logits (fp32): normed. d_x: normed, d_normed, d_x. dW: normed,
w g, dW. db: db. dgamma, dbeta: normed (through n), d_normed, the result.
"""
import pytest
import torch

from bwd_route_b200 import ops
from bwd_route_b200.topk_gate import MoETopKGate

pytestmark = pytest.mark.gpu

SOFT, SIG = ops.MOE_SCORE_SOFTMAX, ops.MOE_SCORE_SIGMOID
ROUNDINGS = {"y": 2, "d_weights": 1, "d_logits": 1, "d_x": 3, "dW": 3, "db": 1, "dgamma": 3, "dbeta": 2}


def _make(T, H, rule, dtype, seed=0, norm=True, bias=True, balance=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    W = (rand(rule.E, H, H) / H ** 0.5).to(dtype)
    b = (rand(rule.E, H) * 0.2).to(dtype) if bias else None
    gamma, beta = ((1 + 0.2 * rand(H)).to(dtype), (0.2 * rand(H)).to(dtype)) if norm else (None, None)
    gate = MoETopKGate(W, b, T, rule, gamma, beta, norm, balance_bias=0.1 * rand(rule.E) if balance else None)
    return gate, (rand(T, H) * 1.5 + 0.3).to(dtype), rand(T, rule.E), rand(T, H).to(dtype)


def _reference(gate, x, logits, d_y):
    rule, T = gate.rule, gate.T
    leaf = lambda t: None if t is None else t.double().requires_grad_()  # noqa: E731
    x, logits, W, b, gamma, beta = map(leaf, (x, logits, gate.W, gate.bias, gate.gamma, gate.beta))
    h = x
    if gate.norm:
        h = (x - x.mean(1, keepdim=True)) / (x.var(1, correction=0, keepdim=True) + gate.eps).sqrt()
        h = h if gamma is None else h * gamma + beta
    s = torch.softmax(logits, 1) if rule.score == SOFT else torch.sigmoid(logits)
    idx = gate.routing.expert_idx.view(T, rule.K).long()
    w = s.gather(1, idx)
    w = rule.scale * (w / w.sum(1, keepdim=True) if rule.renorm else w)
    w.retain_grad()
    y = torch.zeros_like(x)
    for e in range(rule.E):
        comb = (w * (idx == e)).sum(1, keepdim=True)
        z = h @ W[e].T
        y = y + comb * (z if b is None else z + b[e])
    y.backward(d_y.double())
    grad = lambda t: None if t is None else t.grad  # noqa: E731
    return {"y": y.detach(), "d_x": x.grad, "d_logits": logits.grad, "dW": W.grad, "db": grad(b), "dgamma": grad(gamma),
            "dbeta": grad(beta), "d_weights": w.grad, "weights": w.detach()}


def _check(gate, x, logits, d_y):
    want = _reference(gate, x, logits, d_y)
    r = torch.finfo(x.dtype).eps / 2
    for k, n in ROUNDINGS.items():
        if want[k] is None:
            continue
        got = getattr(gate, k).double()
        off = (got - want[k]).norm() / want[k].norm()
        assert off <= 1.5 * n * r, (k, off.item(), 1.5 * n * r)


@pytest.mark.parametrize("rule", [ops.TopKRule(8, 2, SOFT, True), ops.TopKRule(8, 2), ops.TopKRule(16, 4, SIG, True, 2.5, 4, 2, 2),
                                  ops.TopKRule(5, 1, SIG), ops.TopKRule(40, 6, SIG, False)], ids=lambda r: f"E{r.E}K{r.K}")
@pytest.mark.parametrize("T,H,dtype", [(1, 64, torch.bfloat16), (37, 128, torch.float16), (1025, 256, torch.bfloat16),
                                       (300, 320, torch.float16)], ids=str)
def test_step(rule, T, H, dtype):
    gate, x, logits, d_y = _make(T, H, rule, dtype, balance=rule.groups > 1)
    gate.step(x, logits, d_y)
    torch.cuda.synchronize()
    assert ops.moe_top1_device_flags(gate.ws) == 0
    _check(gate, x, logits, d_y)


@pytest.mark.parametrize("norm,bias", [(False, True), (True, False), (False, False)])
def test_step_without_norm_or_bias(norm, bias):
    gate, x, logits, d_y = _make(200, 128, ops.TopKRule(6, 2, SOFT, True), torch.bfloat16, 1, norm, bias)
    gate.step(x, logits, d_y)
    torch.cuda.synchronize()
    want = _reference(gate, x, logits, d_y)
    assert (want["db"] is None) == (not bias)
    _check(gate, x, logits, d_y)


def test_two_gates_at_once_on_two_streams():
    """A workspace each: steps that overlap on the GPU give what they give alone."""
    made = [_make(4000, 256, ops.TopKRule(8, 2, SOFT, True), torch.bfloat16, s) for s in (1, 2)]
    outs = ("y", "d_x", "d_logits", "dW", "db", "dgamma", "dbeta")
    alone = []
    for gate, *a in made:
        gate.step(*a)
        torch.cuda.synchronize()
        alone.append({k: getattr(gate, k).clone() for k in outs})
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(5):
        for (gate, *a), s in zip(made, streams):
            gate.step(*a, stream=s)
    torch.cuda.synchronize()
    for (gate, *_), want in zip(made, alone):
        assert all(torch.equal(getattr(gate, k), want[k]) for k in outs)


def test_a_captured_step_follows_its_inputs():
    gate, x, logits, d_y = _make(700, 128, ops.TopKRule(16, 4, SIG, True, 2.5, 4, 2, 2), torch.bfloat16, 3, balance=True)
    gate.step(x, logits, d_y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gate.step(x, logits, d_y)
    for seed in (5, 6):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (x, logits, d_y, gate.balance_bias):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda") * (0.1 if t is gate.balance_bias else 1.0))
        graph.replay()
        torch.cuda.synchronize()
        _check(gate, x, logits, d_y)
        idx = gate.routing.expert_idx.clone()
        y = gate.y.clone()
        gate.forward(x, logits)
        assert torch.equal(gate.routing.expert_idx, idx) and torch.equal(gate.y, y)


def test_logit_gradients_add_up_with_the_balance_loss():
    """The aux loss writes its gradient, the block adds the one through the weights."""
    T, E = 640, 8
    gate, x, logits, d_y = _make(T, 128, ops.TopKRule(E, 2, SOFT, True), torch.bfloat16, 4)
    gate.step(x, logits, d_y)
    alone = gate.d_logits.clone()
    lam, loss, mean_p = torch.full((1,), 0.05, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(E, device="cuda")
    aux = torch.empty_like(gate.d_logits)
    ws = ops.new_workspace(T, E, 0, "cuda")
    for out in (aux, gate.d_logits):
        ops.moe_aux_loss_fwd_bwd(logits, gate.routing.counts, T, 1, E, lam, out, loss, mean_p, None, ws)
    gate.backward(x, logits, d_y, accumulate_logits=True)
    torch.cuda.synchronize()
    assert torch.equal(gate.d_logits, aux + alone)


def test_refusals():
    W = torch.zeros(4, 64, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        MoETopKGate(W, None, 8, ops.TopKRule(5, 2))
    with pytest.raises(ValueError):
        MoETopKGate(W, None, 8, ops.TopKRule(4, 2), gamma=torch.ones(64, device="cuda"), norm=False)
    gate = MoETopKGate(W, None, 8, ops.TopKRule(4, 2))
    x, logits = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 4, device="cuda")
    with pytest.raises(TypeError):
        gate.forward(x.float(), logits)
    with pytest.raises(ValueError):
        gate.forward(x[:7], logits)
    with pytest.raises(ValueError):
        gate.forward(x, logits[:, :3])
    with pytest.raises(ValueError):
        gate.forward(x, logits.cpu())
    with pytest.raises(TypeError):
        ops.moe_topk_fwd(x.float(), W.float(), None, gate.routing, gate.weights, gate.y.float(), gate.ws)
    with pytest.raises(ValueError):
        ops.moe_topk_fwd(x.t(), W, None, gate.routing, gate.weights, gate.y, gate.ws)
    with pytest.raises(ops.MoeError) as err:
        ops.moe_topk_fwd(x, W, None, gate.routing, gate.weights, gate.y, gate.ws[:512])
    assert err.value.status_name == "MOE_ERR_WORKSPACE"
    with pytest.raises(ops.MoeError) as err:
        ops.moe_topk_fwd(x, W, None, gate.routing, gate.weights, x, gate.ws)
    assert err.value.status_name == "MOE_ERR_ALIAS"
