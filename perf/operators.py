"""The operators of the top-k mixture-of-experts block, case by case: the router
(selection, weights, dispatch lists) and its gradient, the experts' weighted
product and its gradients, and the layer norm in front of them, both directions.

listed() and draw() give cases, prepare() the inputs of one, run() one pass (in
plain torch, or through bwd_route_b200.ops where `own` is true), work() the bytes
and operations a pass cannot do without, exact() its result in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
EPS = 1e-5


# ---------------------------------------------------------------- cases
def _route(name, T, E, K, dtype, score, renorm, scale, bias, groups=1, top_groups=1, best=1, op="route"):
    c = {"op": op, "T": T, "E": E, "K": K, "dtype": dtype, "score": score, "renorm": renorm, "scale": scale,
         "bias": bias, "groups": groups, "top_groups": top_groups, "best": best}
    return dict(c, name=name) if name else c


def _experts(name, op, T, E, K, H):
    c = {"op": op, "T": T, "E": E, "K": K, "H": H}
    return dict(c, name=name) if name else c


def _norm(name, op, T, H, dtype):
    c = {"op": op, "T": T, "H": H, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoding step of eight requests: latency, every feature of the rule on
        _route("route_decode_8", 8, 64, 6, "float32", "sigmoid", True, 2.5, True, 8, 4, 2),
        # a long prompt batch through a wide router with a balance bias and groups
        _route("route_prompt_65536", 65536, 256, 8, "float32", "sigmoid", True, 2.5, True, 8, 4, 2),
        # the gate's usual 8 experts, two of them per token, weights straight from the softmax
        _route("route_bwd_softmax_262144", 262144, 8, 2, "float32", "softmax", False, 1.0, False, op="route_bwd"),
        # an odd number of tokens and experts, 16-bit logits, renormalised sigmoid weights
        _route("route_bwd_sigmoid_20479", 20479, 60, 4, "bfloat16", "sigmoid", True, 1.0, False, op="route_bwd"),
        # decoding: four tokens, so the time goes to the weights of the few experts they hit
        _experts("experts_fwd_decode_4", "experts_fwd", 4, 32, 2, 256),
        # the throughput size of the gate's own workloads at a quarter of the tokens
        _experts("experts_fwd_262144", "experts_fwd", 262144, 8, 2, 256),
        # a small ragged training batch of the 128-wide gate
        _experts("experts_bwd_5003", "experts_bwd", 5003, 4, 2, 128),
        # a training batch of a wider block with more experts
        _experts("experts_bwd_16384", "experts_bwd", 16384, 16, 2, 1024),
        # decoding: one token's context vector
        _norm("norm_fwd_one_row", "norm_fwd", 1, 1024, "bfloat16"),
        # the context tokens of the gate's throughput workload
        _norm("norm_fwd_1048576", "norm_fwd", 1048576, 256, "float32"),
        # an odd number of rows of an odd width, 16-bit
        _norm("norm_bwd_4099", "norm_bwd", 4099, 1001, "float16"),
        # the training pass over a quarter of the throughput workload
        _norm("norm_bwd_262144", "norm_bwd", 262144, 256, "float32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "experts_fwd", "experts_bwd", "norm_fwd", "norm_bwd"])
    if op in ("route", "route_bwd"):
        E = _log_int(rng, 4, 256)
        T = min(_log_int(rng, 1, 262144), 16777216 // E)
        K = rng.randint(1, min(8, E))
        groups, top_groups, best = 1, 1, 1
        divisors = [g for g in range(2, 17) if E % g == 0 and E // g >= 2]
        if divisors and rng.random() < 0.5:
            groups = rng.choice(divisors)
            top_groups = rng.randint(1, groups)
            best = rng.choice([1, 2])
            K = min(K, top_groups * (E // groups))
        return _route(None, T, E, K, rng.choice(["float32", "float32", "bfloat16", "float16"]),
                      rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, rng.choice([1.0, 2.5]),
                      rng.random() < 0.5, groups, top_groups, best, op=op)
    if op in ("experts_fwd", "experts_bwd"):
        H = 64 * _log_int(rng, 1, 16)
        E = _log_int(rng, 2, 64)
        K = rng.randint(1, min(4, E))
        # the plain form computes every expert for every token: its products and its arrays are bounded
        T = min(_log_int(rng, 1, 262144), 137438953472 // (E * H * H), 536870912 // (E * H))
        return _experts(None, op, T, E, K, H)
    H = _log_int(rng, 16, 8192)
    T = min(_log_int(rng, 1, 1048576), (268435456 if op == "norm_fwd" else 67108864) // H)
    return _norm(None, op, T, H, rng.choice(["float32", "bfloat16", "float16"]))


# ---------------------------------------------------------------- inputs
def _dispatch(idx, E):
    """counts, offsets and the stable expert-sorted list of the pairs t * K + k."""
    flat = idx.reshape(-1).long()
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    perm = torch.sort(flat, stable=True, dim=0)[1]
    return counts.int(), offsets.int(), perm.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    empty = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32 = torch.int32
    T, op = case["T"], case["op"]
    s = {"case": case}
    if op in ("route", "route_bwd"):
        E, K = case["E"], case["K"]
        # trained routers prefer some experts: a per-expert offset under the tokens' spread
        s["logits"] = (rand(T, E) * 1.2 + rand(E) * 0.4).to(DTYPES[case["dtype"]])
        s["bias"] = rand(E) * 0.05 if case["bias"] else None
        if op == "route":
            s.update(idx=empty(T * K, dtype=i32), counts=empty(E, dtype=i32), offsets=empty(E + 1, dtype=i32),
                     perm=empty(T * K, dtype=i32), weights=empty(T, K))
        else:
            s["idx"] = _plain_select(s["logits"], s["bias"], case)
            s["d_weights"] = rand(T, K)
            s["d_logits"] = torch.empty_like(s["logits"])
        return s
    H = case["H"]
    if op in ("norm_fwd", "norm_bwd"):
        dt = DTYPES[case["dtype"]]
        # a few channels sit far from zero, as in trained blocks
        s["x"] = (rand(T, H) * (0.5 + rand(H).abs()) + 0.3 * rand(H)).to(dt)
        s["gamma"], s["beta"] = (1 + 0.1 * rand(H)).to(dt), (0.1 * rand(H)).to(dt)
        s["mean"], s["rstd"] = empty(T), empty(T)
        if op == "norm_fwd":
            s["y"] = empty(T, H, dtype=dt)
        else:
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = 1 / torch.sqrt((x - s["mean"][:, None]).square().mean(1) + EPS)
            s["dy"] = rand(T, H).to(dt)
            s.update(dx=empty(T, H, dtype=dt), dgamma=empty(H, dtype=dt), dbeta=empty(H, dtype=dt))
        return s
    E, K = case["E"], case["K"]
    bf = torch.bfloat16
    s["x"] = rand(T, H).to(bf)
    s["W"] = (rand(E, H, H) / math.sqrt(H)).to(bf)
    s["b"] = (rand(E, H) * 0.1).to(bf)
    top, idx = torch.topk(rand(T, E) + 0.5 * rand(E), K, dim=1)
    s["weights"] = torch.softmax(top, 1)
    s["idx"] = idx.reshape(-1).int()
    s["counts"], s["offsets"], s["perm"] = _dispatch(idx, E)
    if op == "experts_fwd":
        s["y"] = empty(T, H, dtype=bf)
    else:
        s["d_out"] = rand(T, H).to(bf)
        s.update(d_x=empty(T, H, dtype=bf), dW=empty(E, H, H, dtype=bf), db=empty(E, H, dtype=bf),
                 d_weights=empty(T, K))
    return s


# ---------------------------------------------------------------- plain forms
def _plain_scores(l, case):
    """Scores of the logits, in the type of l; a row with nothing but -inf scores 0 everywhere."""
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    m = l.amax(1, keepdim=True)
    p = torch.exp(l - torch.where(m == -math.inf, 0.0, m))
    return p / torch.where(m == -math.inf, 1.0, p.sum(1, keepdim=True))


def _plain_select(logits, bias, case):
    """The K chosen experts of each token, best first, ties to the lowest index. The
    choice is one of values next to a border: 64 bits. Without a bias the scores are
    in the order of the logits."""
    l = logits.double()
    T, E = l.shape
    masked = torch.isnan(l) | (l == -math.inf)
    value = _plain_scores(l, case) + (0.0 if bias is None else bias.double())
    order = l if bias is None else value
    value, order = value.masked_fill(masked, -math.inf), order.masked_fill(masked, -math.inf)
    G = case["groups"]
    if G > 1:
        by = order if case["best"] == 1 else value
        score = torch.sort(by.reshape(T, G, E // G), 2, descending=True)[0][:, :, :case["best"]].sum(2)
        kept = torch.sort(score, stable=True, dim=1, descending=True)[1][:, :case["top_groups"]]
        inside = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        inside = inside.repeat_interleave(E // G, 1)
        # masked experts of the kept groups come before all others
        first = torch.sort(inside.int(), stable=True, dim=1, descending=True)[1]
        at = torch.sort(order.gather(1, first).masked_fill(~inside.gather(1, first), -math.inf), stable=True, dim=1,
                        descending=True)[1]
        return first.gather(1, at)[:, :case["K"]].int()
    return torch.sort(order, stable=True, dim=1, descending=True)[1][:, :case["K"]].int()


def _plain_weights(logits, idx, case):
    """Weights in 32 bits; renormalised ones as ratios, which stay finite where every score underflows."""
    l = logits.float()
    if not case["renorm"]:
        return case["scale"] * _plain_scores(l, case).gather(1, idx.long())
    k = l.gather(1, idx.long())
    low = torch.clamp(k, max=0.0) if case["score"] == "sigmoid" else k
    m = low.amax(1, keepdim=True)
    p = torch.exp(low - torch.where(m == -math.inf, 0.0, m))
    if case["score"] == "sigmoid":
        p = p / (1 + torch.exp(-k.abs()))
    return case["scale"] * p / torch.where(m == -math.inf, 1.0, p.sum(1, keepdim=True))


def _plain_route_bwd(s, case):
    l, idx, g = s["logits"].float(), s["idx"].long(), s["d_weights"] * case["scale"]
    k = l.gather(1, idx)
    if case["renorm"]:
        w = _plain_weights(s["logits"], idx, dict(case, scale=1.0))
        d = w * (g - (g * w).sum(1, keepdim=True))  # gradient of the chosen log scores
        d = d if case["score"] == "softmax" else d / (1 + torch.exp(k))
        return torch.zeros_like(l).scatter(1, idx, d).to(s["logits"].dtype)
    p = _plain_scores(l, case)
    if case["score"] == "sigmoid":
        d = torch.zeros_like(l).scatter(1, idx, g) * p / (1 + torch.exp(l))
    else:
        v = torch.zeros_like(l).scatter(1, idx, g)
        d = p * (v - (v * p).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _combine(s, E):
    """[T, E] weights of the experts, 0 where an expert was not chosen."""
    T, K = s["weights"].shape
    return s["weights"].new_zeros(T, E).scatter(1, s["idx"].view(T, K).long(), s["weights"])


def _plain_experts_fwd(s, case):
    T, E, H = case["T"], case["E"], case["H"]
    comb = _combine(s, E)
    z = (s["x"].float() @ s["W"].float().reshape(E * H, H).T).view(T, E, H)
    return ((z + s["b"].float()) * comb[:, :, None]).sum(1).to(s["x"].dtype)


def _plain_experts_bwd(s, case):
    T, E, K, H = case["T"], case["E"], case["K"], case["H"]
    x, W, b, g = s["x"].float(), s["W"].float(), s["b"].float(), s["d_out"].float()
    comb = _combine(s, E)
    back = (g @ W.permute(1, 0, 2).reshape(H, E * H)).view(T, E, H)  # W_e^T g
    d_weights = ((back * x[:, None]).sum(2) + g @ b.T).gather(1, s["idx"].view(T, K).long())
    d_x = (back * comb[:, :, None]).sum(1)
    del back
    scaled = (comb[:, :, None] * g[:, None]).view(T, E * H)
    dW = (scaled.T @ x).view(E, H, H)
    bf = s["x"].dtype
    return {"d_x": d_x.to(bf), "dW": dW.to(bf), "db": (comb.T @ g).to(bf), "d_weights": d_weights}


def _plain_norm(s, case):
    x = s["x"].float()
    if case["op"] == "norm_fwd":
        mean = x.mean(1)
        rstd = 1 / torch.sqrt((x - mean[:, None]).square().mean(1) + EPS)
        y = (x - mean[:, None]) * rstd[:, None] * s["gamma"].float() + s["beta"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    dy = s["dy"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    h = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (h - h.mean(1, keepdim=True) - xhat * (h * xhat).mean(1, keepdim=True))
    dt = s["x"].dtype
    return {"dx": dx.to(dt), "dgamma": (dy * xhat).sum(0, dtype=torch.float64).to(dt),
            "dbeta": dy.sum(0, dtype=torch.float64).to(dt)}


def _plain(s, case):
    op = case["op"]
    if op == "route":
        idx = _plain_select(s["logits"], s["bias"], case)
        counts, offsets, perm = _dispatch(idx, case["E"])
        return {"idx": idx, "weights": _plain_weights(s["logits"], idx, case), "counts": counts, "offsets": offsets,
                "perm": perm}
    if op == "route_bwd":
        return {"d_logits": _plain_route_bwd(s, case)}
    if op == "experts_fwd":
        return {"y": _plain_experts_fwd(s, case)}
    if op == "experts_bwd":
        return _plain_experts_bwd(s, case)
    return _plain_norm(s, case)


# ---------------------------------------------------------------- the framework's calls
_workspaces = {}  # a program keeps one workspace per size


def _handle(s, case):
    """What a program makes once: the rule, the routing's buffers, the workspace."""
    if "handle" not in s:
        from bwd_route_b200 import ops
        T, op = case["T"], case["op"]
        rule = routing = None
        if "E" in case:
            if "score" in case:
                score = ops.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else ops.MOE_SCORE_SOFTMAX
                rule = ops.TopKRule(case["E"], case["K"], score, case["renorm"], case["scale"], case["groups"],
                                    case["top_groups"], case["best"])
            if op != "route_bwd":
                routing = ops.Routing(s["idx"], s["counts"], s["offsets"], s["perm"])
            size = ("topk", T, case["E"], case["K"], case.get("H", 0))
        else:
            size = ("norm", T, case["H"])
        if size not in _workspaces:
            _workspaces[size] = (ops.new_topk_workspace if size[0] == "topk" else ops.new_layer_norm_workspace)(
                *size[1:], "cuda")
        s["handle"] = ops, rule, routing, _workspaces[size]
    return s["handle"]


def _own(s, case):
    ops, rule, routing, ws = _handle(s, case)
    op = case["op"]
    if op == "route":
        ops.moe_topk_route(s["logits"], rule, s["bias"], routing, s["weights"], ws)
        return {"idx": s["idx"].view(case["T"], case["K"]), "weights": s["weights"], "counts": s["counts"],
                "offsets": s["offsets"], "perm": s["perm"]}
    if op == "route_bwd":
        ops.moe_topk_route_bwd(s["logits"], rule, s["idx"], s["d_weights"], s["d_logits"])
        return {"d_logits": s["d_logits"]}
    if op == "experts_fwd":
        ops.moe_topk_fwd(s["x"], s["W"], s["b"], routing, s["weights"], s["y"], ws)
        return {"y": s["y"]}
    if op == "experts_bwd":
        ops.moe_topk_bwd(s["x"], s["W"], s["b"], s["d_out"], routing, s["weights"], s["d_x"], s["dW"], s["db"],
                         s["d_weights"], ws)
        return {"d_x": s["d_x"], "dW": s["dW"], "db": s["db"], "d_weights": s["d_weights"]}
    if op == "norm_fwd":
        ops.moe_layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS, s["y"], s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    ops.moe_layer_norm_bwd(s["x"], s["dy"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"], ws)
    return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------------------------- work and exact results
def work(case):
    T, op = case["T"], case["op"]
    if op in ("route", "route_bwd"):
        E, K = case["E"], case["K"]
        b = 4 if case["dtype"] == "float32" else 2
        if op == "route":  # logits; indices, weights and the sorted list; the bias, counts and offsets
            return {"bytes": T * E * b + 12 * T * K + 12 * E, "flops": 4 * T * E}
        read = T * E * b if case["score"] == "softmax" and not case["renorm"] else T * K * b
        return {"bytes": read + 8 * T * K + T * E * b, "flops": 4 * T * E}
    H = case["H"]
    if op in ("norm_fwd", "norm_bwd"):
        b = 4 if case["dtype"] == "float32" else 2
        if op == "norm_fwd":
            return {"bytes": 2 * T * H * b + 8 * T + 2 * H * b, "flops": 8 * T * H}
        return {"bytes": 3 * T * H * b + 8 * T + 3 * H * b, "flops": 14 * T * H}
    E, K = case["E"], case["K"]
    hit = min(E, T * K)  # experts that some token can choose
    if op == "experts_fwd":
        return {"bytes": 4 * T * H + 2 * hit * H * (H + 1) + 8 * T * K, "flops": 2 * T * K * H * H}
    return {"bytes": 6 * T * H + 4 * E * H * (H + 1) + 12 * T * K, "flops": 4 * T * K * H * H}


def _exact_scores(l, case):
    if case["score"] == "sigmoid":
        return np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    e = np.exp(l - l.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def _exact_route(s, case):
    """Finite logits: one expert after the other, the first index among equals."""
    l = s["logits"].double().cpu().numpy()
    T, E = l.shape
    K, G, S = case["K"], case["groups"], E // case["groups"]
    rows = np.arange(T)
    scores = _exact_scores(l, case)
    v = l.copy() if s["bias"] is None else scores + s["bias"].double().cpu().numpy()
    if G > 1:
        by = np.sort((v if case["best"] == 1 or s["bias"] is not None else scores).reshape(T, G, S), 2)
        left = by[:, :, -case["best"]:].sum(2)
        keep = np.zeros((T, G), bool)
        for _ in range(case["top_groups"]):
            at = left.argmax(1)
            keep[rows, at] = True
            left[rows, at] = -np.inf
        v[~np.repeat(keep, S, 1)] = -np.inf
    idx = np.empty((T, K), np.int64)
    for k in range(K):
        idx[:, k] = v.argmax(1)
        v[rows, idx[:, k]] = -np.inf
    w = np.take_along_axis(scores, idx, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdims=True)
    flat = idx.reshape(-1)
    counts = np.bincount(flat, minlength=E)
    i32 = np.int32
    return {"idx": idx.astype(i32), "weights": case["scale"] * w, "counts": counts.astype(i32),
            "offsets": np.concatenate([[0], np.cumsum(counts)]).astype(i32),
            "perm": np.argsort(flat, kind="stable").astype(i32)}


def _exact_route_bwd(s, case):
    """The chain rule through d w / d score and d score / d logit, written out."""
    l = s["logits"].double().cpu().numpy()
    idx = s["idx"].cpu().numpy().astype(np.int64)
    g = case["scale"] * s["d_weights"].double().cpu().numpy()
    p = _exact_scores(l, case)
    v = np.take_along_axis(p, idx, 1)
    if case["renorm"]:
        total = v.sum(1, keepdims=True)
        g = g / total - (g * v).sum(1, keepdims=True) / total ** 2
    up = np.zeros_like(l)  # gradient of the scores
    np.put_along_axis(up, idx, g, 1)
    if case["score"] == "sigmoid":
        return {"d_logits": up * p * (1 - p)}
    return {"d_logits": p * up - p * (p * up).sum(1, keepdims=True)}


def _exact_experts(s, case):
    """Expert by expert over the pairs that chose it."""
    T, E, K, H = case["T"], case["E"], case["K"], case["H"]
    x, w = s["x"].double(), s["weights"].double()
    idx = s["idx"].view(T, K).long()
    if case["op"] == "experts_fwd":
        y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
        for e in range(E):
            t, k = (idx == e).nonzero(as_tuple=True)
            y.index_add_(0, t, w[t, k][:, None] * (x[t] @ s["W"][e].double().T + s["b"][e].double()))
        return {"y": y}
    g = s["d_out"].double()
    out = {"d_x": torch.zeros_like(x), "dW": torch.zeros(E, H, H, dtype=torch.float64, device=x.device),
           "db": torch.zeros(E, H, dtype=torch.float64, device=x.device), "d_weights": torch.zeros_like(w)}
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        We, wt = s["W"][e].double(), w[t, k][:, None]
        out["d_x"].index_add_(0, t, wt * (g[t] @ We))
        out["dW"][e] = (wt * g[t]).T @ x[t]
        out["db"][e] = (wt * g[t]).sum(0)
        out["d_weights"][t, k] = ((x[t] @ We.T + s["b"][e].double()) * g[t]).sum(1)
    return out


def _exact_norm(s, case):
    x, gamma = s["x"].double(), s["gamma"].double()
    if case["op"] == "norm_fwd":
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        return {"y": (x - mean[:, None]) * rstd[:, None] * gamma + s["beta"].double(), "mean": mean, "rstd": rstd}
    mean, rstd, dy = s["mean"].double()[:, None], s["rstd"].double()[:, None], s["dy"].double()
    n = (x - mean) * rstd
    inner = (dy * gamma).sum(1, keepdim=True), (dy * gamma * n).sum(1, keepdim=True)
    return {"dx": (dy * gamma - (inner[0] + n * inner[1]) / case["H"]) * rstd, "dgamma": (dy * n).sum(0),
            "dbeta": dy.sum(0)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s, case)
    if op == "route_bwd":
        return _exact_route_bwd(s, case)
    if op in ("experts_fwd", "experts_bwd"):
        return _exact_experts(s, case)
    return _exact_norm(s, case)
