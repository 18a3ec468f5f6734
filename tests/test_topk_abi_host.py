"""Host-side checks of the top-k block's C ABI (include/moe_topk.h), without a GPU:
what the header declares is exported and bound, and bad arguments are refused with
the documented status before anything touches the GPU."""
import ctypes
import os
import re

import pytest
import torch

from bwd_route_b200 import build as libbuild
from bwd_route_b200 import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_topk.h")

OK, INVALID, SHAPE, MISALIGNED, ALIAS, WORKSPACE = 0, 1, 2, 3, 4, 5
F32, BF16, F16 = 0, 1, 2

# Fake device addresses, 16 MiB apart: the checks compare and align them only.
A = [0x7F0000000000 + (i << 24) for i in range(32)]


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return ops.lib()


def test_every_declared_symbol_is_exported_and_bound(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    fns = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(moe_\w+)\s*\(", text, flags=re.M)))
    assert fns == sorted(ops.EXPORTED_TOPK)
    for name in fns:
        assert hasattr(L, name) and getattr(L, name).argtypes is not None, name
    version = int(re.search(r"#define MOE_TOPK_ABI_VERSION (\d+)", text).group(1))
    assert L.moe_topk_abi_version() == version


def norm_fwd(L, **k):
    v = dict(x=A[0], dtype=BF16, T=10, H=64, ldx=64, gamma=A[1], beta=A[2], pd=BF16, eps=1e-5, y=A[3], mean=A[4],
             rstd=A[5])
    v.update(k)
    return L.moe_layer_norm_fwd(v["x"], v["dtype"], v["T"], v["H"], v["ldx"], v["gamma"], v["beta"], v["pd"], v["eps"],
                                v["y"], v["mean"], v["rstd"], None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(ldx=63), INVALID), (dict(dtype=3), INVALID),
    (dict(pd=F16), INVALID), (dict(pd=-1), INVALID), (dict(eps=-1e-5), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(T=2 ** 31 - 256), SHAPE), (dict(H=8193, ldx=8193), SHAPE), (dict(ldx=2 ** 31 + 1), SHAPE),
    (dict(x=A[0] + 1), MISALIGNED), (dict(y=A[3] + 1), MISALIGNED), (dict(gamma=A[1] + 1), MISALIGNED),
    (dict(mean=A[4] + 2), MISALIGNED), (dict(rstd=A[5] + 2), MISALIGNED),
    (dict(pd=F32, gamma=A[1] + 2), MISALIGNED),
    (dict(y=A[0] + 2), ALIAS), (dict(y=A[0], ldx=80), ALIAS), (dict(y=A[1] - 20), ALIAS), (dict(mean=A[0] + 128), ALIAS),
    (dict(rstd=A[4] + 36), ALIAS), (dict(mean=A[3] + 10 * 128 - 4), ALIAS), (dict(beta=A[3] + 2), ALIAS),
    (dict(T=0), OK), (dict(T=0, x=None, y=None), OK),
])
def test_layer_norm_fwd_refuses(L, change, status):
    assert norm_fwd(L, **change) == status


def norm_bwd(L, **k):
    v = dict(x=A[0], dy=A[1], dtype=BF16, T=10, H=64, ldx=64, gamma=A[2], pd=BF16, mean=A[3], rstd=A[4], dx=A[5],
             dg=A[6], db=A[7], ws=A[8], n=1 << 20)
    v.update(k)
    return L.moe_layer_norm_bwd(v["x"], v["dy"], v["dtype"], v["T"], v["H"], v["ldx"], v["gamma"], v["pd"], v["mean"],
                                v["rstd"], v["dx"], v["dg"], v["db"], v["ws"], v["n"], None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(ldx=10), INVALID), (dict(dtype=7), INVALID), (dict(pd=F16), INVALID),
    (dict(x=None), INVALID), (dict(dy=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(H=9000, ldx=9000), SHAPE), (dict(dx=A[5] + 1), MISALIGNED), (dict(dg=A[6] + 1), MISALIGNED),
    (dict(ws=A[8] + 16), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(n=256), WORKSPACE),
    (dict(dx=A[1] + 2), ALIAS), (dict(dx=A[0]), ALIAS), (dict(dg=A[7] + 126), ALIAS), (dict(dg=A[1], dx=A[1]), ALIAS),
    (dict(ws=A[1]), ALIAS), (dict(db=A[8] + 512), ALIAS), (dict(mean=A[8] + 512), ALIAS),
    (dict(dx=None, dg=None, db=None), OK),
])
def test_layer_norm_bwd_refuses(L, change, status):
    assert norm_bwd(L, **change) == status


def test_layer_norm_workspace_bytes(L):
    f = L.moe_layer_norm_workspace_bytes
    assert f(0, 64) == 256 and f(1, 64) == 256 + 512 and f(10 ** 6, 64) == 256 + 1024 * 512
    assert f(-1, 64) == 0 and f(5, 0) == 0 and f(5, 8193) == 0 and f(2 ** 31, 64) == 0


def rule(**k):
    v = dict(E=64, K=6, score=1, flags=1, scale=2.5, groups=8, top_groups=4, group_best=2)
    v.update(k)
    return ops.TopKRuleC(*(v[n] for n, _ in ops.TopKRuleC._fields_))


BAD_RULES = [
    (dict(score=2), INVALID), (dict(flags=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(E=0, K=0), SHAPE), (dict(E=257, groups=1, top_groups=1), SHAPE),
    (dict(K=0), SHAPE), (dict(K=17), SHAPE), (dict(E=4, K=5, groups=1, top_groups=1), SHAPE), (dict(groups=0), SHAPE),
    (dict(groups=7), SHAPE), (dict(groups=64, top_groups=8, group_best=1), SHAPE), (dict(top_groups=0), SHAPE),
    (dict(top_groups=9), SHAPE), (dict(K=9, top_groups=1), SHAPE), (dict(group_best=0), SHAPE),
    (dict(group_best=3), SHAPE), (dict(E=32, groups=32, top_groups=8, group_best=2), SHAPE),
]


def route(L, r=None, **k):
    v = dict(x=A[0], dtype=F32, T=10, ld=64, bias=A[1], idx=A[2], counts=A[3], offsets=A[4], perm=A[5], w=A[6], ws=A[7],
             n=1 << 20)
    v.update(k)
    out = ops.RoutingC(v["idx"], v["counts"], v["offsets"], v["perm"])
    return L.moe_topk_route(v["x"], v["dtype"], v["T"], v["ld"], r or rule(), v["bias"], out, v["w"], v["ws"], v["n"], None)


def route_bwd(L, r=None, **k):
    v = dict(x=A[0], dtype=F32, T=10, ld=64, idx=A[2], dw=A[3], d=A[4])
    v.update(k)
    return L.moe_topk_route_bwd(v["x"], v["dtype"], v["T"], v["ld"], r or rule(), v["idx"], v["dw"], v["d"], 0, None)


@pytest.mark.parametrize("change,status", BAD_RULES)
def test_rules_that_no_call_accepts(L, change, status):
    r = rule(**change)
    assert route(L, r, ld=300) == status
    assert route_bwd(L, r, ld=300) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(ld=63), INVALID), (dict(dtype=5), INVALID), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(idx=None), INVALID), (dict(counts=None), INVALID), (dict(offsets=None), INVALID),
    (dict(perm=None), INVALID), (dict(T=2 ** 31 // 6), SHAPE), (dict(ld=2 ** 31 + 1), SHAPE),
    (dict(x=A[0] + 2), MISALIGNED), (dict(bias=A[1] + 2), MISALIGNED), (dict(w=A[6] + 1), MISALIGNED),
    (dict(perm=A[5] + 2), MISALIGNED), (dict(ws=A[7] + 128), MISALIGNED), (dict(ws=None), WORKSPACE),
    (dict(n=256), WORKSPACE), (dict(idx=A[0] + 2556), ALIAS), (dict(perm=A[2] + 236), ALIAS), (dict(w=A[1] + 252), ALIAS),
    (dict(counts=A[4] + 4), ALIAS), (dict(x=A[7]), ALIAS), (dict(bias=A[7] + 4096), ALIAS), (dict(w=A[7] + 512), ALIAS),
])
def test_route_refuses(L, change, status):
    assert route(L, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(ld=1), INVALID), (dict(x=None), INVALID), (dict(idx=None), INVALID),
    (dict(dw=None), INVALID), (dict(d=None), INVALID), (dict(d=A[4] + 2), MISALIGNED), (dict(dw=A[3] + 2), MISALIGNED),
    (dict(d=A[0]), ALIAS), (dict(d=A[3] + 16), ALIAS), (dict(T=0), OK), (dict(T=0, x=None, d=None), OK),
])
def test_route_bwd_refuses(L, change, status):
    assert route_bwd(L, **change) == status


def test_topk_workspace_bytes(L):
    f = L.moe_topk_workspace_bytes
    assert f(1, 64, 6, 0) == 256 + 2 * 256 and f(0, 64, 6, 0) == 256
    assert f(10 ** 6, 256, 8, 0) == 256 + 2 * 1024 * 1024
    for bad in ((-1, 8, 2, 0), (1, 0, 1, 0), (1, 257, 1, 0), (1, 8, 0, 0), (1, 8, 9, 0), (1, 64, 17, 0), (2 ** 31, 8, 1, 0),
                (1, 8, 2, -1)):
        assert f(*bad) == 0


BIG = [0x600000000000 + (i << 32) for i in range(16)]  # 4 GiB apart


def experts(L, bwd, **k):
    v = dict(x=BIG[0], W=BIG[1], b=BIG[2], dtype=BF16, g=BIG[3], idx=BIG[4], counts=BIG[5], offsets=BIG[6], perm=BIG[7],
             w=BIG[8], T=10, E=8, K=2, H=128, y=BIG[9], dx=BIG[9], dW=BIG[10], db=BIG[11], dw=BIG[12], ws=BIG[13],
             n=1 << 30)
    v.update(k)
    r = None if v.get("no_routing") else ops.RoutingC(v["idx"], v["counts"], v["offsets"], v["perm"])
    if bwd:
        return L.moe_topk_bwd(v["x"], v["W"], v["b"], v["dtype"], v["g"], r, v["w"], v["T"], v["E"], v["K"], v["H"], v["dx"],
                              v["dW"], v["db"], v["dw"], v["ws"], v["n"], None)
    return L.moe_topk_fwd(v["x"], v["W"], v["b"], v["dtype"], r, v["w"], v["T"], v["E"], v["K"], v["H"], v["y"], v["ws"],
                          v["n"], None)


@pytest.mark.parametrize("bwd", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("change,status", [
    (dict(dtype=F32), INVALID), (dict(dtype=9), INVALID), (dict(T=-1), INVALID), (dict(no_routing=True), INVALID),
    (dict(x=None), INVALID), (dict(W=None), INVALID), (dict(w=None), INVALID), (dict(offsets=None), INVALID),
    (dict(perm=None), INVALID), (dict(E=0), SHAPE), (dict(E=257), SHAPE), (dict(K=0), SHAPE), (dict(K=9), SHAPE),
    (dict(E=64, K=17), SHAPE), (dict(H=0), SHAPE), (dict(H=96), SHAPE), (dict(H=4160), SHAPE), (dict(T=2 ** 30), SHAPE),
    (dict(x=BIG[0] + 8), MISALIGNED), (dict(W=BIG[1] + 2), MISALIGNED), (dict(b=BIG[2] + 8), MISALIGNED),
    (dict(w=BIG[8] + 2), MISALIGNED), (dict(perm=BIG[7] + 1), MISALIGNED), (dict(ws=BIG[13] + 64), MISALIGNED),
    (dict(ws=None), WORKSPACE), (dict(n=4096), WORKSPACE), (dict(x=BIG[13]), ALIAS), (dict(perm=BIG[13] + 1024), ALIAS),
])
def test_experts_refuse(L, bwd, change, status):
    assert experts(L, bwd, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(y=None), INVALID), (dict(y=BIG[9] + 8), MISALIGNED), (dict(y=BIG[0]), ALIAS), (dict(y=BIG[2] + 64), ALIAS),
    (dict(y=BIG[13] + (1 << 20)), ALIAS), (dict(T=0), OK),
])
def test_experts_fwd_refuses(L, change, status):
    assert experts(L, False, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(g=None), INVALID), (dict(idx=None), INVALID), (dict(dx=BIG[9] + 8), MISALIGNED), (dict(dW=BIG[10] + 8), MISALIGNED),
    (dict(db=BIG[11] + 2), MISALIGNED), (dict(dw=BIG[12] + 2), MISALIGNED), (dict(dx=BIG[3]), ALIAS), (dict(dx=BIG[0]), ALIAS),
    (dict(db=BIG[10] + 128), ALIAS), (dict(dw=BIG[9] + 64), ALIAS), (dict(dW=BIG[13]), ALIAS),
    (dict(dx=None, dW=None, db=None, dw=None), OK),
])
def test_experts_bwd_refuses(L, change, status):
    assert experts(L, True, **change) == status


def test_experts_workspace_bytes(L):
    f = L.moe_topk_workspace_bytes
    assert f(10, 8, 2, 128) > f(10, 8, 2, 0) > 0
    assert f(1000, 8, 2, 256) >= 2 * 1000 * 2 * 256  # a row of every pair
    assert f(1000, 8, 1, 256) < f(1000, 8, 2, 256)
    assert f(10, 8, 2, 96) == 0 and f(10, 8, 2, 8192) == 0


def test_binding_refuses_tensors_it_cannot_pass():
    with pytest.raises(ValueError):
        ops.moe_layer_norm_fwd(torch.zeros(2, 4), None, None, 1e-5, torch.zeros(2, 4))
