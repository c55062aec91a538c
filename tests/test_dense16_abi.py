"""Argument checks of the 16-bit products and the routing by scores (no GPU
needed): bad calls are refused before any HIP call, and the binding refuses
tensors that are not what the call says."""
import ctypes

import pytest

import quantized_latent_moe_amd as lm

torch = pytest.importorskip("torch")

A = [0x10000 * (i + 1) for i in range(8)]  # aligned, never dereferenced on these paths
EINVAL = 1
F32, BF16, F16 = 0, 1, 2


def _dense(x=A[0], xs=64, w=A[1], kind=BF16, T=4, N=96, K=64, bias=None, act=0, res=None, rk=0, rs=0, y=A[2], yk=0,
           ys=96, q=None):
    return lm.lib().lat_moe_dense_16(x, xs, w, kind, T, N, K, bias, act, res, rk, rs, y, yk, ys, q, None)


def _gated(x=A[0], xs=64, w=A[1], kind=BF16, T=4, F=96, K=64, bias=None, act=2, h=A[2], hk=0, hs=96):
    return lm.lib().lat_moe_gated_16(x, xs, w, kind, T, F, K, bias, act, h, hk, hs, None)


OPERANDS = [dict(x=None), dict(w=None), dict(x=A[0] + 8), dict(w=A[1] + 2), dict(kind=F32), dict(kind=3), dict(kind=-1),
            dict(xs=56), dict(xs=68), dict(xs=(1 << 20) + 8), dict(xs=-64), dict(T=-1), dict(T=1 << 31), dict(K=0),
            dict(K=60), dict(K=65544, xs=65544), dict(bias=A[3] + 4), dict(act=-1), dict(act=5)]


def test_dense_16_refusals():
    bad = OPERANDS + [dict(N=0), dict(N=(1 << 20) + 1, ys=1 << 21), dict(T=(1 << 31) - 1, N=1 << 20, ys=1 << 20),
                      dict(y=None), dict(y=A[2] + 8), dict(yk=3), dict(ys=95), dict(ys=1 << 31), dict(q=A[4] + 4),
                      dict(N=80, ys=80, q=A[4]), dict(res=A[3]), dict(res=A[3], rs=95), dict(res=A[3], rs=96, rk=7),
                      dict(res=A[3] + 4, rs=96), dict(res=A[3], rs=1 << 31), dict(res=A[2], rs=96, rk=1),
                      dict(res=A[2], rs=104)]
    for b in bad:
        assert _dense(**b) == EINVAL, b
    # nothing to do, and what is not given is not looked at
    assert _dense(x=None, w=None, y=None, T=0, rk=9, rs=-1, yk=9, ys=-1) == 0
    for b in (dict(kind=F32), dict(K=60), dict(N=0), dict(act=9)):
        assert _dense(T=0, **b) == EINVAL


def test_gated_16_refusals():
    bad = OPERANDS + [dict(F=0), dict(F=(1 << 19) + 1, hs=1 << 20), dict(h=None), dict(h=A[2] + 4), dict(hk=3),
                      dict(hs=95), dict(hs=1 << 31)]
    for b in bad:
        assert _gated(**b) == EINVAL, b
    assert _gated(x=None, w=None, h=None, T=0) == 0


def _router(logits=A[0], bias=None, T=4, E=64, k=4, idx=A[1], w=A[2], score=0, groups=1, top_groups=1, group_score=1,
            renormalise=1, scale=1.0):
    o = lm.Routing(score, groups, top_groups, group_score, renormalise, scale)
    return lm.lib().lat_moe_router_topk_ex(logits, bias, T, E, k, ctypes.byref(o), idx, w, None)


def test_router_topk_ex_refusals():
    bad = [dict(logits=None), dict(idx=None), dict(w=None), dict(logits=A[0] + 4), dict(idx=A[1] + 4), dict(w=A[2] + 8),
           dict(bias=A[3] + 4), dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=1025), dict(k=0), dict(k=65, E=128),
           dict(k=65), dict(score=2), dict(score=-1), dict(groups=0), dict(groups=65, E=1040), dict(groups=5),
           dict(groups=8, top_groups=0), dict(groups=8, top_groups=9), dict(groups=16, top_groups=1, k=5),
           dict(groups=8, top_groups=2, group_score=2), dict(groups=64, top_groups=8), dict(scale=float("nan")),
           dict(scale=float("inf"))]
    for b in bad:
        assert _router(**b) == EINVAL, b
    assert lm.lib().lat_moe_router_topk_ex(A[0], None, 4, 64, 4, None, A[1], A[2], None) == EINVAL
    assert _router(logits=None, idx=None, w=None, T=0) == 0
    # a group's score is not looked at where every group is kept
    assert _router(T=0, groups=64, top_groups=64, group_score=7) == 0
    assert _router(T=0, groups=64, top_groups=8, group_score=0) == 0


def test_binding_refuses_cpu_tensors_and_unknown_names():
    x, w, y = torch.zeros(4, 64).bfloat16(), torch.zeros(96, 64).bfloat16(), torch.zeros(4, 96)
    for call in (lambda: lm.dense_16(x, w, y=y), lambda: lm.gated_16(x, w, y[:, :48]),
                 lambda: lm.router_topk_ex(torch.zeros(4, 8), 2, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))):
        with pytest.raises(ValueError, match="current GPU"):
            call()
    for bad in (x.float(), x[0], x.to(torch.int16)):
        with pytest.raises(ValueError, match="2-dimensional"):
            lm.dense_16(bad, w, y=y)
    with pytest.raises(ValueError, match="activation"):
        lm._choice("activation", "swish", lm.ACTIVATIONS)
