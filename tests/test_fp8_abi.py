"""Argument checks of the e4m3 entry points and the norm (no GPU needed): bad
calls are refused before any HIP call, and the binding refuses tensors that
are not what the call says."""
import pytest

import quantized_latent_moe_amd as lm

torch = pytest.importorskip("torch")

A = [0x10000 * (i + 1) for i in range(16)]  # aligned, never dereferenced on these paths
EINVAL, EWORKSPACE = 1, 2


def test_quantize_fp8_refusals():
    f = lm.lib().lat_moe_quantize_fp8
    for xt, rows, cols in [(3, 4, 64), (-1, 4, 64), (0, -1, 64), (0, 4, 0), (0, 4, 8), (0, 4, 40), (0, 4, 65552),
                           (0, 1 << 31, 64), (0, 1 << 23, 65536)]:
        assert f(A[0], xt, rows, cols, A[1], A[2], None) == EINVAL, (xt, rows, cols)
    for i in range(3):
        for bad in (None, A[i] + 4):
            p = A[:3]
            p[i] = bad
            assert f(p[0], 0, 4, 64, p[1], p[2], None) == EINVAL
    assert f(None, 1, 0, 64, None, None, None) == 0


def _norm(x=A[0], xt=0, res=None, rt=0, w=A[1], eps=1e-6, T=4, C=64, ro=None, y=A[2], yt=0, q=None, c=None, s=None):
    return lm.lib().lat_moe_rmsnorm(x, xt, res, rt, w, eps, T, C, ro, y, yt, q, c, s, None)


def test_rmsnorm_refusals():
    bad = [dict(x=None), dict(w=None), dict(x=A[0] + 8), dict(w=A[1] + 4), dict(y=A[2] + 8), dict(xt=3), dict(yt=-1),
           dict(res=A[3], rt=5), dict(ro=A[3], rt=5), dict(res=A[3] + 2), dict(ro=A[3] + 2), dict(q=A[4] + 4),
           dict(c=A[5], s=A[6] + 4), dict(c=A[5] + 8, s=A[6]), dict(c=A[5]), dict(s=A[6]), dict(y=None),
           dict(T=-1), dict(T=1 << 31), dict(C=0), dict(C=8), dict(C=72), dict(C=32784), dict(C=48, q=A[4]),
           dict(eps=0.0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
           dict(y=A[0], yt=1)]
    for b in bad:
        assert _norm(**b) == EINVAL, b
    assert _norm(x=None, w=None, y=None, T=0) == 0
    # a type whose array is not given is not looked at
    assert _norm(T=0, rt=9, y=None, yt=9) == 0


def test_dense_fp8_refusals():
    f = lm.lib().lat_moe_dense_fp8
    x, xs, w, ws, y, b, q = A[:7]
    for T, N, K in [(-1, 64, 64), (4, 0, 64), (4, 64, 0), (4, 64, 8), (4, 64, 72), (4, 64, 65552), (4, (1 << 20) + 1, 64),
                    (1 << 31, 64, 64), ((1 << 31) - 1, 1 << 20, 64)]:
        assert f(x, xs, w, ws, T, N, K, y, None, None, None) == EINVAL, (T, N, K)
    assert f(x, xs, w, ws, 4, 64, 64, None, None, None, None) == EINVAL
    assert f(x, xs, w, ws, 4, 72, 64, None, None, q, None) == EINVAL
    for i in range(4):
        for bad in (None, A[i] + 8):
            p = [x, xs, w, ws]
            p[i] = bad
            assert f(*p, 4, 64, 64, y, None, None, None) == EINVAL
    assert f(x, xs, w, ws, 4, 64, 64, y + 4, None, None, None) == EINVAL
    assert f(x, xs, w, ws, 4, 64, 64, None, b + 4, None, None) == EINVAL
    assert f(x, xs, w, ws, 4, 64, 64, None, None, q + 4, None) == EINVAL
    assert f(None, None, None, None, 0, 64, 64, None, None, None, None) == 0


def test_ffn_fp8_refusals_and_workspace():
    size = lm.ffn_fp8_workspace_size
    for T, C, F in [(-1, 64, 64), (4, 8, 64), (4, 64, 8), (4, 72, 64), (4, 64, 72), (4, 65552, 64), (4, 64, 65552),
                    (1 << 31, 64, 64), (4, 1 << 32, 64), ((1 << 31) - 1, 64, 65536), (4, 32768, 32768)]:
        assert size(T, C, F) == 0, (T, C, F)
    for T, C, F in [(0, 64, 64), (1, 64, 64), (64, 512, 1040), (65, 512, 1040), (5268, 4096, 8192)]:
        assert size(T, C, F) >= max(1, T * F + 4 * T * -(-F // 128)), (T, C, F)
    f = lm.lib().lat_moe_ffn_fp8
    p = A[:6]
    y, b, h, hs, ws = A[6:11]
    need = size(4, 64, 128)
    assert f(*p, 4, 64, 128, y, None, None, None, ws, need - 1, None) == EWORKSPACE
    assert f(*p, 4, 64, 128, None, None, None, None, ws, need, None) == EINVAL
    assert f(*p, 4, 64, 128, y, None, h, None, ws, need, None) == EINVAL
    assert f(*p, 4, 64, 128, y, None, None, hs, ws, need, None) == EINVAL
    assert f(*p, 4, 64, 120, y, None, None, None, ws, need, None) == EINVAL
    for i in range(6):
        for bad in (None, A[i] + 4):
            g = list(p)
            g[i] = bad
            assert f(*g, 4, 64, 128, y, None, None, None, ws, need, None) == EINVAL
    for bad in (dict(y=y + 4), dict(b=b + 2), dict(h=h + 1), dict(hs=hs + 4), dict(ws=ws + 8), dict(ws=None)):
        a = dict(y=y, b=b, h=h, hs=hs, ws=ws, **{}) | bad
        assert f(*p, 4, 64, 128, a["y"], a["b"], a["h"], a["hs"], a["ws"], need, None) == EINVAL, bad
    assert f(*[None] * 6, 0, 64, 128, None, None, None, None, None, 0, None) == 0


def test_binding_refuses_host_tensors():
    f8 = torch.float8_e4m3fn
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="current GPU"):
        lm.quantize_fp8(x, torch.zeros(2, 64, dtype=f8), torch.zeros(2, 1))
    with pytest.raises(ValueError, match="current GPU"):
        lm.rmsnorm(x, torch.ones(64), 1e-6, y=x)
    with pytest.raises(ValueError, match="current GPU"):
        lm.dense_fp8(x.to(f8), torch.zeros(2, 1), x.to(f8), torch.zeros(1, 1), y_f32=torch.zeros(2, 2))
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        lm.quantize_fp8(x.double(), torch.zeros(2, 64, dtype=f8), torch.zeros(2, 1))
    with pytest.raises(ValueError, match="2-dimensional"):
        lm.dense_fp8(x[0].to(f8), torch.zeros(2, 1), x.to(f8), torch.zeros(1, 1), y_f32=torch.zeros(2, 2))
