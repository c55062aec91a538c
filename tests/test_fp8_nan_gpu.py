"""GPU tests of NaN codes in the e4m3 products: they reach the outputs that they
enter (of q8_1 rows the whole block of 32, whose scale becomes a NaN) and no
others, through every kind of kernel; NaN rows behind the last token and the
last weight row, and NaN codes of the next row behind a ragged K, are not read."""
import numpy as np
import pytest

from oracle import fp8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402
from tests.test_fp8_gpu import F8, _cut, _dev, _ffn_inputs, _tol, _w, _x  # noqa: E402


def _call(x, xs, w, ws, exact):
    T, N = x.shape[0], w.shape[0]
    y = torch.empty((T, N), device="cuda")
    b = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    q = torch.empty((T, N // 32, 36), dtype=torch.uint8, device="cuda") if N % 32 == 0 else None
    lm.dense_fp8(x, xs, w, ws, y_f32=y, y_bf16=b, y_q8_1=q, exact=exact)
    torch.cuda.synchronize()
    return y, b, q


def _scales_of(q):
    """The fp16 scale of each q8_1 block."""
    return q[..., :2].contiguous().view(torch.float16)[..., 0]


# streaming kernel, groups of 32 tokens, and tiles of every size with each kind of products
@pytest.mark.parametrize("T,N,K", [(5, 96, 144), (33, 64, 272), (70, 288, 144), (2200, 100, 144), (2100, 1056, 144),
                                   (700, 4128, 272), (4133, 2080, 144)])
@pytest.mark.parametrize("exact", [True, False])
def test_dense_nan_codes(T, N, K, exact):
    rng = np.random.default_rng(T + K)
    (x, xs), (w, ws) = _x(rng, T + 1, K), _w(rng, N + 1, K)
    x[T], w[N] = 0x7F, 0xFF
    xd, xsd, wd, wsd = _dev(x), _dev(xs), _dev(w), _dev(ws[:fp8.blocks(N)])
    y, b, q = _call(xd[:T], xsd[:T], wd[:N], wsd, exact)
    t = np.arange(max(0, T - 40), T)
    ref, mag = fp8.dense(x[t], xs[t], w[:N], ws[:fp8.blocks(N)])
    cut = 0.0 if exact or T <= 16 else _cut(x[t], xs[t], w[:N], ws[:fp8.blocks(N)])
    assert (np.abs(y.cpu().numpy()[t] - ref) <= _tol(ref, mag, K) + cut).all()
    # a token's NaN near the ragged end, a weight row's at the first place
    bad_x, bad_w = x.copy(), w.copy()
    bad_x[2, K - 2], bad_x[T - 1, 7], bad_w[37, 0] = 0x7F, 0xFF, 0xFF
    y2, b2, q2 = _call(_dev(bad_x)[:T], xsd[:T], _dev(bad_w)[:N], wsd, exact)
    nan = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    nan[2] = nan[T - 1] = True
    nan[:, 37] = True
    assert torch.equal(torch.isnan(y2), nan) and torch.equal(torch.isnan(b2), nan)
    assert torch.equal(y2[~nan], y[~nan]) and torch.equal(b2[~nan], b[~nan])
    if q is not None:
        blocks = nan.view(T, N // 32, 32).any(2)
        assert torch.equal(torch.isnan(_scales_of(q2)), blocks)
        assert torch.equal(q2[~blocks], q[~blocks])


@pytest.mark.parametrize("exact", [None, True])
@pytest.mark.parametrize("T,C,F", [(5, 144, 272), (70, 272, 144), (700, 272, 1040), (2100, 400, 2064), (2500, 144, 1040)])
def test_ffn_nan_codes(T, C, F, exact):
    rng = np.random.default_rng(T)
    x, xs, gu, gus, d, ds = _ffn_inputs(rng, T + 1, C, F)
    x[T] = 0x7F
    gu, d = np.concatenate([gu, np.full((1, C), 0x7F, np.uint8)]), np.concatenate([d, np.full((1, F), 0xFF, np.uint8)])
    xsd, gusd, dsd, gud, dd = _dev(xs)[:T], _dev(gus), _dev(ds), _dev(gu)[:2 * F], _dev(d)[:C]
    ws = torch.full((lm.ffn_fp8_workspace_size(T, C, F),), 0xFF, dtype=torch.uint8, device="cuda")

    def run(codes):
        b = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
        hc = torch.empty((T, F), dtype=torch.uint8, device="cuda").view(F8)
        hs = torch.empty((T, fp8.blocks(F)), device="cuda")
        b1 = torch.empty_like(b)
        lm.ffn_fp8(_dev(codes)[:T], xsd, gud, gusd, dd, dsd, ws, y_bf16=b, h_fp8=hc, h_scales=hs, exact=exact)
        lm.ffn_fp8(_dev(codes)[:T], xsd, gud, gusd, dd, dsd, ws, y_bf16=b1, exact=exact)
        torch.cuda.synchronize()
        assert torch.equal(b.view(torch.int16), b1.view(torch.int16))
        return b, hc.view(torch.uint8), hs

    b, hc, hs = run(x)
    assert torch.isfinite(b).all() and torch.isfinite(hs).all() and not (hc & 0x7F == 0x7F).any()
    bad = x.copy()
    bad[3, C - 1] = bad[T - 1, 0] = 0x7F
    b2, hc2, hs2 = run(bad)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[3] = keep[T - 1] = False
    assert torch.isnan(b2[~keep]).all()
    assert torch.equal(b2[keep], b[keep]) and torch.equal(hc2[keep], hc[keep]) and torch.equal(hs2[keep], hs[keep])
