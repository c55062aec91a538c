"""GPU tests of e4m3 tiles whose workgroups take one tile after the other: steps
in several runs of scales, the last run not full, ragged ends in every
direction, and more tiles than workgroups.  Rows of every token tile are
compared with the oracle, all of their columns, so every tile is."""
import numpy as np
import pytest

from oracle import fp8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402
from tests import _tiles  # noqa: E402
from tests._gpu import say  # noqa: E402
from tests.test_fp8_gpu import F8, _cut, _dev, _ffn_inputs, _tol, _w, _x  # noqa: E402
from tests.test_fp8_precision_gpu import _check_h  # noqa: E402


def _rows_of_every_tile(rng, T, tokens):
    first = np.arange(0, T, tokens)
    return np.unique(np.concatenate([first, np.minimum(first + tokens, T) - 1, np.minimum(first + rng.integers(0, tokens, len(first)), T - 1)]))


def _expect(product, tile, T, N, K):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    c = _tiles.choose(product, T, N, K, cus)
    say(f"product {product} T={T} N={N} K={K}: tile {c.cols} x {c.tokens}, {c.tiles} tiles on {cus} CUs")
    assert (c.cols, c.tokens) == tile and c.stays and c.tiles > cus


@pytest.mark.parametrize("product,tile,T,N,K", [w for w in _tiles.WALKS if w[0] <= _tiles.DENSE_EXACT])
def test_dense(product, tile, T, N, K):
    _expect(product, tile, T, N, K)
    exact = product == _tiles.DENSE_EXACT
    rng = np.random.default_rng(T + K)
    (x, xs), (w, ws) = _x(rng, T, K), _w(rng, N, K)
    y = torch.full((T + 1, N), float("nan"), device="cuda")
    b = torch.full((T + 1, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    lm.dense_fp8(*(_dev(a) for a in (x, xs, w, ws)), y_f32=y[:T], y_bf16=b[:T], exact=exact)
    torch.cuda.synchronize()
    assert torch.isnan(y[T]).all() and torch.isnan(b[T]).all()       # the row behind the last stays
    assert torch.equal(b[:T], y[:T].to(torch.bfloat16))
    t = _rows_of_every_tile(rng, T, tile[1])
    ref, mag = fp8.dense(x[t], xs[t], w, ws)
    tol = _tol(ref, mag, K) + (0.0 if exact else _cut(x[t], xs[t], w, ws))
    assert (np.abs(y[:T].cpu().numpy()[t] - ref) <= tol).all()


@pytest.mark.parametrize("product,tile,T,F,C", [w for w in _tiles.WALKS if w[0] >= _tiles.GATED])
def test_gated(product, tile, T, F, C):
    _expect(product, tile, T, F, C)
    exact = product == _tiles.GATED_EXACT
    rng = np.random.default_rng(T + C)
    args = _ffn_inputs(rng, T, C, F)
    x, xs, gu, gus, d, ds = args
    work = torch.full((lm.ffn_fp8_workspace_size(T, C, F),), 0xFF, dtype=torch.uint8, device="cuda")
    b = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
    hc = torch.full((T + 1, F), 0x55, dtype=torch.uint8, device="cuda")
    hs = torch.full((T + 1, fp8.blocks(F)), float("nan"), device="cuda")
    lm.ffn_fp8(*(_dev(a) for a in args), work, y_bf16=b, h_fp8=hc[:T].view(F8), h_scales=hs[:T], exact=exact or None)
    torch.cuda.synchronize()
    assert (hc[T] == 0x55).all() and torch.isnan(hs[T]).all() and torch.isfinite(hs[:T]).all()
    t = _rows_of_every_tile(rng, T, tile[1])
    G, Gm = fp8.dense(x[t], xs[t], gu[:F], gus[0])
    U, Um = fp8.dense(x[t], xs[t], gu[F:], gus[1])
    dG, dU = _tol(G, Gm, C), _tol(U, Um, C)
    if not exact:
        dG, dU = dG + _cut(x[t], xs[t], gu[:F], gus[0]), dU + _cut(x[t], xs[t], gu[F:], gus[1])
    h, s = hc.cpu().numpy()[t], hs.cpu().numpy()[t]
    _check_h(h, s, G, U, dG, dU)
    ref, mag = fp8.dense(h, s, d, ds)
    tol = _tol(ref, mag, F) + (0.0 if exact else _cut(h, s, d, ds))
    assert (np.abs(b.float().cpu().numpy()[t] - ref) <= tol * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8).all()


@pytest.mark.parametrize("exact", [True, False])
def test_more_tiles_than_one_row_of_the_grid(exact):
    """More than 2^20 workgroups of a tile each come in rows of 2^20: many tokens
    by one weight row, tokens of which a pattern of 4096 repeats."""
    T, N, K, n = (1 << 26) + 77, 1, 2064, 4096
    c = _tiles.choose(_tiles.DENSE_EXACT if exact else _tiles.DENSE, T, N, K)
    assert not c.stays and c.tiles > 1 << 20
    rng = np.random.default_rng(1)
    (x, xs), (w, ws) = _x(rng, n, K), _w(rng, N, K)
    xd, xsd, wd, wsd = (_dev(a) for a in (x, xs, w, ws))
    whole = T // n * n
    X, XS = torch.empty((T, K), dtype=torch.uint8, device="cuda"), torch.empty((T, xs.shape[1]), device="cuda")
    for big, small in ((X, xd.view(torch.uint8)), (XS, xsd)):
        big[:whole].view(whole // n, n, -1).copy_(small.expand(whole // n, n, -1))
        big[whole:] = small[:T - whole]
    y = torch.full((T, N), float("nan"), device="cuda")
    lm.dense_fp8(X.view(F8), XS, wd, wsd, y_f32=y, exact=exact)
    torch.cuda.synchronize()
    first = y[:n]
    assert (y[:whole].view(-1, n, N) == first).all() and torch.equal(y[whole:], first[:T - whole])
    ref, mag = fp8.dense(x, xs, w, ws)
    assert (np.abs(first.cpu().numpy() - ref) <= _tol(ref, mag, K) + (0.0 if exact else _cut(x, xs, w, ws))).all()
    del X, XS, y, first
    torch.cuda.empty_cache()


def test_exact_gated_offsets_beyond_32_bits():
    """H past 2^32 values, rounded where it is made with exact products: the last
    rows are those of a call of their own."""
    T, C, F = 140003, 144, 32768
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = lambda *s: torch.randint(0, 0x7E, s, dtype=torch.uint8, device="cuda", generator=g).view(F8)
    scales = lambda *s: torch.rand(s, device="cuda", generator=g) * 1e-3
    x, xs, gu, gus = codes(T, C), scales(T, 2), codes(2 * F, C), scales(2, F // 128, 2)
    d, ds = codes(C, F), scales(2, F // 128)
    at = T // 4 * 4 - 10000
    out = []
    for first in (0, at):
        n = T - first
        h, hs = torch.full((n, F), 0x7F, dtype=torch.uint8, device="cuda").view(F8), torch.full((n, F // 128), float("nan"), device="cuda")
        y = torch.full((n, C), float("nan"), device="cuda")
        work = torch.empty(lm.ffn_fp8_workspace_size(n, C, F), dtype=torch.uint8, device="cuda")
        lm.ffn_fp8(x[first:], xs[first:], gu, gus, d, ds, work, y_f32=y, h_fp8=h, h_scales=hs, exact=True)
        torch.cuda.synchronize()
        out.append((h.view(torch.uint8)[at - first:].clone(), hs[at - first:].clone(), y[at - first:].clone()))
        assert torch.isfinite(hs).all() and torch.isfinite(y).all() and not (h.view(torch.uint8)[::97] & 0x7F == 0x7F).any()
    assert all(torch.equal(a, b) for a, b in zip(*out))
