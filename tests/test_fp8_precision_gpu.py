"""GPU tests of how exact the e4m3 products are: what a call without a choice
does, and the two choices.

Exact products are told from those of the e4m3 matrix unit, which cuts small
products beside a large one, by rows whose every eighth value is as large as
e4m3 goes, against weights under which those products cancel: what the small
products add up to is left.  All products are whole numbers and every partial
sum stays below 2^24, so with exact products the sums have no error at all, in
any order; the scales are powers of two."""
import numpy as np
import pytest

import oracle
from oracle import fp8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402
from tests._gpu import say  # noqa: E402
from tests.test_fp8_gpu import F8, _cut, _dev, _ffn_inputs, _tol, _w  # noqa: E402

SMALL = np.array([-3, -2, -1, 1, 2, 3])


def _cancelling(rng, T, N, K):
    """Codes x [T, K], w [N, K]: small whole numbers, and 448 x 448 products that
    cancel in pairs eight columns apart."""
    x, w = rng.choice(SMALL, (T, K)).astype(np.float64), rng.choice(SMALL, (N, K)).astype(np.float64)
    for k in range(0, K - 15, 16):
        x[:, k] = x[:, k + 8] = 448
        w[:, k] = 448
        w[:, k + 8] = -448
    return fp8.encode(x), fp8.encode(w)


def _check_h(hc, hs, G, U, dG, dU):
    """H's codes and scales against silu(G) U, where G and U are off by at most dG and dU."""
    F = G.shape[1]
    H = fp8.silu_product(G, U)
    # |d silu| <= 1.1 |dG|; exp, the division and the product in fp32: 8 roundings
    dH = 1.1 * dG * (np.abs(U) + dU) + np.abs(fp8.silu_product(G, 1.0)) * dU + np.abs(H) * 8 * 2.0 ** -24
    pad = lambda a: np.pad(a, ((0, 0), (0, -F % 128))).reshape(len(a), -1, 128)
    top, dtop = np.abs(pad(H)).max(2), pad(dH).max(2)
    assert (np.abs(hs * 448.0 - top) <= dtop * 1.001 + top * 2.0 ** -22 + 448 * 2.0 ** -126).all()
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 scales of a subnormal one
    s = np.repeat(hs.astype(np.float64), 128, 1)[:, :F]
    assert (np.abs(fp8.rows(hc, hs) - H)
            <= dH * 1.2 + np.maximum(np.abs(H) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -18)).all()


def _call_ffn(args, T, C, F, exact, f32):
    x, xs, gu, gus, d, ds = (_dev(a) for a in args)
    ws = torch.full((lm.ffn_fp8_workspace_size(T, C, F),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.full((T, C), float("nan"), device="cuda") if f32 else None
    b = torch.full((T, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    hc = torch.full((T, F), 0x55, dtype=torch.uint8, device="cuda").view(F8)
    hs = torch.full((T, fp8.blocks(F)), float("nan"), device="cuda")
    lm.ffn_fp8(x, xs, gu, gus, d, ds, ws, y_f32=y, y_bf16=b, h_fp8=hc, h_scales=hs, exact=exact)
    torch.cuda.synchronize()
    return y, b, hc.view(torch.uint8), hs


# H through fp32 memory (tiles of 32 columns), and rounded where it is made, there
# also with more tiles than workgroups, steps in several runs of scales and a ragged end of K
GATED = [(1, 128, 128), (16, 400, 272), (17, 128, 16), (64, 400, 272), (200, 256, 1040), (700, 656, 272), (70, 144, 65536),
         (17, 272, 65536), (700, 272, 4112), (2500, 656, 1040), (5200, 400, 528), (2300, 1168, 2064)]


@pytest.mark.parametrize("T,C,F", GATED)
def test_ffn_exact(T, C, F):
    rng = np.random.default_rng(T + C + F)
    x, gu = _cancelling(rng, T, 2 * F, C)
    xs = np.ones((T, fp8.blocks(C)), np.float32)
    gus = np.full((2, fp8.blocks(F), fp8.blocks(C)), 2.0 ** -5, np.float32)
    d, ds = _w(rng, C, F)
    args = (x, xs, gu, gus, d, ds)
    y, b, hc, hs = _call_ffn(args, T, C, F, True, True)
    t = np.unique(np.concatenate([np.arange(min(T, 40)), np.arange(max(0, T - 40), T), rng.integers(0, T, 20)]))
    G, U = (fp8.rows(x[t], xs[t]) @ fp8.decode(g).T / 32 for g in (gu[:F], gu[F:]))
    assert np.abs(G).max() < 100 and (np.abs(G) > 0.5).mean() > 0.3
    hcn, hsn = hc.cpu().numpy()[t], hs.cpu().numpy()[t]
    _check_h(hcn, hsn, G, U, np.zeros_like(G), np.zeros_like(U))
    ref, mag = fp8.dense(hcn, hsn, d, ds)
    assert (np.abs(y.cpu().numpy()[t] - ref) <= _tol(ref, mag, F)).all()
    assert torch.equal(b, y.to(torch.bfloat16))
    # the same without the fp32 y, and without rows for H
    _, b2, hc2, hs2 = _call_ffn(args, T, C, F, True, False)
    assert torch.equal(b2, b) and torch.equal(hc2, hc) and torch.equal(hs2, hs)


@pytest.mark.parametrize("T,C,F", [(9, 272, 144), (17, 400, 272), (200, 256, 1040), (700, 1168, 4112)])
def test_ffn_choices_on_random_data(T, C, F):
    """Gates and H of a call without a choice are those of exact=False; H of
    exact products is H of the oracle, within the bound for fp32 sums."""
    rng = np.random.default_rng(T)
    args = _ffn_inputs(rng, T, C, F)
    x, xs, gu, gus, d, ds = args
    ya, ba, ha, sa = _call_ffn(args, T, C, F, None, True)
    yf, bf, hf, sf = _call_ffn(args, T, C, F, False, True)
    _, bn, hn, sn = _call_ffn(args, T, C, F, None, False)
    assert torch.equal(ha, hf) and torch.equal(sa, sf) and torch.equal(ha, hn) and torch.equal(sa, sn)
    assert torch.equal(bn, bf) and torch.equal(bf, yf.to(torch.bfloat16)) and torch.equal(ba, ya.to(torch.bfloat16))
    _, _, he, se = _call_ffn(args, T, C, F, True, True)
    if T <= 16:
        assert torch.equal(he, ha) and torch.equal(se, sa) and torch.equal(ya, yf)
    else:
        h = ha.cpu().numpy()
        ref, mag = fp8.dense(h, sa.cpu().numpy(), d, ds)
        t = np.arange(0, T, max(1, T // 20))
        cut = _cut(h[t], sa.cpu().numpy()[t], d, ds)
        assert (np.abs(yf.cpu().numpy() - ref)[t] <= _tol(ref, mag, F)[t] + cut).all()
    G, Gm = fp8.dense(x, xs, gu[:F], gus[0])
    U, Um = fp8.dense(x, xs, gu[F:], gus[1])
    _check_h(he.cpu().numpy(), se.cpu().numpy(), G, U, _tol(G, Gm, C), _tol(U, Um, C))
    say(f"ffn T={T} C={C} F={F}: H codes that exact products change {(he != ha).float().mean().item():.5f}")


def _call_dense(d, T, N, exact, f32=False, bf16=False, q8=False):
    y = torch.full((T, N), float("nan"), device="cuda") if f32 else None
    b = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda") if bf16 else None
    q = torch.full((T, N // 32, 36), 0x55, dtype=torch.uint8, device="cuda") if q8 else None
    lm.dense_fp8(*d, y_f32=y, y_bf16=b, y_q8_1=q, exact=exact)
    torch.cuda.synchronize()
    return y, b, q


# streaming kernel, groups of 32 tokens, and tiles of every size of both kinds
@pytest.mark.parametrize("T,N,K", [(16, 96, 144), (17, 96, 144), (33, 64, 400), (300, 544, 656), (700, 4128, 656),
                                   (2100, 1056, 144), (4133, 2080, 144), (1500, 4128, 272)])
def test_dense_choices(T, N, K):
    rng = np.random.default_rng(T + N)
    x, w = _cancelling(rng, T, N, K)
    xs = np.ones((T, fp8.blocks(K)), np.float32)
    ws = np.full((fp8.blocks(N), fp8.blocks(K)), 2.0 ** -5, np.float32)
    d = tuple(_dev(a) for a in (x, xs, w, ws))
    ref = fp8.rows(x, xs) @ fp8.decode(w).T / 32                 # exactly
    y = _call_dense(d, T, N, None, f32=True)[0]
    assert np.array_equal(y.cpu().numpy(), ref)
    # exact=True: the rounded outputs alone are those of the exact y
    _, b, q = _call_dense(d, T, N, True, bf16=True, q8=True)
    assert torch.equal(b, y.to(torch.bfloat16)) and np.array_equal(q.cpu().numpy(), oracle.quantize_q8_1(ref.astype(np.float32)))
    assert torch.equal(_call_dense(d, T, N, True, bf16=True)[1], b)
    assert torch.equal(_call_dense(d, T, N, True, q8=True)[2], q)
    # exact=False: one fp32 y by the matrix unit, whose roundings are those of a call without a choice
    yf, bf, qf = _call_dense(d, T, N, False, f32=True, bf16=True, q8=True)
    t = np.unique(np.concatenate([np.arange(min(T, 40)), np.arange(max(0, T - 40), T)]))
    cut = _cut(x[t], xs[t], w, ws) if T > 16 else 0.0
    assert (np.abs(yf.cpu().numpy()[t] - ref[t]) <= cut + np.abs(ref[t]) * 2.0 ** -20).all()
    assert torch.equal(bf, yf.to(torch.bfloat16)) and np.array_equal(qf.cpu().numpy(), oracle.quantize_q8_1(yf.cpu().numpy()))
    _, bn, qn = _call_dense(d, T, N, None, bf16=True, q8=True)
    assert torch.equal(bn, bf) and torch.equal(qn, qf)
    assert torch.equal(yf, y) == (T <= 16)


def test_c_entry_points_without_a_choice():
    """lat_moe_dense_fp8 and lat_moe_ffn_fp8 are the calls with LAT_MOE_PRODUCTS_AUTO."""
    rng = np.random.default_rng(5)
    T, C, F = 70, 272, 144
    a = tuple(_dev(v) for v in _ffn_inputs(rng, T, C, F))
    ws = torch.empty(lm.ffn_fp8_workspace_size(T, C, F), dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()
    st = torch.cuda.current_stream().cuda_stream
    for f32 in (True, False):
        y = [torch.empty(T, C, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda") for _ in range(2)]
        lm.ffn_fp8(*a, ws, **{"y_f32" if f32 else "y_bf16": y[0]})
        o = (p(y[1]), None) if f32 else (None, p(y[1]))
        assert lm.lib().lat_moe_ffn_fp8(*map(p, a), T, C, F, *o, None, None, p(ws), ws.numel(), st) == 0
        torch.cuda.synchronize()
        assert torch.equal(*y)
        z = [torch.empty(T, 2 * F, dtype=y[0].dtype, device="cuda") for _ in range(2)]
        w = torch.ones(fp8.blocks(2 * F), fp8.blocks(C), device="cuda")
        lm.dense_fp8(a[0], a[1], a[2], w, **{"y_f32" if f32 else "y_bf16": z[0]})
        o = (p(z[1]), None, None) if f32 else (None, p(z[1]), None)
        assert lm.lib().lat_moe_dense_fp8(p(a[0]), p(a[1]), p(a[2]), p(w), T, 2 * F, C, *o, st) == 0
        torch.cuda.synchronize()
        assert torch.equal(*z)


@pytest.mark.parametrize("T", [16, 40, 700])
def test_subnormal_codes(T):
    """Products of the smallest codes, subnormal ones among them: whole numbers of
    2^-18 with few bits, which add up exactly."""
    rng = np.random.default_rng(T)
    N, K = 160, 272
    x = (rng.integers(0, 12, (T, K)) | rng.choice([0, 128], (T, K))).astype(np.uint8)
    w = (rng.integers(0, 12, (N, K)) | rng.choice([0, 128], (N, K))).astype(np.uint8)
    xs, ws = np.ones((T, fp8.blocks(K)), np.float32), np.ones((fp8.blocks(N), fp8.blocks(K)), np.float32)
    d = tuple(_dev(a) for a in (x, xs, w, ws))
    ref = fp8.decode(x) @ fp8.decode(w).T
    # all codes have the same exponent as the operand holds it: nothing is cut
    for exact in (True, False):
        y = _call_dense(d, T, N, exact, f32=True)[0]
        assert np.array_equal(y.cpu().numpy(), ref)


@pytest.mark.parametrize("T,C,F", [(40, 272, 400), (700, 400, 2064)])
def test_exact_calls_captured(T, C, F):
    """The gated block and a projection with exact products in a graph, replayed
    between eager calls of other products on the same workspace."""
    rng = np.random.default_rng(T)
    a = tuple(_dev(v) for v in _ffn_inputs(rng, T, C, F))
    w, ws = (_dev(v) for v in _w(rng, 96, C))
    work = torch.empty(lm.ffn_fp8_workspace_size(T, C, F), dtype=torch.uint8, device="cuda")
    out = [torch.empty(T, C, device="cuda"), torch.empty(T, 3, 36, dtype=torch.uint8, device="cuda")]

    def step():
        lm.ffn_fp8(*a, work, y_f32=out[0], exact=True)
        lm.dense_fp8(*a[:2], w, ws, y_q8_1=out[1], exact=True)

    step()
    torch.cuda.synchronize()
    eager = [o.clone() for o in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    for _ in range(4):
        for o in out:
            o.zero_()
        work.fill_(0xFF)
        lm.ffn_fp8(*a, work, y_bf16=other, exact=False)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, e) for o, e in zip(out, eager))
