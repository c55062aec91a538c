"""GPU tests of the norm and of the e4m3 rounding of rows, against the oracle.

The roundings are exact: q8_1 bytes, e4m3 codes and scales equal those that the
oracle's rule makes of the fp32 y that the same call returns.  y itself: v is
the fp32 sum (exact here), r = 1/sqrt(.) has one fp32 rounding (its 64-bit sum
errs by less than 2^-40), and two products follow, so
    |y - y_ref| <= |y_ref| (1 + 2^-24)^3 - |y_ref| < 3.1 * 2^-24 |y_ref|,
plus half a step of the output type, plus 2^-149 (2^-25 in fp16) near zero.
"""
import numpy as np
import pytest

import oracle
from oracle import fp8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
F8 = torch.float8_e4m3fn


def _np(t):
    if t.dtype == F8:
        return t.view(torch.uint8).cpu().numpy()
    return t.float().cpu().numpy() if t.dtype in (BF16, F16) else t.cpu().numpy()


def _rows(rng, T, C, dtype, scale=1.0):
    x = rng.standard_normal((T, C)) * np.exp(0.7 * rng.standard_normal((1, C))) * scale
    return torch.from_numpy(x.astype(np.float32)).cuda().to(dtype)


def _norm(x, w, eps, residual, y_type, q8_1=True, in_place=False):
    T, C = x.shape
    o = {"y": torch.full((T, C), float("nan"), dtype=y_type, device="cuda"),
         "c": torch.full((T, C), 0x55, dtype=torch.uint8, device="cuda").view(F8),
         "s": torch.full((T, fp8.blocks(C)), float("nan"), device="cuda"),
         "q": torch.full((T, C // 32, 36), 0x55, dtype=torch.uint8, device="cuda") if q8_1 and C % 32 == 0 else None,
         "r": None if residual is None else residual if in_place else torch.full_like(residual, float("nan"))}
    lm.rmsnorm(x, w, eps, residual=residual, residual_out=o["r"], y=o["y"], y_q8_1=o["q"], y_fp8=o["c"],
               y_scales=o["s"])
    torch.cuda.synchronize()
    return o


def _check(o, x, w, eps, residual):
    v, ref = fp8.rmsnorm(_np(x), _np(w), eps, None if residual is None else _np(residual))
    y = _np(o["y"]).astype(np.float64)
    half = {F32: 0.0, BF16: 2.0 ** -8, F16: 2.0 ** -11}[o["y"].dtype]
    floor = {F32: 2.0 ** -149, BF16: 2.0 ** -134, F16: 2.0 ** -25}[o["y"].dtype]
    assert (np.abs(y - ref) <= np.abs(ref) * (3.1 * 2.0 ** -24 + half * (1 + 2.0 ** -20)) + floor).all()
    if residual is not None:
        assert np.array_equal(_np(o["r"]), _np(torch.from_numpy(v).to(o["r"].dtype)))


@pytest.mark.parametrize("C", [16, 32, 48, 128, 496, 512, 528, 1024, 2048, 2064, 4096, 4112, 7168, 8192, 8208, 32768])
@pytest.mark.parametrize("T", [1, 5])
def test_norm_of_fp32_rows_and_its_roundings(T, C):
    rng = np.random.default_rng(C + T)
    x, res = _rows(rng, T, C, F32), _rows(rng, T, C, F32, 2.0)
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(C)).astype(np.float32)).cuda()
    o = _norm(x, w, 1e-6, res, F32)
    _check(o, x, w, 1e-6, res)
    y = _np(o["y"])
    codes, scales = fp8.quantize(y)
    assert np.array_equal(_np(o["s"]), scales)
    assert np.array_equal(_np(o["c"]), codes)
    if C % 32 == 0:
        q = torch.empty((T, C // 32, 36), dtype=torch.uint8, device="cuda")
        lm.quantize_q8_1(o["y"], q)
        assert torch.equal(o["q"], q)
        assert np.array_equal(_np(o["q"]), oracle.quantize_q8_1(y))


@pytest.mark.parametrize("xt", [F32, BF16, F16])
@pytest.mark.parametrize("rt", [None, F32, BF16, F16])
@pytest.mark.parametrize("yt", [F32, BF16, F16])
def test_norm_types(xt, rt, yt):
    rng = np.random.default_rng(7)
    T, C = 67, 1040
    x = _rows(rng, T, C, xt)
    res = None if rt is None else _rows(rng, T, C, rt, 3.0)
    w = torch.from_numpy((1 + 0.3 * rng.standard_normal(C)).astype(np.float32)).cuda()
    o = _norm(x, w, 1e-5, res, yt)
    _check(o, x, w, 1e-5, res)
    o32 = _norm(x, w, 1e-5, res, F32)           # the 8-bit rows do not depend on y's type
    assert torch.equal(o["c"].view(torch.uint8), o32["c"].view(torch.uint8)) and torch.equal(o["s"], o32["s"])
    assert np.array_equal(_np(o32["c"]), fp8.quantize(_np(o32["y"]))[0])


def test_norm_in_place_and_without_residual():
    rng = np.random.default_rng(8)
    T, C = 33, 4096
    x, res = _rows(rng, T, C, BF16), _rows(rng, T, C, BF16)
    w = torch.ones(C, device="cuda")
    ref = _norm(x, w, 1e-6, res, BF16)
    stream, xin = res.clone(), x.clone()
    lm.rmsnorm(xin, w, 1e-6, residual=stream, residual_out=stream, y=xin)
    torch.cuda.synchronize()
    assert torch.equal(stream, ref["r"]) and torch.equal(xin, ref["y"])
    # residual_out without residual: x itself, in the stream's type
    out = torch.empty((T, C), dtype=F16, device="cuda")
    lm.rmsnorm(x, w, 1e-6, residual_out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, x.float().to(F16))


def test_norm_row_extremes():
    """Rows of zeros, of one value, huge and tiny ones; a row with a NaN or an
    infinity leaves the others as they are."""
    rng = np.random.default_rng(9)
    C = 512
    x = rng.standard_normal((8, C)).astype(np.float32)
    x[0] = 0
    x[1] = 0
    x[1, 77] = 3.0
    x[2] *= 1e30
    x[3] *= 1e-30
    x[4] = 65504.0
    w = torch.ones(C, device="cuda")
    xt = torch.from_numpy(x).cuda()
    o = _norm(xt, w, 1e-6, None, F32)
    _check(o, xt, w, 1e-6, None)
    assert np.array_equal(_np(o["c"]), fp8.quantize(_np(o["y"]))[0])
    assert np.array_equal(_np(o["q"]), oracle.quantize_q8_1(_np(o["y"])))
    bad = xt.clone()
    bad[5, 3], bad[6, 100] = float("nan"), float("inf")
    ob = _norm(bad, w, 1e-6, None, F32)
    keep = [0, 1, 2, 3, 4, 7]
    assert torch.equal(ob["y"][keep], o["y"][keep])
    assert torch.equal(ob["c"].view(torch.uint8)[keep], o["c"].view(torch.uint8)[keep])


def test_norm_leaves_other_memory_alone_and_repeats():
    rng = np.random.default_rng(10)
    T, C = 9, 2064
    x = _rows(rng, T, C, F32)
    w = torch.ones(C, device="cuda")
    buf = torch.full((T + 2, C), 7.0, device="cuda")
    lm.rmsnorm(x, w, 1e-6, y=buf[1:T + 1])
    again = torch.empty((T, C), device="cuda")
    lm.rmsnorm(x, w, 1e-6, y=again)
    torch.cuda.synchronize()
    assert (buf[0] == 7).all() and (buf[-1] == 7).all() and torch.equal(buf[1:T + 1], again)
    lm.rmsnorm(torch.empty((0, C), device="cuda"), w, 1e-6, y=torch.empty((0, C), device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,C", [(1, 16), (3, 128), (7, 144), (130, 400), (33, 4096), (2, 65536), (1000, 272)])
def test_quantize_fp8_is_the_rule_exactly(T, C, dtype):
    rng = np.random.default_rng(T * C)
    x = _rows(rng, T, C, dtype)
    x[T // 2, :128] = 0
    if T > 2 and dtype == F32:
        x[1] *= 1e-37
        x[2] *= 1e37
    codes = torch.full((T, C), 0x55, dtype=torch.uint8, device="cuda").view(F8)
    scales = torch.full((T, fp8.blocks(C)), float("nan"), device="cuda")
    lm.quantize_fp8(x, codes, scales)
    torch.cuda.synchronize()
    rc, rs = fp8.quantize(_np(x))
    assert np.array_equal(_np(scales), rs)
    assert np.array_equal(_np(codes), rc)


def test_quantize_fp8_nan_stays_in_its_block():
    x = torch.ones((2, 400), device="cuda")
    x[0, 130], x[1, 0] = float("nan"), float("inf")
    codes, scales = torch.empty((2, 400), dtype=F8, device="cuda"), torch.empty((2, 4), device="cuda")
    lm.quantize_fp8(x, codes, scales)
    v = codes.float() * scales.repeat_interleave(128, 1)[:, :400]
    torch.cuda.synchronize()
    assert (v[0, :128] == 1).all() and (v[0, 256:] == 1).all() and (v[1, 128:] == 1).all()


def test_refusals_on_the_device():
    x, w = torch.zeros((4, 64), device="cuda"), torch.ones(64, device="cuda")
    y = torch.empty_like(x)
    with pytest.raises(ValueError, match="contiguous"):
        lm.rmsnorm(torch.zeros((64, 4), device="cuda").t(), w, 1e-6, y=y)
    with pytest.raises(ValueError, match="shape"):
        lm.rmsnorm(x, torch.ones(32, device="cuda"), 1e-6, y=y)
    with pytest.raises(ValueError, match="expected"):
        lm.rmsnorm(x, w, 1e-6, residual=x, residual_out=y.to(BF16))
    with pytest.raises(lm.LatMoeError, match="error 1"):
        lm.rmsnorm(x, w, 0.0, y=y)
    with pytest.raises(lm.LatMoeError, match="error 1"):
        lm.rmsnorm(x, w, 1e-6)
    with pytest.raises(ValueError, match="current GPU"):
        lm.rmsnorm(x, w.cpu(), 1e-6, y=y)


def test_norm_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(11)
    T, C = 6, 4096
    x, res = _rows(rng, T, C, BF16), _rows(rng, T, C, BF16)
    w = torch.ones(C, device="cuda")
    ref = _norm(x, w, 1e-6, res, BF16)
    o = {"r": torch.empty_like(res), "c": torch.empty((T, C), dtype=F8, device="cuda"),
         "s": torch.empty((T, C // 128), device="cuda")}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    lm.rmsnorm(x, w, 1e-6, residual=res, residual_out=o["r"], y_fp8=o["c"], y_scales=o["s"], stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(o["r"], ref["r"]) and torch.equal(o["s"], ref["s"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lm.rmsnorm(x, w, 1e-6, residual=res, residual_out=o["r"], y_fp8=o["c"], y_scales=o["s"])
    for _ in range(3):
        o["s"].fill_(-1.0)
        o["r"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o["r"], ref["r"]) and torch.equal(o["s"], ref["s"])
        assert torch.equal(o["c"].view(torch.uint8), ref["c"].view(torch.uint8))


@pytest.mark.parametrize("what,rows", [("norm", (1 << 26) + 3), ("quantize", (1 << 28) + 5)])
def test_more_threads_than_one_grid_dimension_holds(what, rows):
    """2^32 threads and more, and elements past 2^32: short rows, of which a
    pattern of 1024 repeats."""
    C, n = 16, 1024
    base = _rows(np.random.default_rng(31), n, C, BF16)
    w = torch.from_numpy(np.random.default_rng(32).standard_normal(C).astype(np.float32)).cuda()

    def run(x):
        codes = torch.full(x.shape, 0x55, dtype=torch.uint8, device="cuda").view(F8)
        scales = torch.full((x.shape[0], 1), float("nan"), device="cuda")
        if what == "norm":
            lm.rmsnorm(x, w, 1e-5, y_fp8=codes, y_scales=scales)
        else:
            lm.quantize_fp8(x, codes, scales)
        torch.cuda.synchronize()
        return codes.view(torch.uint8), scales

    x = torch.empty(rows, C, dtype=BF16, device="cuda")
    whole = rows // n * n
    x[:whole].view(-1, n, C).copy_(base.expand(whole // n, n, C))
    x[whole:] = base[:rows - whole]
    codes, scales = run(x)
    del x
    c, s = run(base)
    for at in range(0, whole, n << 16):
        end = min(whole, at + (n << 16))
        assert (codes[at:end].view(-1, n, C) == c).all() and (scales[at:end].view(-1, n, 1) == s).all()
    assert torch.equal(codes[whole:], c[:rows - whole]) and torch.equal(scales[whole:], s[:rows - whole])
