"""GPU tests of the 16-bit products against the 64-bit oracle.

Whole-number inputs: every product and every partial sum is a whole number
below 2^24, so the fp32 sums are exact in any order, and outputs have to be
equal bit for bit.

Gaussian inputs: v = sum of K exact products + bias in fp32.  Each addition
rounds (or cuts) by at most 2^-23 of a partial sum, which is at most the sum
of magnitudes m: |v - v*| <= (K + 2) 2^-23 m.  The activations have slopes of
at most 1.13; what they add is, of |v|, 0.75e-7 for gelu (the formula), and for
exp(z) with |z| <= |v| + 0.1 |v|^3 a relative error of (2 + 2 |z|) 2^-23 of a
factor whose derivative in z is at most 1/4, with four operations around it:
|v| (8 + |z| exp(-|z|)...) 2^-23 <= |v| 12 2^-23.  A rounding to `type` is off by
half a step.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402
from oracle import rows16  # noqa: E402
from tests import _tiles16  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -23


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(g, shape, lo, hi):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").float()


def _apart(t, extra):
    """The same rows, `extra` values further apart, with NaN in between."""
    big = torch.full((t.shape[0] + 1, t.shape[1] + extra), float("nan"), dtype=t.dtype, device="cuda")
    v = big[:t.shape[0], :t.shape[1]]
    v.copy_(t)
    return v, big


def _out(T, N, kind, extra=0):
    return _apart(torch.full((T, N), float("nan"), dtype=TYPES[kind], device="cuda"), extra)


def _untouched(v, big):
    assert torch.isnan(big[v.shape[0]:]).all() and torch.isnan(big[:, v.shape[1]:]).all()


# around every boundary of tokens (1, 4, 8, 16, 32, 64, 128, 192, 256), of weight rows and of steps of K
CASES = [(1, 1, 8), (1, 128, 4096), (2, 17, 64), (3, 100, 72), (4, 4, 136), (4, 128, 1000), (4, 4096, 512), (5, 33, 256),
         (8, 130, 2056), (9, 64, 64), (15, 257, 88), (16, 48, 1024), (17, 96, 520), (31, 1000, 64), (32, 128, 2048),
         (33, 16, 128), (63, 65, 200), (64, 64, 8), (65, 128, 1096), (100, 20, 3000), (127, 250, 120), (129, 300, 192),
         (191, 512, 256), (257, 258, 264), (300, 1024, 320), (517, 516, 136), (700, 129, 72), (1030, 770, 448),
         (2049, 40, 104), (1500, 2304, 64), (3001, 1100, 128)]


@pytest.mark.parametrize("T,N,K", CASES, ids=str)
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_dense_whole_numbers(T, N, K, kind):
    """Bit for bit, with rows apart, bias, ReLU and a residual in place."""
    g = _gen(T * 7 + N * 3 + K)
    x, w = _ints(g, (T, K), -4, 4).to(TYPES[kind]), _ints(g, (N, K), -5, 5).to(TYPES[kind])
    bias, res = _ints(g, (N,), -50, 50), _ints(g, (T, N), -90, 90)
    ref, mag = rows16.product(x, w, bias)
    assert mag.max() < 2 ** 24
    y, big = _out(T, N, "f32")
    lm.dense_16(x, w, bias=bias, y=y)
    torch.cuda.synchronize()
    assert torch.equal(y.double(), ref)
    _untouched(y, big)
    # ReLU and residual, rows apart; every type of y, the residual in place
    ref = rows16.dense(x, w, bias, "relu", res)
    xa, _ = _apart(x, 24)
    for out in ("f32", "bf16", "f16"):
        for extra in (8, 3):
            y, big = _apart(res.to(TYPES[out]), extra)
            lm.dense_16(xa, w, bias=bias, activation="relu", residual=y, y=y)
            torch.cuda.synchronize()
            assert torch.equal(y, ref.float().to(TYPES[out])), (out, extra)
            _untouched(y, big)


@pytest.mark.parametrize("T,N,K", CASES, ids=str)
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_gated_whole_numbers(T, N, K, kind):
    g = _gen(T * 5 + N + K)
    # |gate|, |up| <= 4096: their product is below 2^24
    lim = max(1, int((4000 / K) ** 0.5)) if K < 4000 else 1
    x, w = _ints(g, (T, K), -lim, lim), _ints(g, (2 * N, K), -1, 1)
    keep = min(1.0, 2000 / (K * lim))
    w *= torch.rand(w.shape, generator=g, device="cuda") < keep
    x, w, bias = x.to(TYPES[kind]), w.to(TYPES[kind]), _ints(g, (2 * N,), -9, 9)
    ref = rows16.gated(x, w, bias, "relu")
    assert rows16.product(x, w, bias)[1].max() < 4096 and ref.abs().max() < 2 ** 24
    for out, extra in (("f32", 0), ("f32", 8), ("bf16", 0), ("f16", 5)):
        h, big = _out(T, N, out, extra)
        lm.gated_16(x, w, h, bias=bias, activation="relu")
        torch.cuda.synchronize()
        assert torch.equal(h, ref.float().to(TYPES[out])), (out, extra)
        _untouched(h, big)


@pytest.mark.parametrize("case,variants", _tiles16.RAGGED, ids=str)
def test_every_tile_whole_numbers(case, variants):
    """Each tile, and two launches in a row, with ragged ends: both products, bit for bit."""
    T, N, K = case
    g = _gen(T + N + K)
    kind, other = (torch.bfloat16, torch.float16) if T % 2 else (torch.float16, torch.bfloat16)
    x, w = _ints(g, (T, K), -3, 3).to(kind), _ints(g, (N, K), -1, 1)
    w *= torch.rand(w.shape, generator=g, device="cuda") < min(1.0, 600 / K)
    w, bias, res = w.to(kind), _ints(g, (N,), -50, 50), _ints(g, (T, N), -90, 90)
    v, mag = rows16.product(x, w, bias)
    assert mag.max() < 4096
    xa, _ = _apart(x, 8)
    # plain, then with everything and rows of an odd length: fp32 from fp32, the operands' type from it, the other one
    y, big = _out(T, N, "f32", 1)
    lm.dense_16(xa, w, bias=bias, y=y)
    torch.cuda.synchronize()
    assert torch.equal(y.double(), v)
    _untouched(y, big)
    del y, big
    ref = (rows16.activation(v, "relu") + res).float()
    for out in (torch.float32, kind, other):
        y, big = _apart(res.to(out), 3)
        lm.dense_16(x, w, bias=bias, activation="relu", residual=y, y=y)
        torch.cuda.synchronize()
        assert torch.equal(y, ref.to(out)), out
        _untouched(y, big)
    y = torch.empty(T, N, dtype=kind, device="cuda")
    lm.dense_16(x, w, bias=bias, activation="relu", residual=res, y=y)
    torch.cuda.synchronize()
    assert torch.equal(y, ref.to(kind))
    F = N // 2
    ref = (rows16.activation(v[:, :F], "relu") * v[:, F:]).float()
    for out in (torch.float32, kind):
        h, big = _apart(torch.full((T, F), float("nan"), dtype=out, device="cuda"), 5)
        lm.gated_16(xa, w, h, bias=bias, activation="relu")
        torch.cuda.synchronize()
        assert torch.equal(h, ref.to(out)), out
        _untouched(h, big)


@pytest.mark.parametrize("T,N,K", [(6007, 1312, 72), (3135, 1312, 72), (329, 5760, 72), (914, 4256, 80), (497, 3968, 712),
                                   (508, 992, 688), (4133, 4128, 2056)], ids=str)
def test_q8_1_rows_of_every_tile(T, N, K):
    g = _gen(T)
    x, w = torch.randn(T, K, generator=g, device="cuda").half(), torch.randn(N, K, generator=g, device="cuda").half()
    y, q = torch.empty(T, N, device="cuda"), torch.full((T, N // 32, 36), 9, dtype=torch.uint8, device="cuda")
    beside, want = q.clone(), q.clone()
    lm.dense_16(x, w, y_q8_1=q)
    lm.dense_16(x, w, y=y, y_q8_1=beside)
    lm.quantize_q8_1(y, want)
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(beside, want)


def _act_tol(v, e):
    """e: the error of v.  The activation's slope, its formula, and its arithmetic."""
    return 1.13 * e + v.abs() * (0.75e-7 + 12 * U)


@pytest.mark.parametrize("T,N,K", [(1, 40, 64), (4, 128, 4096), (13, 300, 1000), (30, 72, 512), (200, 96, 2048),
                                   (333, 1025, 264), (1100, 640, 136)], ids=str)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_gaussian_within_the_bound(T, N, K, act):
    g = _gen(T + N + K)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    for kind, out in (("bf16", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f16", "f16")):
        x, w = rnd(T, K).to(TYPES[kind]), (2 * rnd(2 * N, K) * K ** -0.5).to(TYPES[kind])
        bias, res = rnd(2 * N), rnd(T, N).to(TYPES[out])
        v, mag = rows16.product(x, w, bias)
        e = (K + 2) * U * mag
        half = torch.finfo(TYPES[out]).eps / 2
        y, _ = _out(T, N, out)
        lm.dense_16(x, w[:N], bias=bias[:N], activation=act, residual=res, y=y)
        h, _ = _out(T, N, out)
        lm.gated_16(x, w, h, bias=bias, activation=act)
        torch.cuda.synchronize()
        a, ea = rows16.activation(v[:, :N], act), _act_tol(v[:, :N], e[:, :N])
        ref = a + res.double()
        tol = ea + U * ref.abs()
        assert ((y.double() - ref).abs() <= tol + half * (ref.abs() + tol)).all(), (kind, out)
        ref = a * v[:, N:]
        tol = ea * (v[:, N:].abs() + e[:, N:]) + a.abs() * e[:, N:] + U * ref.abs()
        tiny = torch.finfo(TYPES[out]).smallest_normal * half  # below it a step no longer shrinks
        assert ((h.double() - ref).abs() <= tol + half * (ref.abs() + tol) + tiny).all(), (kind, out)
        # what the sums lose is far below their bound: rounding errors of either sign
        if out == "f32" and act == "none":
            off = (y.double() - v[:, :N] - res.double()).square().mean().sqrt() / v.square().mean().sqrt()
            assert off < 2e-6


@pytest.mark.parametrize("T,N,K", [(1, 32, 64), (4, 1024, 4096), (20, 96, 320), (130, 64, 1000), (600, 1056, 520)], ids=str)
def test_q8_1_rows(T, N, K):
    """The bytes that quantize_q8_1 makes of the fp32 y, alone and beside it."""
    g = _gen(T + K)
    x, w = torch.randn(T, K, generator=g, device="cuda").bfloat16(), torch.randn(N, K, generator=g, device="cuda").bfloat16()
    w[:32] = 0  # blocks of zeros
    res = torch.randn(T, N, generator=g, device="cuda").half()
    res[:, :32] = 0
    y, q = torch.full((T, N), float("nan"), device="cuda"), torch.full((T, N // 32, 36), 9, dtype=torch.uint8, device="cuda")
    alone, want = q.clone(), q.clone()
    lm.dense_16(x, w, activation="silu", residual=res, y=y, y_q8_1=q)
    lm.dense_16(x, w, activation="silu", residual=res, y_q8_1=alone)
    lm.quantize_q8_1(y, want)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and torch.equal(q, want) and torch.equal(alone, want)


@pytest.mark.parametrize("T", [3, 16, 40, 300])
def test_nan_and_infinity_stay_where_they_are(T):
    g = _gen(T)
    N, K = 150, 200
    x, w = torch.randn(T, K, generator=g, device="cuda").half(), torch.randn(2 * N, K, generator=g, device="cuda").half()
    y0, h0 = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
    lm.dense_16(x, w[:N], activation="gelu", y=y0)
    lm.gated_16(x, w, h0)
    for value in (float("nan"), float("inf")):
        xn, wn = x.clone(), w.clone()
        xn[T - 1, K - 1] = value
        wn[7, 0] = value
        y, h = torch.empty_like(y0), torch.empty_like(h0)
        lm.dense_16(xn, wn[:N], activation="gelu", y=y)
        lm.gated_16(xn, wn, h)
        torch.cuda.synchronize()
        for a, b in ((y, y0), (h, h0)):
            hit = torch.zeros(T, N, dtype=torch.bool, device="cuda")
            hit[T - 1] = True
            hit[:, 7] = True
            assert torch.equal(a[~hit], b[~hit])
            if value != value:
                assert torch.isnan(a[hit]).all()
    # a NaN output's q8_1 block has a NaN scale, other blocks are as they were
    xn = x.clone()
    xn[0, 0] = float("nan")
    q0, q = (torch.empty(T, 2, 36, dtype=torch.uint8, device="cuda") for _ in range(2))
    lm.dense_16(x, w[:64], y_q8_1=q0)
    lm.dense_16(xn, w[:64], y_q8_1=q)
    torch.cuda.synchronize()
    assert torch.isnan(q[0, :, :2].contiguous().view(torch.float16)).all() and torch.equal(q[1:], q0[1:])
    # subnormal inputs count
    s = torch.full((T, 64), 2.0 ** -24, device="cuda").half()
    y = torch.empty(T, 64, device="cuda")
    lm.dense_16(s, torch.ones(64, 64, device="cuda").half(), y=y)
    torch.cuda.synchronize()
    assert (y == 64 * 2.0 ** -24).all()


def test_empty_and_offsets_past_32_bits():
    lm.dense_16(torch.empty(0, 64, device="cuda").half(), torch.zeros(8, 64, device="cuda").half(),
                y=torch.empty(0, 8, device="cuda"))
    # rows of x and y that begin past 2^32 bytes
    T, K, N = 2100, 64, 40
    base = torch.zeros(T, 1 << 20, device="cuda", dtype=torch.bfloat16)
    x = base[:, (1 << 20) - K:]
    g = _gen(1)
    x.copy_(_ints(g, (T, K), -9, 9))
    w = _ints(g, (N, K), -9, 9).bfloat16()
    out = torch.zeros(T, 1 << 20, device="cuda")
    y = out[:, :N]
    lm.dense_16(x, w, y=y)
    torch.cuda.synchronize()
    assert torch.equal(y.double(), x.double() @ w.double().t()) and (out[:, N:].abs().amax() == 0)


def test_two_streams_and_a_graph():
    """Calls in flight on two streams, and captured ones replayed with eager
    work in between, give what they give alone."""
    g = _gen(2)
    shapes = [(4, 512, 1024), (40, 256, 512), (400, 700, 320)]
    sets = []
    for T, N, K in shapes:
        x, w = torch.randn(T, K, generator=g, device="cuda").half(), torch.randn(2 * N, K, generator=g, device="cuda").half()
        sets.append((x, w, torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda").half()))

    def run():
        for x, w, y, h in sets:
            lm.dense_16(x, w[:y.shape[1]], activation="silu", y=y)
            lm.gated_16(x, w, h)

    run()
    torch.cuda.synchronize()
    want = [(y.clone(), h.clone()) for _, _, y, h in sets]
    same = lambda: all(torch.equal(y, a) and torch.equal(h, b) for (_, _, y, h), (a, b) in zip(sets, want))  # noqa: E731
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()
    for s in side:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    busy = torch.randn(1 << 20, device="cuda")
    for _ in range(4):
        for _, _, y, h in sets:
            y.fill_(float("nan"))
            h.fill_(float("nan"))
        graph.replay()
        busy.mul_(1.0001)
        torch.cuda.synchronize()
        assert same()


def test_binding_refuses_what_the_call_does_not_say():
    x, w, y = torch.zeros(4, 64, device="cuda").half(), torch.zeros(96, 64, device="cuda").half(), torch.zeros(4, 96, device="cuda")
    for call, what in ((lambda: lm.gated_16(x, w[:95], y), "gate rows"), (lambda: lm.gated_16(x, w, y), "shape"),
                       (lambda: lm.dense_16(x, w.bfloat16(), y=y), "w: expected"), (lambda: lm.dense_16(x, w.t(), y=y), "w: expected"),
                       (lambda: lm.dense_16(x, w, y=y[:3]), "shape"), (lambda: lm.dense_16(x, w, y=y.double()), "float32"),
                       (lambda: lm.dense_16(x, w, y=y.t().contiguous().t()), "neighbours"),
                       (lambda: lm.dense_16(x.t().contiguous().t(), w, y=y), "neighbours"),
                       (lambda: lm.dense_16(x, w, y=y, bias=torch.zeros(95, device="cuda")), "bias"),
                       (lambda: lm.dense_16(x, w, y=y, residual=y.cpu()), "current GPU"),
                       (lambda: lm.dense_16(x, w, y=y, activation="swish"), "activation")):
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(lm.LatMoeError):  # nothing to write
        lm.dense_16(x, w)
    with pytest.raises(lm.LatMoeError):  # rows of x that do not begin at a multiple of 16 bytes
        lm.dense_16(torch.zeros(4, 68, device="cuda").half()[:, :64], w, y=y)
