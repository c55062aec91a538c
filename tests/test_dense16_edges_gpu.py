"""GPU tests of the 16-bit tiles where they are seldom: K below one step, and
NaN, infinities and subnormal values inside the matrix and at its ends."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402
from oracle import rows16  # noqa: E402
from tests import _tiles16  # noqa: E402


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(g, shape, lo, hi):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").float()


@pytest.mark.parametrize("K", [8, 24, 56])
@pytest.mark.parametrize("T,N,variant", [(8127, 1306, 0), (6763, 1046, 1), (6625, 530, 2), (260, 6678, 3), (525, 6694, 4),
                                         (4225, 68, 5), (2051, 18, 6)], ids=str)
def test_less_than_one_step(K, T, N, variant):
    """The first step is the last one, and cut; whole numbers, bit for bit, with x's rows apart and NaN between them."""
    assert [v for v, _ in _tiles16.launches(T, N, K)] == [variant]
    g = _gen(T + K)
    kind = torch.bfloat16 if K == 24 else torch.float16
    wide = torch.full((T, K + 40), math.nan, device="cuda", dtype=kind)
    x, w, bias = wide[:, 16:16 + K], _ints(g, (N, K), -5, 5).to(kind), _ints(g, (N,), -50, 50)
    x.copy_(_ints(g, (T, K), -4, 4))
    v, _ = rows16.product(x, w, bias)
    y = torch.full((T, N), math.nan, device="cuda")
    lm.dense_16(x, w, bias=bias, y=y)
    h = torch.full((T, N // 2), math.nan, device="cuda")
    lm.gated_16(x, w, h, bias=bias, activation="relu")
    torch.cuda.synchronize()
    assert torch.equal(y.double(), v)
    assert torch.equal(h.double(), v[:, :N // 2].clamp(min=0) * v[:, N // 2:])


TILES = [((6007, 1312, 72), [1]), ((3135, 1312, 72), [2]), ((329, 5760, 72), [3]), ((914, 4256, 80), [4]),
         ((497, 3968, 712), [5]), ((508, 992, 688), [6]), ((4133, 4128, 2056), [0, 4])]


@pytest.mark.parametrize("case,variants", TILES, ids=str)
def test_nan_and_infinity_in_tiles(case, variants):
    """Each reaches its own row, column or element, and no other output changes by a bit."""
    T, N, K = case
    assert [v for v, _ in _tiles16.launches(T, N, K)] == variants
    g = _gen(T)
    kind = torch.bfloat16 if T % 2 else torch.float16
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, bias, res = rnd(T, K).to(kind), rnd(N, K).to(kind), rnd(N), rnd(T, N).to(kind)

    def run(x, w, bias, res):
        y, z, h = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda", dtype=kind), torch.empty(T, N // 2, device="cuda")
        q, beside = (torch.empty(T, N // 32, 36, dtype=torch.uint8, device="cuda") for _ in range(2))
        lm.dense_16(x, w, bias=bias, y=y)
        lm.dense_16(x, w, bias=bias, residual=res, y=z)
        lm.dense_16(x, w, y_q8_1=q)
        lm.dense_16(x, w, bias=bias, residual=res, y=torch.empty_like(y), y_q8_1=beside)
        lm.gated_16(x, w, h, bias=bias, activation="relu")
        torch.cuda.synchronize()
        return y, z, h, q, beside

    clean = run(x, w, bias, res)
    rows, cols = [5, T - 1], [7, N - 1]
    for value in (math.nan, math.inf):
        xn, wn, bn, rn = x.clone(), w.clone(), bias.clone(), res.clone()
        xn[5, 0], xn[T - 1, K - 1] = value, -value
        wn[7, K - 1], wn[N - 1, 0] = value, value
        bn[40] = value
        rn[9, 70], rn[T - 2, N - 2] = value, value
        dirty = run(xn, wn, bn, rn)
        of_x = torch.zeros(T, N, dtype=torch.bool, device="cuda")
        of_x[rows] = True
        of_x[:, cols] = True
        of_bias = of_x.clone()
        of_bias[:, 40] = True
        of_res = of_bias.clone()
        of_res[9, 70] = of_res[T - 2, N - 2] = True
        pair = of_bias[:, :N // 2] | of_bias[:, N // 2:]
        for a, b, hit in ((dirty[0], clean[0], of_bias), (dirty[1], clean[1], of_res), (dirty[2], clean[2], pair)):
            assert torch.equal(a[~hit], b[~hit])
            if value != value:
                assert torch.isnan(a[hit]).all()
            elif a is not dirty[2]:  # a gate product of -inf is cut to 0
                assert not torch.isfinite(a[hit]).any()
        for a, b, hit in ((dirty[3], clean[3], of_x), (dirty[4], clean[4], of_res)):
            block = hit.view(T, N // 32, 32).any(2)
            assert torch.equal(a[~block], b[~block])
            d = a[..., :2].contiguous().view(torch.float16)[..., 0][block]
            assert torch.isnan(d).all() if value != value else not torch.isfinite(d).any()


@pytest.mark.parametrize("case,variants", TILES, ids=str)
def test_subnormal_values_in_tiles(case, variants):
    """fp16 inputs below the smallest normal number count, and so do outputs."""
    T, N, K = case
    g = _gen(T + 1)
    x, w = (_ints(g, (T, K), -8, 8) * 2.0 ** -24).half(), _ints(g, (N, K), -3, 3).half()
    v, _ = rows16.product(x, w)
    y, z = torch.full((T, N), math.nan, device="cuda"), torch.full((T, N), math.nan, device="cuda").half()
    lm.dense_16(x, w, y=y)
    lm.dense_16(x, w, y=z)
    torch.cuda.synchronize()
    assert torch.equal(y.double(), v) and torch.equal(z, v.half())
