"""GPU tests of the activations of the 16-bit products, apart from the sums.

v is exact in fp32: of every row of x one value is not 0, so that a product of
two 16-bit values is the sum, and the bias adds one rounding, which the
reference makes too.  What is left is the activation's own error, held to the
bounds that the header states:

  gelu       1e-7 |v|, and 1e-5 of itself for v >= -6
  silu, gelu_tanh, v s(z) with the logistic function s and z = v or
             2 sqrt(2 / pi) (v + 0.044715 v^3): (5 + 4 max(-z, 0)) 2^-23 of
             themselves for z >= -87; beyond both are below 2e-36

The last: exp2 and the reciprocal are off by 1 ulp (2^-23), the sum and the
product by half of one; z log2(e) is off by 0.63 2^-23 z, z of the tanh by up to
2.75 2^-23 z, which the quotient takes times 1 - s(z), (1 - s(z)) z <= 0.28 for
z > 0.  fp32 outputs below 2^-126 are in steps of 2^-149.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402
from tests import _tiles16  # noqa: E402

U = 2.0 ** -23
STREAMED = [((1, 4099, 72), [-1]), ((4, 8192, 64), [-1]), ((7, 3000, 136), [-1]), ((16, 2050, 264), [-1]),
            ((60, 514, 72), [-1])]
EXTREME = [0.0, -0.0, 1e-45, -1e-40, 1e-20, -1e-7, 6.0, -6.0, -6.5, 12.0, -12.0, -13.5, 40.0, -40.0, 87.0, -87.0, -88.0,
           -89.0, -104.0, 1e4, -1e4, 1e18, -1e18, 3e38, -3e38]


def _reference(v, act):
    """The activation in 64 bits, and what the header allows."""
    v = v.double()
    if act == "gelu":
        ref = v * 0.5 * torch.special.erfc(-v * math.sqrt(0.5))
        own = torch.where(v >= -6, 1e-5 * ref.abs(), torch.full_like(v, math.inf))
        return ref, torch.minimum(1e-7 * v.abs(), own)
    z = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    ref = v * torch.sigmoid(z)
    # sigmoid in 64 bits keeps its relative accuracy for z < 0
    return ref, torch.where(z >= -87, (5 + 4 * (-z).clamp(min=0)) * U * ref.abs(), torch.full_like(v, 2e-36))


@pytest.mark.parametrize("case,variants", _tiles16.RAGGED + STREAMED, ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activation_within_the_stated_bound(case, variants, act):
    T, N, K = case
    assert [v for v, _ in _tiles16.launches(T, N, K)] == variants
    g = torch.Generator(device="cuda").manual_seed(T + 3 * N + K)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    kind = torch.bfloat16 if T % 2 else torch.float16
    x, w, k0 = torch.zeros(T, K, device="cuda", dtype=kind), rnd(N, K).to(kind), (5 * T) % K
    x[:, k0] = (torch.exp(0.7 * rnd(T)) * torch.sign(rnd(T))).to(kind)
    x[::7, k0] = 0  # there v is the bias
    bias = torch.where(torch.rand(N, generator=g, device="cuda") < 0.5, 4 * rnd(N), torch.exp(6 * rnd(N) - 6) * torch.sign(rnd(N)))
    bias[::3] = 0
    bias[1:1 + len(EXTREME)] = torch.tensor(EXTREME, device="cuda")[:N - 1]
    v = x[:, k0].float()[:, None] * w[:, k0].float() + bias
    y = torch.full((T, N), float("nan"), device="cuda")
    lm.dense_16(x, w, bias=bias, activation=act, y=y)
    torch.cuda.synchronize()
    ref, tol = _reference(v, act)
    bad = ((y.double() - ref).abs() > tol + 2.0 ** -148) | ~torch.isfinite(y)
    assert not bad.any(), (int(bad.sum()), v[bad][:4].tolist(), y[bad][:4].tolist(), ref[bad][:4].tolist())
    # the gated pair with up products of exactly one
    F = N // 2
    wg, bg = w.clone(), bias.clone()
    wg[F:], bg[F:] = 0, 1
    h = torch.full((T, F), float("nan"), device="cuda")
    lm.gated_16(x, wg[:2 * F], h, bias=bg[:2 * F], activation=act)
    torch.cuda.synchronize()
    bad = ((h.double() - ref[:, :F]).abs() > tol[:, :F] + 2.0 ** -148) | ~torch.isfinite(h)
    assert not bad.any(), (int(bad.sum()), v[:, :F][bad][:4].tolist(), h[bad][:4].tolist(), ref[:, :F][bad][:4].tolist())


def test_gelu_of_every_size():
    """A sweep of 32-bit values of either sign as biases, every size from 2^-30 to 2^5 and every 64th value between 1/64 and 8."""
    lo, hi = (torch.tensor([b]).view(torch.int32).item() for b in (1 / 64, 8.0))
    bits = torch.arange(lo, hi, 64, dtype=torch.int32, device="cuda")
    far = torch.exp2(-30 + 35 * torch.rand(1 << 18, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda"))
    v = torch.cat([bits.view(torch.float32), far])
    v = torch.cat([v, -v])
    v = v[:v.numel() // 8192 * 8192]
    x, w = torch.zeros(1, 8, device="cuda").bfloat16(), torch.zeros(1 << 20, 8, device="cuda").bfloat16()
    for part in v.split(1 << 20):
        n = part.numel()
        y = torch.empty(1, n, device="cuda")
        lm.dense_16(x, w[:n], bias=part, activation="gelu", y=y)
        torch.cuda.synchronize()
        ref, tol = _reference(part, "gelu")
        bad = (y[0].double() - ref).abs() > tol
        assert not bad.any(), (int(bad.sum()), part[bad][:4].tolist(), ((y[0].double() - ref).abs() / part.abs()).max().item())


@pytest.mark.parametrize("case,variants", [((300, 514, 72), [6]), ((329, 5746, 72), [3]), ((4, 514, 72), [-1])], ids=str)
def test_infinite_sums(case, variants):
    """v of +inf stays, of -inf is what the formula gives (-inf times 0), NaN stays; their neighbours are as without them."""
    T, N, K = case
    assert [v for v, _ in _tiles16.launches(T, N, K)] == variants
    g = torch.Generator(device="cuda").manual_seed(T)
    x, w = torch.randn(T, K, generator=g, device="cuda").half(), torch.randn(N, K, generator=g, device="cuda").half()
    bias = torch.zeros(N, device="cuda")
    there = [(3, math.inf), (200, -math.inf), (N - 1, math.nan), (N - 2, math.inf)]
    for act in ("none", "relu", "silu", "gelu", "gelu_tanh"):
        y, want = torch.empty(T, N, device="cuda"), torch.empty(T, N, device="cuda")
        lm.dense_16(x, w, bias=bias, activation=act, y=want)
        at = bias.clone()
        for n, value in there:
            at[n] = value
        lm.dense_16(x, w, bias=at, activation=act, y=y)
        torch.cuda.synchronize()
        assert (y[:, [3, N - 2]] == math.inf).all() and torch.isnan(y[:, N - 1]).all(), act
        low = y[:, 200]
        assert {"none": low == -math.inf, "relu": low == 0}.get(act, torch.isnan(low)).all(), act
        rest = torch.ones(N, dtype=torch.bool, device="cuda")
        rest[[n for n, _ in there]] = False
        assert torch.equal(y[:, rest], want[:, rest])
