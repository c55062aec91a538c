"""GPU tests of the routing by scores at its ends, against the 64-bit oracle:
groups of one and of a few experts with lanes that hold none, biases of the
type's lowest value, and picks whose scores are all 0."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402
from oracle import rows16  # noqa: E402

LOWEST = torch.finfo(torch.float32).min


def _check(logits, k, **kw):
    T = logits.shape[0]
    idx, w = torch.full((T, k), -7, dtype=torch.int32, device="cuda"), torch.full((T, k), math.nan, device="cuda")
    lm.router_topk_ex(logits, k, idx, w, **kw)
    torch.cuda.synchronize()
    ridx, rw = rows16.router(logits, k, **kw)
    assert torch.equal(idx, ridx)
    # quotients of fp32 scores in 64 bits, rounded once; a score may be a rounding off
    assert ((w.double() - rw).abs() <= 3 * 2.0 ** -24 * rw.abs() + 2.0 ** -149).all()
    return idx, w


@pytest.mark.parametrize("E,G,tg", [(1, 1, 1), (2, 2, 1), (5, 5, 3), (8, 8, 3), (16, 16, 5), (13, 13, 12), (33, 11, 4), (65, 13, 3),
                                    (66, 3, 2), (129, 3, 1), (130, 13, 2), (193, 1, 1), (195, 15, 7), (255, 5, 2), (256, 16, 1),
                                    (40, 40, 9), (257, 1, 1), (512, 64, 9), (1024, 32, 3)], ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_few_experts_a_group(E, G, tg, score):
    g = torch.Generator(device="cuda").manual_seed(E + G)
    logits = 2 * torch.randn(133, E, generator=g, device="cuda")
    logits[::9, ::2] = -math.inf
    bias = 0.2 * torch.randn(E, generator=g, device="cuda")
    most = min(tg * (E // G), 64)
    for k in sorted({1, min(16, most), most}):
        _check(logits, k, bias=bias, score=score, groups=G, top_groups=tg, group_score="max")
        if E // G > 1:
            _check(logits, k, bias=bias, score=score, groups=G, top_groups=tg, group_score="top2", renormalise=False, scale=0.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_lowest_biases(score):
    """A bias of the lowest finite value closes no expert, but its c is the lowest: as a group's second it counts as 0."""
    g = torch.Generator(device="cuda").manual_seed(4)
    logits = torch.randn(300, 64, generator=g, device="cuda")
    for every in (2, 7):
        bias = 0.1 * torch.randn(64, generator=g, device="cuda")
        bias[::every] = LOWEST
        for mode in ("max", "top2"):
            for k in (8, 32):
                _check(logits, k, bias=bias, score=score, groups=8, top_groups=4, group_score=mode)
    # one open expert beside a lowest one: its group is ranked by it alone
    bias = torch.tensor([LOWEST, 0.0, -0.2, -0.2], device="cuda")
    idx, w = _check(torch.zeros(1, 4, device="cuda"), 2, bias=bias, score="sigmoid", groups=2, top_groups=1)
    assert idx.tolist() == [[2, 3]]
    idx, w = _check(torch.zeros(1, 4, device="cuda"), 2, bias=bias - torch.tensor([0, 0, 0.2, 0.2], device="cuda"), score="sigmoid",
                    groups=2, top_groups=1)
    assert idx.tolist() == [[1, 0]] and w.tolist() == [[0.5, 0.5]]


@pytest.mark.parametrize("E,k", [(8, 3), (64, 8), (300, 20)])
def test_scores_that_are_all_zero(E, k):
    """Sigmoids below 2^-150 are 0 in fp32: ids in order, weights 0 and not a quotient of zeros."""
    logits = torch.full((70, E), -200.0, device="cuda")
    logits[1::2, 1] = -110.0
    for renormalise in (True, False):
        idx, w = _check(logits, k, score="sigmoid", renormalise=renormalise)
        assert (w == 0).all() and idx[0].tolist() == list(range(k))
    # one pick with a score has all of the weight
    logits[:, 5] = -3.0
    idx, w = _check(logits, k, score="sigmoid", scale=2.5)
    assert (idx[:, 0] == 5).all() and (w[:, 0] == 2.5).all() and (w[:, 1:] == 0).all()
