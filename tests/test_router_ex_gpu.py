"""GPU tests of the routing by scores against the 64-bit oracle.

Ids have to be equal: both sides rank fp32 roundings of 64-bit scores, and
everything after that is comparisons and single fp32 additions.  Weights are
64-bit quotients of those scores, rounded once to fp32 and, as the scores may
differ by a rounding where 64-bit values lie next to a border, off by at most
three halves of a step: 3 * 2^-24 relative.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402
from oracle import rows16  # noqa: E402

INF = float("inf")


def _run(logits, k, **kw):
    T = logits.shape[0]
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), float("nan"), device="cuda")
    lm.router_topk_ex(logits, k, idx[:T], w[:T], **kw)
    torch.cuda.synchronize()
    assert (idx[T:] == -7).all() and torch.isnan(w[T:]).all()
    return idx[:T], w[:T]


def _check(logits, k, **kw):
    idx, w = _run(logits, k, **kw)
    ridx, rw = rows16.router(logits, k, **kw)
    bad = (idx != ridx).nonzero()
    assert not len(bad), (bad[:3].tolist(), idx[bad[0, 0]].tolist(), ridx[bad[0, 0]].tolist())
    assert ((w.double() - rw).abs() <= 3 * 2.0 ** -24 * rw.abs() + 2.0 ** -149).all()


SHAPES = [(1, 1, 1, 1, 1), (3, 8, 2, 1, 1), (5, 8, 8, 4, 4), (64, 16, 3, 2, 1), (4, 128, 8, 8, 4), (1000, 128, 8, 8, 4),
          (777, 256, 8, 8, 4), (300, 256, 16, 4, 1), (301, 64, 6, 1, 1), (129, 60, 5, 4, 2), (70, 96, 9, 3, 2),
          (255, 160, 6, 8, 3), (256, 192, 4, 64, 2), (33, 1024, 64, 64, 32), (10, 1024, 64, 2, 1), (40, 513, 7, 27, 3),
          (90, 24, 12, 2, 1), (4097, 32, 4, 4, 2), (50, 300, 33, 1, 1), (2, 1000, 40, 8, 5)]


@pytest.mark.parametrize("T,E,k,G,tg", SHAPES, ids=str)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ids_equal_and_weights_near(T, E, k, G, tg, score):
    g = torch.Generator(device="cuda").manual_seed(T + E + k)
    logits = torch.randn(T, E, generator=g, device="cuda") * (0.3 + 3 * torch.rand(T, 1, generator=g, device="cuda"))
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    for mode in ("max", "top2"):
        if mode == "top2" and E // G < 2 and tg < G:
            continue
        for b in (None, bias):
            _check(logits, k, bias=b, score=score, groups=G, top_groups=tg, group_score=mode)
    _check(logits, k, bias=bias, score=score, groups=G, top_groups=tg, group_score="max", renormalise=False, scale=2.5)


@pytest.mark.parametrize("T", [6, 500])
@pytest.mark.parametrize("E,k,G,tg", [(96, 8, 1, 1), (64, 6, 8, 2), (256, 8, 8, 4), (1024, 10, 4, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_and_closed_experts(T, E, k, G, tg, score):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = 0.5 * torch.randint(-2, 3, (T, E), generator=g, device="cuda").float()  # many exact ties
    logits[::5, 1::2] = -INF
    logits[1] = -INF                      # a row that leaves nothing
    logits[2] = -INF
    logits[2, [3, E // 2, E - 1]] = torch.tensor([1.0, 1.0, 0.5], device="cuda")  # fewer than k are left
    logits[3, : E // 2] = float("nan")
    logits[4, 2] = INF
    logits[5] = 3.0e38
    bias = 0.25 * torch.randint(-1, 2, (E,), generator=g, device="cuda").float()
    shut = bias.clone()
    shut[::3] = -INF
    shut[1] = float("nan")
    low = bias.clone()
    low[5:9] = torch.finfo(torch.float32).min
    high = bias.clone()
    high[5:9] = 3.4e38
    for b in (None, bias, shut, low, high):
        for mode in ("max", "top2"):
            _check(logits, k, bias=b, score=score, groups=G, top_groups=tg, group_score=mode, scale=-1.5)
    idx, w = _run(logits, k, score=score, groups=G, top_groups=tg)
    assert idx[1].tolist() == list(range(k)) and (w[1] == 0).all() and torch.isfinite(w).all()


def test_near_scores_keep_their_order():
    """Neighbouring fp32 logits: their scores differ in 64 bits and may round to one."""
    g = torch.Generator(device="cuda").manual_seed(3)
    base = torch.randn(2000, 1, generator=g, device="cuda").expand(2000, 128).contiguous().view(torch.int32)
    logits = (base + torch.randint(0, 4, (2000, 128), generator=g, device="cuda", dtype=torch.int32)).view(torch.float32)
    bias = 1e-7 * torch.randint(-2, 3, (128,), generator=g, device="cuda").float()
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            _check(logits, 8, bias=b, score=score)


def test_extreme_logits():
    logits = torch.tensor([[-1e30, 0.0, 1e30, 88.0, 89.0, -88.0, -104.0, -745.0],
                           [-746.0, -750.0, -1000.0, -3.4e38, -700.0, -120.0, -103.0, -87.5],
                           [17.0, 18.0, 16.9, 40.0, 800.0, 3.4e38, 16.0, 15.0]], device="cuda")
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            _check(logits, 8, score=score, renormalise=renormalise)


def test_graph_replays_and_streams():
    g = torch.Generator(device="cuda").manual_seed(9)
    sets = [(torch.randn(T, 128, generator=g, device="cuda"), torch.empty(T, 8, dtype=torch.int32, device="cuda"),
             torch.empty(T, 8, device="cuda")) for T in (4, 900)]
    bias = 0.1 * torch.randn(128, generator=g, device="cuda")

    def run():
        for l, i, w in sets:
            lm.router_topk_ex(l, 8, i, w, bias=bias, score="sigmoid", groups=8, top_groups=4)

    run()
    torch.cuda.synchronize()
    want = [(i.clone(), w.clone()) for _, i, w in sets]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    other, busy = torch.cuda.Stream(), torch.randn(1 << 18, device="cuda")
    for r in range(4):
        for _, i, w in sets:
            i.fill_(-1)
            w.fill_(float("nan"))
        if r < 3:
            graph.replay()
            busy.mul_(1.0001)
        else:
            other.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(other):
                run()
            torch.cuda.current_stream().wait_stream(other)
        torch.cuda.synchronize()
        assert all(torch.equal(i, a) and torch.equal(w, b) for (_, i, w), (a, b) in zip(sets, want))


def test_empty_batch_is_left_alone():
    lm.router_topk_ex(torch.empty(0, 8, device="cuda"), 2, torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                      torch.empty(0, 2, device="cuda"))
    torch.cuda.synchronize()
