"""Pins of the 64-bit oracle of the 16-bit products and the routing by scores:
closed forms and brute force, without the GPU."""
import itertools
import math

import pytest

torch = pytest.importorskip("torch")

from oracle import rows16  # noqa: E402


def test_activations_closed_forms():
    v = torch.tensor([-3.0, -1.0, 0.0, 0.5, 2.0], dtype=torch.float64)
    for i, x in enumerate(v.tolist()):
        phi = 0.5 * (1 + math.erf(x / math.sqrt(2)))
        tanh = 0.5 * (1 + math.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
        want = {"none": x, "relu": max(x, 0.0), "silu": x / (1 + math.exp(-x)), "gelu": x * phi, "gelu_tanh": x * tanh}
        for name, y in want.items():
            assert abs(rows16.activation(v, name)[i].item() - y) < 1e-14, (name, x)


def test_products_by_loops():
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(3, 8, generator=g).bfloat16(), torch.randn(6, 8, generator=g).bfloat16()
    b, r = torch.randn(6, generator=g), torch.randn(3, 6, generator=g)
    y, h = rows16.dense(x, w, b, "silu", r), rows16.gated(x, w, b, "gelu")
    for t in range(3):
        v = [sum(float(x[t, k]) * float(w[n, k]) for k in range(8)) + float(b[n]) for n in range(6)]
        for n in range(6):
            assert abs(y[t, n].item() - (v[n] / (1 + math.exp(-v[n])) + float(r[t, n]))) < 1e-12
        for f in range(3):
            assert abs(h[t, f].item() - 0.5 * v[f] * (1 + math.erf(v[f] / math.sqrt(2))) * v[3 + f]) < 1e-12


def test_router_log_integers():
    """Softmax of ln(1..n) is i / sum: the weights of the picks are known."""
    l = torch.log(torch.tensor([[1.0, 4.0, 2.0, 3.0]]))
    idx, w = rows16.router(l, 2)
    assert idx.tolist() == [[1, 3]] and torch.allclose(w, torch.tensor([[4 / 7, 3 / 7]], dtype=torch.float64), atol=1e-7)
    idx, w = rows16.router(l, 2, renormalise=False, scale=2.0)
    assert torch.allclose(w, torch.tensor([[0.8, 0.6]], dtype=torch.float64), atol=1e-7)
    # a bias moves the picks, not the weights
    idx, w = rows16.router(l, 2, bias=torch.tensor([1.0, 0.0, 0.0, 0.0]), renormalise=False)
    assert idx.tolist() == [[0, 1]] and torch.allclose(w, torch.tensor([[0.1, 0.4]], dtype=torch.float64), atol=1e-7)


def test_router_groups_by_brute_force():
    g = torch.Generator().manual_seed(5)
    for trial in range(40):
        G, size = [(2, 3), (4, 2), (3, 4)][trial % 3]
        E, tg = G * size, 1 + trial % 2
        l, b = torch.randn(1, E, generator=g), 0.3 * torch.randn(E, generator=g)
        for mode in ("max", "top2"):
            idx, w = rows16.router(l, 2, b, "sigmoid", G, tg, mode, True, 1.5)
            c = (torch.sigmoid(l[0].double()).float() + b).tolist()
            sums = [sum(sorted(c[q * size:(q + 1) * size])[-(1 if mode == "max" else 2):]) for q in range(G)]
            groups = max(itertools.combinations(range(G), tg), key=lambda s: sum(sums[q] for q in s))
            picks = sorted((e for e in range(E) if e // size in groups), key=lambda e: -c[e])[:2]
            assert idx[0].tolist() == picks
            s = [1 / (1 + math.exp(-l[0, e].item())) for e in picks]
            assert all(abs(w[0, j].item() - 1.5 * s[j] / sum(s)) < 1e-6 for j in range(2))


def test_router_closed_experts():
    inf = math.inf
    l = torch.tensor([[0.0, -inf, 1.0, math.nan], [-inf, -inf, -inf, -inf], [inf, 0.0, 0.0, 0.0]])
    for score in ("softmax", "sigmoid"):
        idx, w = rows16.router(l, 3, score=score)
        assert idx.tolist() == [[2, 0, 1], [0, 1, 2], [0, 1, 2]]
        assert w[0, 2] == 0 and abs(w[0].sum().item() - 1) < 1e-12 and (w[1] == 0).all() and torch.isfinite(w).all()
    # closed by the bias; the second of a group counts as 0 where it is closed
    idx, w = rows16.router(torch.zeros(1, 4), 2, torch.tensor([-inf, 0.2, 0.0, -0.6]), "sigmoid", 2, 1)
    assert idx.tolist() == [[1, 0]] and w.tolist() == [[1.0, 0.0]]
