"""GPU test of a latent-MoE layer's run of the 16-bit operators with the stage:
norm, router's logits, routing, latent D to q8_1, expert stage, latent U onto
the residual stream, and the shared expert, stage by stage against the oracle
and captured in a graph."""
import numpy as np
import pytest

import oracle
from oracle import rows16
from quantized_latent_moe_amd.inputs import Workload, make_inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402


@pytest.mark.parametrize("T", [4, 150])
def test_layer(T):
    wl = Workload("layer", T=T, L=256, F=96, E=16, k=2)
    I = make_inputs(wl)
    H, S = 512, 320  # hidden width, shared expert's width
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, gain = rnd(T, H).bfloat16(), 1 + 0.1 * rnd(H)
    wr, wd, wu = ((rnd(n, k) * k ** -0.5).bfloat16() for n, k in ((wl.E, H), (wl.L, H), (H, wl.L)))
    wgu, wdn = (rnd(2 * S, H) * H ** -0.5).bfloat16(), (rnd(H, S) * S ** -0.5).bfloat16()
    rbias = 0.05 * rnd(wl.E)
    gu, dn = torch.from_numpy(I.gateup_q3k).cuda(), torch.from_numpy(I.down_iq4nl).cuda()
    shapes = lm.shapes(T, wl.L, wl.F, wl.E, wl.k)
    ws = torch.empty(lm.workspace_size(shapes), dtype=torch.uint8, device="cuda")
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    n, logits, idx, w = bf(T, H), f32(T, wl.E), torch.empty(T, wl.k, dtype=torch.int32, device="cuda"), f32(T, wl.k)
    z, y, yb = torch.empty(T, wl.L // 32, 36, dtype=torch.uint8, device="cuda"), f32(T, wl.L), bf(T, wl.L)
    routed, h, out = bf(T, H), bf(T, S), bf(T, H)

    def layer():
        lm.rmsnorm(x, gain, 1e-6, y=n)
        lm.dense_16(n, wr, y=logits)
        lm.router_topk_ex(logits, wl.k, idx, w, bias=rbias, score="sigmoid", groups=4, top_groups=2, scale=1.5)
        lm.dense_16(n, wd, y_q8_1=z)
        lm.expert_forward(z, idx, w, gu, dn, shapes, y, ws)
        yb.copy_(y)
        lm.dense_16(yb, wu, residual=x, y=routed)
        lm.gated_16(n, wgu, h)
        lm.dense_16(h, wdn, residual=routed, y=out)

    layer()
    torch.cuda.synchronize()
    near = lambda a, ref, mag, K, eps: ((a.double() - ref).abs() <= (K + 8) * 2.0 ** -23 * mag + eps / 2 * (ref.abs() + 1e-6)).all()  # noqa: E731
    ref, mag = rows16.product(n, wr)
    assert near(logits, ref, mag, H, 0)
    ridx, rw = rows16.router(logits, wl.k, rbias, "sigmoid", 4, 2, "top2", True, 1.5)
    assert torch.equal(idx, ridx) and ((w.double() - rw).abs() <= 3 * 2.0 ** -24 * rw).all()
    lat = f32(T, wl.L)
    want = torch.empty_like(z)
    lm.dense_16(n, wd, y=lat)
    lm.quantize_q8_1(lat, want)
    assert torch.equal(z, want) and near(lat, *rows16.product(n, wd), H, 0)
    st = oracle.forward(z.cpu().numpy(), idx.cpu().numpy(), w.cpu().numpy(), I.gateup_q3k, I.down_iq4nl, wl.L, wl.F, wl.E)
    err = float(np.abs(y.cpu().numpy() - st.y).max() / np.sqrt(np.mean(st.y ** 2)))
    assert err <= 1e-2
    eps = 2.0 ** -7
    ref, mag = rows16.product(yb, wu)
    assert near(routed, ref + x.double(), mag + x.double().abs(), wl.L, eps)
    v, mag = rows16.product(n, wgu)
    ref = rows16.activation(v[:, :S], "silu") * v[:, S:]
    e = (H + 16) * 2.0 ** -23 * mag
    assert ((h.double() - ref).abs() <= 1.2 * e[:, :S] * (v[:, S:].abs() + e[:, S:]) + v[:, :S].abs() * e[:, S:] + eps / 2 * ref.abs() + 1e-6).all()
    ref, mag = rows16.product(h, wdn)
    assert near(out, ref + routed.double(), mag + routed.double().abs(), S, eps)

    want = [t.clone() for t in (logits, idx, w, z, y, routed, h, out)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    busy = torch.randn(1 << 20, device="cuda")
    for _ in range(3):
        for t in (logits, idx, w, z, y, routed, h, out):
            t.zero_()
        graph.replay()
        busy.mul_(1.0001)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((logits, idx, w, z, y, routed, h, out), want))
