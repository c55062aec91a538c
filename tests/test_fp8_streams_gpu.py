"""GPU test of e4m3 products of the tile kernels in flight on two streams."""
import numpy as np
import pytest

from oracle import fp8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import quantized_latent_moe_amd as lm  # noqa: E402
from tests import _tiles  # noqa: E402
from tests.test_fp8_gpu import _dev, _ffn_inputs, _tol, _w  # noqa: E402


def test_tiles_at_once_on_two_streams():
    """A gated block and two projections (e4m3 and exact products) of each of two
    cases, a stream each, all by tile kernels: every call gives what it gives
    alone, and the projections what the oracle says."""
    rng = np.random.default_rng(78)
    cases, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for T, C, F, N in ((700, 656, 1040, 2070), (2100, 400, 512, 1056)):
        assert _tiles.choose(_tiles.DENSE_EXACT, T, N, C).tiles > 100 and N * T > 256 * 16 * 32
        ffn, dense = _ffn_inputs(rng, T, C, F), _w(rng, N, C)
        work = torch.empty(lm.ffn_fp8_workspace_size(T, C, F), dtype=torch.uint8, device="cuda")
        out = [(torch.full((T, C), float("nan"), dtype=torch.bfloat16, device="cuda"),
                torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda"),
                torch.full((T, N), float("nan"), device="cuda")) for _ in range(9)]
        cases.append((ffn, dense, tuple(map(_dev, ffn)), tuple(map(_dev, dense)), work, out))

    def run(case, i):
        _, _, ffn, dense, work, out = case
        y, b, f = out[i]
        lm.ffn_fp8(*ffn, work, y_bf16=y)
        lm.dense_fp8(*ffn[:2], *dense, y_bf16=b)
        lm.dense_fp8(*ffn[:2], *dense, y_f32=f)

    for case in cases:
        run(case, 0)
    torch.cuda.synchronize()
    for i in range(1, 9):
        for case, stream in zip(cases, streams):
            with torch.cuda.stream(stream):
                run(case, i)
    torch.cuda.synchronize()
    for ffn, dense, _, _, _, out in cases:
        for i in range(1, 9):
            assert all(torch.equal(a, b) for a, b in zip(out[0], out[i]))
        assert torch.isfinite(out[0][0]).all()
        ref, mag = fp8.dense(ffn[0], ffn[1], *dense)
        assert (np.abs(out[0][2].cpu().numpy() - ref) <= _tol(ref, mag, ffn[0].shape[1])).all()
        f = out[0][2].double()
        assert ((out[0][1].double() - f).abs() <= f.abs() * 2.0 ** -8 + f.square().mean().sqrt() * 1e-2).all()
