"""The e4m3 oracle against closed forms and torch's own e4m3 conversion (CPU)."""
import numpy as np
import pytest

from oracle import fp8

torch = pytest.importorskip("torch")


def test_decode_matches_torch_on_every_code():
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.DECODE, ref, equal_nan=True)


def test_encode_rounds_to_nearest_even():
    mag = fp8.DECODE[:127]
    mid = (mag[1:] + mag[:-1]) / 2                       # every tie
    codes = fp8.encode(mid)
    assert (codes % 2 == 0).all() and (np.abs(fp8.decode(codes) - mid) == (mag[1:] - mag[:-1]) / 2).all()
    assert np.array_equal(fp8.encode(fp8.DECODE[:127]), np.arange(127))
    assert np.array_equal(fp8.encode(-fp8.DECODE[1:127]), np.arange(1, 127) + 128)
    v = np.random.default_rng(0).uniform(-448, 448, 20000).astype(np.float32)
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(v), ref)


@pytest.mark.parametrize("C", [16, 128, 144, 400])
def test_quantize_is_within_half_a_step(C):
    v = (np.random.default_rng(C).standard_normal((9, C)) * 3).astype(np.float32)
    v[3] = 0
    v[4] *= 1e-30
    codes, scales = fp8.quantize(v)
    assert scales.shape == (9, fp8.blocks(C)) and (scales[3] == fp8.SCALE_MIN).all() and (codes[3] == 0).all()
    s = np.repeat(scales.astype(np.float64), 128, 1)[:, :C]
    # half a step of a normal value is 2^-4 of it, of a subnormal one 2^-10 of the scale; the two fp32
    # roundings of v / scale move a value by 2^-23 more, and can turn a tie
    assert (np.abs(fp8.rows(codes, scales) - v) <= np.maximum(np.abs(v) * (2.0 ** -4 + 2.0 ** -22), s * 2.0 ** -10 * (1 + 2.0 ** -10))).all()


def test_rmsnorm_of_constant_rows():
    x = np.full((2, 64), 3.0, np.float32)
    v, y = fp8.rmsnorm(x, np.arange(64), 1e-30, np.full((2, 64), -1.0, np.float32))
    assert (v == 2).all() and np.allclose(y, np.arange(64)[None], rtol=1e-14)


def test_silu_product_extremes():
    h = fp8.silu_product(np.array([0.0, -800.0, 800.0, -2.0]), np.array([5.0, 3.0, 2.0, 1.0]))
    assert h[0] == 0 and abs(h[1]) < 1e-300 and h[2] == 1600 and np.isclose(h[3], -2 / (1 + np.exp(2.0)))
