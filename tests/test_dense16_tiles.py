"""The choice of the 16-bit products' tiles (CPU): the cases that the GPU tests
take have the variants that they are meant for, and all variants are among them."""
import pytest

from tests import _tiles16


@pytest.mark.parametrize("case,variants", _tiles16.RAGGED, ids=str)
def test_ragged_cases_take_their_variants(case, variants):
    got = _tiles16.launches(*case)
    assert [v for v, _ in got] == variants
    if len(got) > 1:
        assert got[0][1] % 256 == 0 and got[0][1] < case[0]


def test_every_variant_is_there():
    assert {v[0] for _, v in _tiles16.RAGGED} == set(range(7))
    taken = {v for T in (17, 64, 300, 517, 1100, 5268, 21000) for N in (64, 1024, 2064, 4100, 8192) for K in (64, 656, 4096)
             for v, _ in _tiles16.launches(T, N, K)}
    assert taken == set(range(-1, 7))


def test_streaming_kernel_fills_the_chip():
    for T, N, rows in ((1, 128, 4), (4, 1024, 4), (4, 2048, 8), (8, 8192, 8), (16, 2048, 8), (16, 8192, 16), (64, 1024, 16)):
        assert _tiles16.launches(T, N, 4096) == [(-1, rows)]
