"""The choice of e4m3 tiles (CPU): the cases that the GPU tests walk through take
the tiles that they are meant for."""
import pytest

from tests import _tiles


@pytest.mark.parametrize("product,tile,T,N,K", _tiles.WALKS)
def test_walks_take_their_tile_and_a_second_one(product, tile, T, N, K):
    c = _tiles.choose(product, T, N, K)
    nb = -(-K // 128)
    assert (c.cols, c.tokens) == tile and c.stays
    assert c.tiles > 256 and c.tiles % 256
    assert nb > 4 and nb % 4 and K % 128 and T % c.tokens and N % c.cols


def test_every_tile_that_stays_is_walked():
    walked = {(p, _tiles.choose(p, T, N, K).variant) for p, _, T, N, K in _tiles.WALKS}
    seen = {(p, c.variant): c.stays for p in range(4) for T in (17, 64, 300, 700, 2100, 4133, 9000, 21000)
            for N in (64, 272, 1024, 2064, 4096, 8192) for K in (128, 656, 4096) for c in [_tiles.choose(p, T, N, K)]}
    assert len(seen) == 4 + 3 + 4 + 2                  # every variant is taken by some product
    assert walked == {k for k, stays in seen.items() if stays}
