"""The binding of the routing by scores (CPU): sizes that do not fit the call's 32 bits are refused, not cut to them."""
import pytest

import quantized_latent_moe_amd as lm

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("sizes", [dict(k=4 - (1 << 32)), dict(k=(1 << 32) + 4), dict(groups=1 - (1 << 32)), dict(groups=1 << 32),
                                   dict(top_groups=1 - (1 << 32)), dict(top_groups=(1 << 32) + 1)], ids=str)
def test_sizes_beyond_32_bits_are_refused(sizes):
    k = sizes.pop("k", 4)
    with pytest.raises(ValueError, match="sizes"):
        lm.router_topk_ex(torch.zeros(4, 64), k, torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4, 4), **sizes)
