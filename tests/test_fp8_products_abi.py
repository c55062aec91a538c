"""The choice of products of the e4m3 entry points: values outside the three
are refused before any HIP call (no GPU needed)."""
import pytest

import quantized_latent_moe_amd as lm

A = [0x10000 * (i + 1) for i in range(16)]  # aligned, never dereferenced on these paths
EINVAL = 1


@pytest.mark.parametrize("products", [-1, 3, 1 << 30])
def test_products_outside_the_three_are_refused(products):
    c = lm.lib()
    assert c.lat_moe_dense_fp8_ex(*A[:4], 4, 64, 64, A[4], None, None, products, None) == EINVAL
    need = lm.ffn_fp8_workspace_size(4, 64, 128)
    assert c.lat_moe_ffn_fp8_ex(*A[:6], 4, 64, 128, A[6], None, None, None, products, A[7], need, None) == EINVAL


@pytest.mark.parametrize("products", [0, 1, 2])
def test_no_rows_with_each_choice(products):
    c = lm.lib()
    assert c.lat_moe_dense_fp8_ex(*[None] * 4, 0, 64, 64, None, None, None, products, None) == 0
    assert c.lat_moe_ffn_fp8_ex(*[None] * 6, 0, 64, 128, None, None, None, None, products, None, 0, None) == 0


def test_the_other_checks_come_with_each_choice():
    c = lm.lib()
    for products in (0, 1, 2):
        assert c.lat_moe_dense_fp8_ex(*A[:4], 4, 64, 64, None, None, None, products, None) == EINVAL
        assert c.lat_moe_dense_fp8_ex(*A[:4], 4, 64, 72, A[4], None, None, products, None) == EINVAL
        assert c.lat_moe_ffn_fp8_ex(*A[:6], 4, 64, 128, A[6], None, None, None, products, A[7], 1, None) == 2


def test_binding_takes_true_false_or_none():
    assert [lm._products(v) for v in (None, True, False)] == [0, 1, 2]
    for bad in (2, 1, 0, "exact"):
        with pytest.raises(ValueError, match="True, False or None"):
            lm._products(bad)
