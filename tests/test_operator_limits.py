"""Descriptions of the experts' products at their limits, on the host."""
import pytest

import permute_ep_layout_amd as epl

pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    epl.ensure_built()
    epl.load()


def product(rows, expected=0, E=8, K=2048, N=1024):
    return epl.Product(rows, expected, E, K, N, 0, 0, 1, 0)


@pytest.mark.parametrize("rows", [8, 800, 4096, 9000])
def test_weight_gradient_goes_by_the_expected_rows(rows):
    """A buffer of the receive side's capacity with `rows` of them used takes
    the workspace, and so the kernel, that the rows by themselves would."""
    size = epl.epl_weight_grad_workspace_bytes
    assert size(product(65536, expected=rows)) == size(product(rows))
    assert size(product(65536, expected=1 << 40)) == size(product(65536))
    sizes = {size(product(n)) for n in (8, 4096, 65536)}
    assert len(sizes) > 1                     # (they differ)


def test_rows_that_32_bit_counts_cannot_step_past():
    """Kernels advance by tiles: a block that ended at the last 32-bit count
    would be stepped over, so such buffers are refused."""
    most = 2 ** 31 - 1
    for rows in (most, most - 31, most - 1022):
        p = product(rows, K=8, N=8)
        assert epl.epl_product_validate(p) == epl.EPL_EINVAL
        assert epl.epl_product_workspace_bytes(p) == 0
    assert epl.epl_product_validate(product(most - 1023, K=8, N=8)) == epl.EPL_OK
