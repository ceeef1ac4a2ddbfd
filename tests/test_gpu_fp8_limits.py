"""The 8-bit casts and products at the ends of what their descriptions accept,
and the variants of their kernels that only large batches take, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

import permute_ep_layout_amd as epl  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    epl.load()


@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_more_weight_blocks_than_a_launch_has_workgroups(fmt):
    """2^24 blocks of 128 values, at 256 threads each: 2^32 threads. A block's
    largest is 448 times a power of two, and every step to its code is exact."""
    E, K = 2048, 1 << 20
    blocks = E * K // 128
    power = torch.arange(blocks, device=DEV) * 7 % 61 - 30
    w = torch.zeros(E, 1, K, dtype=torch.bfloat16, device=DEV)
    w.view(blocks, 128)[:, 5] = (448 * torch.exp2(power.double())).to(torch.bfloat16)
    codes = torch.full((E, 1, K), 0x5A, dtype=torch.uint8, device=DEV)
    scale = torch.full((E, 1, K // 128), 0x5A, device=DEV,
                       dtype=torch.uint8 if fmt == "ue8m0" else torch.float32)
    epl.quantize_weight(w, out=codes, out_scale=scale)
    del w
    made = codes.view(blocks, 128)
    assert (made[:, 5] == 0x7E).all()
    made[:, 5] = 0
    assert not made.any()
    want = power + 127 if fmt == "ue8m0" else torch.exp2(power.double())
    assert torch.equal(scale.view(-1), want.to(scale.dtype))
