"""The limited waits of the products and the distillation kernels on the GPU."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_mask_search_b200 as tsl  # noqa: E402


def _ones(rows, cols):
    return torch.full((rows, cols), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)     # code of 1


@pytest.mark.parametrize("m", [1, 100, 2048])
def test_product_behind_a_long_one_on_few_sms(m):
    # the first takes some 250 ms on 8 SMs; the second starts early on the others and waits for it
    k = 2 ** 30
    scales = torch.full(tsl.scale_shape(1, k), 127, dtype=torch.uint8, device="cuda")
    long = tsl.QuantizedMatrix(_ones(1, k), scales)
    x, w = torch.randn((m, 4096), device="cuda"), torch.randn((4096, 4096), device="cuda")
    a, b = tsl.tsenor_quantize(x), tsl.tsenor_quantize(w, "tile")
    want = tsl.tsenor_matmul(a, b)
    tsl.tsenor_matmul(long, long, dtype=torch.float32)
    got = tsl.tsenor_matmul(a, b)
    assert torch.equal(got, want)
    assert tsl.tsenor_error_count() == 0
