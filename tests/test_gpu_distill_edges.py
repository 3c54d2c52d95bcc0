"""The distillation calls where numbers leave the ordinary range: logits that are not finite in rows without
entries."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_mask_search_b200 as tsl  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# few rows (slices of a cluster), many (a row to a block, wide and narrow), rows that start off 16 bytes
@pytest.mark.parametrize("rows,vocab", [(8, 9), (8, 3001), (8, 200000), (160, 40000), (700, 5001)])
@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("dtype", TYPES)
def test_lse_of_rows_without_entries_is_that_of_their_logits(rows, vocab, top, dtype):
    z = torch.randn((rows, vocab), generator=_gen(1), device="cuda").to(TYPES[dtype])
    z[1, vocab // 2] = torch.nan
    z[2, 0] = torch.inf
    z[3, vocab - 1], z[3, 1] = torch.inf, torch.nan
    z[4] = -torch.inf
    z[5] = -torch.inf
    z[5, vocab // 3] = torch.nan
    z[6, : vocab // 2] = -torch.inf
    z[7] = torch.inf
    index = torch.full((rows, top), -1, dtype=torch.int32, device="cuda")
    loss, lse = tsl.tsenor_distill_loss(z, index, torch.zeros((rows, top), device="cuda"), 2.0)
    want = torch.logsumexp(z.double() / 2, 1)
    assert torch.equal(lse.isnan(), want.isnan())
    assert torch.equal(lse.isposinf(), want.isposinf()) and torch.equal(lse.isneginf(), want.isneginf())
    fine = want.isfinite()
    # sums of one thread's share and the tree, as for any row
    tol = 2.0 ** -24 * (4 * want.abs() + vocab / 256 + 128)
    assert bool(((lse.double() - want).abs()[fine] <= tol[fine]).all())
    assert bool((loss == 0).all())
    assert tsl.tsenor_error_count() == 0
