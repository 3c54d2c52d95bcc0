"""The distillation calls where numbers leave the ordinary range: logits that are not finite in rows without
entries, temperatures far below 1 and logits far from 0."""
import numpy as np
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


def _reference(z, index, top_logits, temp, weight):
    """(gradient, how far fp32 may be from it), rows of entries only."""
    s, t = z.double() / temp, top_logits.double() / temp
    logp = t - torch.logsumexp(t, 1, keepdim=True)
    gap = s - torch.logsumexp(s, 1, keepdim=True)
    p, q = logp.exp(), gap.exp()
    i = index.long()
    w = temp * weight.double()[:, None]
    grad = w * (q - torch.zeros_like(s).scatter_add(1, i, p))
    # (z - max) / T is a difference (2^-24 of itself), a product with a rounded 1/T log2 e (three more), an exponential
    # (2^-22); the sum adds those of its terms, the additions of one thread's share and the tree. p likewise. What a
    # finite lse of up to 64 adds by its own rounding, 2^-24 of it, is among the 128.
    eps = 2.0 ** -24
    off = q * eps * (8 * gap.abs() + z.shape[1] / 256 + 128)
    off = off + torch.zeros_like(s).scatter_add(1, i, p * eps * (8 * logp.abs() + 4 * index.shape[1] + 64))
    half = torch.finfo(z.dtype).eps / 2
    tol = w * (off + 2.0 ** -120)                        # exponentials below 2^-126 are 0
    return grad, tol + half * (grad.abs() + tol) + torch.finfo(z.dtype).tiny


@pytest.mark.parametrize("rows,vocab,top", [(1, 2, 1), (3, 32000, 20), (2, 262144, 64), (300, 5003, 8), (300, 4096, 300)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("temp,shift,scale", [(0.1, 0.0, 30.0), (0.01, 0.0, 30.0), (1e-3, 0.0, 30.0), (1e-6, 0.0, 30.0), (1e-6, 0.0, 1e-5),
                                              (1.0, 1e4, 3.0), (1.0, -1e4, 3.0), (0.5, 1e6, 3.0), (1.0, 63.0, 3.0),
                                              (1e6, 0.0, 1e7), (1e37, 0.0, 1e37)])
def test_gradient_at_low_temperatures_and_far_logits(rows, vocab, top, dtype, temp, shift, scale):
    z = (torch.randn((rows, vocab), generator=_gen(2), device="cuda") * scale + shift).to(TYPES[dtype])
    teacher = z.float() + torch.randn((rows, vocab), generator=_gen(3), device="cuda") * temp
    value, index = teacher.topk(min(top, vocab), 1)
    index, value = index.to(torch.int32), value.contiguous()
    weight = torch.rand((rows,), generator=_gen(4), device="cuda")
    want, tol = _reference(z, index, value, float(np.float32(temp)), weight)
    _, lse = tsl.tsenor_distill_loss(z, index, value, temp)
    _, step = tsl.tsenor_distill_step(z, index, value, temp, weight=weight)
    grad = tsl.tsenor_distill_grad(z, index, value, lse, temp, weight=weight)
    for got in (step, grad):
        assert bool(((got.double() - want).abs() <= tol).all())
    assert torch.equal(grad, tsl.tsenor_distill_grad(z, index, value, lse, temp, weight=weight, grad=z))
    assert tsl.tsenor_error_count() == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_of_ordinary_and_far_rows_in_one_call(dtype):
    # rows of every kind beside one another, in place, rows off 16 bytes, a failing one among the far ones
    rows, vocab = 37, 70001
    buf = torch.zeros((rows, vocab + 3), dtype=TYPES[dtype], device="cuda")
    z = buf[:, 1:vocab + 1]
    z.copy_(torch.randn((rows, vocab), generator=_gen(5), device="cuda") * 3)
    z[::3] += 8192.0
    value, index = torch.topk(z.float(), 9, 1)
    index, value = index.to(torch.int32), value.contiguous()
    index[5] = -1
    z[9, 77] = torch.nan
    _, lse = tsl.tsenor_distill_loss(z, index, value)
    _, step = tsl.tsenor_distill_step(z, index, value)
    lse[9] = 8200.0                                      # what the row's lse would be without the NaN
    tsl.tsenor_error_count()
    grad = tsl.tsenor_distill_grad(z, index, value, lse)
    assert tsl.tsenor_error_count() == 1
    keep = torch.arange(rows, device="cuda") != 5
    keep[9] = False
    want, tol = _reference(z[keep], index[keep], value[keep], 1.0, torch.ones((int(keep.sum()),), device="cuda"))
    for got in (step, grad):
        assert bool(((got[keep].double() - want).abs() <= tol).all()) and bool((got[~keep] == 0).all())
    tsl.tsenor_distill_grad(z, index, value, lse, grad=z)
    assert torch.equal(z, grad) and bool((buf[:, 0] == 0).all()) and bool((buf[:, vocab + 1:] == 0).all())
    assert tsl.tsenor_error_count() == 1
