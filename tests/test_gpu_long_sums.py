"""Products over many blocks, where every block has to count: sums that are exact, and sums whose error is bounded by
what the tensor cores cut, on operands that spread their magnitude over all blocks.  Each block of the contracted axis
has a power of two that cancels between the operands, so that a scale of another block shows."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_mask_search_b200 as tsl  # noqa: E402

# one share, several, tiles that a block walks, pairs; sums that end inside a block
SIZES = [(1, 300, 20000), (100, 200, 30000), (31, 4100, 2050), (300, 64, 4000), (130, 9100, 3333), (1000, 4100, 2000), (2300, 4100, 3300)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _integer(shape, low, high, seed):
    return torch.randint(low, high + 1, shape, generator=_gen(seed), device="cuda")


def _scales(e):
    """Scale bytes of exponents e (rows, blocks of 128) by the documented index."""
    rows, blocks = e.shape
    shape = tsl.scale_shape(rows, 128 * blocks)
    out = torch.full((shape[0] * shape[1] * 512,), 127, dtype=torch.uint8, device="cuda")
    r, b = torch.arange(rows, device="cuda")[:, None], torch.arange(blocks, device="cuda")[None, :]
    out[((b // 4) * shape[1] + r // 128) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = (e + 127).to(torch.uint8)
    return out.view(shape)


def _stored(x, e, along_rows):
    """x (rows, k) with a scale 2^e for each row and block of k, stored as it is or with k along the rows."""
    x = (x.t() if along_rows else x).float()
    rows, cols = x.shape
    codes = torch.zeros((rows, (cols + 15) // 16 * 16), device="cuda")
    codes[:, :cols] = x
    codes = codes.to(torch.float8_e4m3fn)[:, :cols]
    return tsl.QuantizedMatrix(codes, None, _scales(e)) if along_rows else tsl.QuantizedMatrix(codes, _scales(e))


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("form", tsl.FORMS)
def test_sums_of_whole_numbers_are_exact(form, m, n, k):
    # codes of -3 to 3: sums below 9 * 30000 < 2^19, whole, and every product above 2^-25 of them, so that nothing is cut
    blocks = (k + 127) // 128
    a, b = _integer((m, k), -3, 3, k), _integer((n, k), -3, 3, k + 1)
    shift, up, right = _integer((1, blocks), -20, 20, 1), _integer((m, 1), -10, 10, 2), _integer((n, 1), -10, 10, 3)
    qa, qb = _stored(a, shift + up, form == "tn"), _stored(b, right - shift, form != "nt")
    want = torch.ldexp(a.double() @ b.double().t(), up + right.t())
    assert torch.equal(tsl.tsenor_matmul(qa, qb, form, dtype=torch.float32).double(), want)
    assert torch.equal(tsl.tsenor_matmul(qa, qb, form), want.to(torch.bfloat16))     # rounded once


@pytest.mark.parametrize("m,n,k", [(100, 200, 30000), (300, 500, 5000), (2300, 4100, 3300)])
@pytest.mark.parametrize("form", tsl.FORMS)
def test_sums_are_off_by_what_is_cut(form, m, n, k):
    blocks = (k + 127) // 128
    factor = torch.exp2(_integer((blocks,), -20, 20, 4).float()).repeat_interleave(128)[:k]
    x = torch.randn((m, k), generator=_gen(5), device="cuda") * factor
    y = torch.randn((n, k), generator=_gen(6), device="cuda") / factor
    qa = tsl.tsenor_quantize(x.t().contiguous(), "column") if form == "tn" else tsl.tsenor_quantize(x)
    qb = tsl.tsenor_quantize(y, "row") if form == "nt" else tsl.tsenor_quantize(y.t().contiguous(), "column")
    va, vb = tsl.tsenor_dequantize(qa).double(), tsl.tsenor_dequantize(qb).double()
    va, vb = va.t() if form == "tn" else va, vb if form == "nt" else vb.t()
    # the largest running sum, at a block's end or within a block
    run, high, inner = (torch.zeros((m, n), dtype=torch.float64, device="cuda") for _ in range(3))
    for c in range(0, k, 128):
        p, q = va[:, c:c + 128], vb[:, c:c + 128]
        run += p @ q.t()
        high = torch.maximum(high, run.abs())
        inner = torch.maximum(inner, p.abs() @ q.abs().t())
    # a step adds 32 products to the sum, each of the 33 cut by less than 2^-25 of the largest, and its result by
    # 2^-23 (37 times 2^-25 in all, 64 should a step be two); then up to 8 shares
    tol = (k / 32 + 9) * 64 * 2.0 ** -25 * (high + inner)
    out = tsl.tsenor_matmul(qa, qb, form, dtype=torch.float32).double()
    assert bool(((out - run).abs() <= tol).all())
    assert float((out - run).norm()) <= float(tol.norm())
