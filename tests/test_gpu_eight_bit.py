"""The 8-bit quantisers and products against their definitions in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_mask_search_b200 as tsl  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _x(rows, cols, dtype, seed, spread=True):
    x = torch.randn((rows, cols), generator=_gen(seed), device="cuda")
    if spread:
        x = x * torch.randn((cols,), generator=_gen(seed + 1), device="cuda").mul(3).exp()
        x = x * torch.randn((rows, 1), generator=_gen(seed + 2), device="cuda").mul(3).exp()
    return x.to(TYPES[dtype])


def _words(keep):
    """Mask words of truth values (rows, cols)."""
    rows, cols = keep.shape
    full = torch.zeros((rows, (cols + 31) // 32 * 32), dtype=torch.int64, device=keep.device)
    full[:, :cols] = keep
    return (full.view(rows, -1, 32) << torch.arange(32, device=keep.device)).sum(2).to(torch.int32)


def _block_of(n, size):
    return torch.arange(n, device="cuda") // size


def _reference(x, block, keep=None):
    """(values the codes stand for before scaling, exponent of each entry's block), fp64 and int."""
    x = x.double()
    if keep is not None:
        x = torch.where(keep, x, 0.0)
    rows, cols = x.shape
    h, w = {"row": (1, 128), "column": (128, 1), "tile": (128, 128)}[block]
    br, bc = _block_of(rows, h), _block_of(cols, w)
    finite = torch.where(x.isfinite(), x, 0.0).abs()
    part = torch.zeros((rows, (cols + w - 1) // w), dtype=torch.float64, device="cuda")
    part = part.scatter_reduce(1, bc.expand(rows, -1), finite, "amax")
    big = torch.zeros(((rows + h - 1) // h, part.shape[1]), dtype=torch.float64, device="cuda")
    big = big.scatter_reduce(0, br[:, None].expand(-1, part.shape[1]), part, "amax")
    f, e = torch.frexp(big)                      # big = f 2^e, 448 = 0.875 * 2^9
    e = torch.where(big > 0, (e - 9 + (f > 0.875).int()).clamp(min=-126), 0)
    e = e[br][:, bc]
    y = torch.ldexp(x, -e)
    step = torch.ldexp(torch.ones_like(y), (torch.frexp(torch.where(y.isfinite(), y, 0.0))[1] - 1).clamp(min=-6) - 3)
    q = torch.where(x.isfinite(), (y / step).round() * step, torch.nan)
    return q, e


def _bytes(s, rows, cols):
    """The scale byte of every row and block of 128 columns, read by the documented index; and the unused bytes."""
    r = torch.arange(rows, device="cuda")[:, None]
    c = torch.arange(0, cols, 128, device="cuda")[None, :]
    tiles = (rows + 127) // 128
    at = ((c // 512) * tiles + r // 128) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + (c // 128) % 4
    flat = s.reshape(-1)
    rest = torch.ones_like(flat, dtype=torch.bool)
    rest[at.reshape(-1)] = False
    return flat[at].int(), flat[rest]


def _check_quantized(q, x, block, keep=None):
    rows, cols = x.shape
    want, e = _reference(x, block, keep)
    got = q.values.double()
    assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(want, nan=1e9))
    if block != "column":
        b, rest = _bytes(q.scales, rows, cols)
        assert torch.equal(b - 127, e[:, ::128]) and bool((rest == 127).all())
    if block != "row":
        b, rest = _bytes(q.scales_t, cols, rows)
        assert torch.equal(b - 127, e[::128].t()) and bool((rest == 127).all())


SHAPES = [(1, 1), (1, 4096), (5, 7), (128, 128), (129, 513), (200, 1000), (77, 640), (640, 77), (1000, 136), (256, 2056)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", tsl.BLOCKS)
def test_quantize_is_the_definition_bit_for_bit(rows, cols, dtype, block):
    x = _x(rows, cols, dtype, rows * 7 + cols)
    _check_quantized(tsl.tsenor_quantize(x, block), x, block)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_pair_equals_the_two_calls(rows, cols, dtype):
    x = _x(rows, cols, dtype, rows + cols)
    q, t = tsl.tsenor_quantize_pair(x)
    _check_quantized(q, x, "row")
    _check_quantized(t, x, "column")
    assert q.scales_t is None and t.scales is None


@pytest.mark.parametrize("block", tsl.BLOCKS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (33, 95), (130, 300), (256, 512)])
def test_quantize_with_a_mask(block, rows, cols):
    x = _x(rows, cols, "bf16", 3)
    keep = torch.rand((rows, cols), generator=_gen(9), device="cuda") < 0.5
    if rows > 1:
        keep[1] = False                          # a row that keeps nothing
    keep[:, cols // 2] = False
    x[~keep] = float("nan")                      # what a masked entry holds does not matter
    x[(~keep) & (torch.rand((rows, cols), generator=_gen(10), device="cuda") < 0.5)] = float("inf")
    q = tsl.tsenor_quantize(x, block, mask=_words(keep))
    _check_quantized(q, x, block, keep)
    assert bool((q.values.float()[~keep] == 0).all())


@pytest.mark.parametrize("block", tsl.BLOCKS)
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_extreme_values(block, dtype):
    x = torch.zeros((256, 384), device="cuda", dtype=TYPES[dtype])
    x[0, 0], x[1, 1], x[2, 130], x[3, 131] = float("nan"), float("inf"), -float("inf"), 3.0e38
    x[130, 0], x[131, 1], x[132, 2] = 1e-38, 448.0, 449.0
    x[200, 300], x[201, 301] = 1e-40, -2e-45 if dtype == "f32" else -1e-40
    x[4, 260:] = 0.0                             # all-zero blocks keep scale 1
    q = tsl.tsenor_quantize(x, block)
    _check_quantized(q, x, block)


@pytest.mark.parametrize("block", tsl.BLOCKS)
@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_strided_and_unaligned_rows(block, dtype):
    big = _x(150, 700, dtype, 4)
    for x in (big[3:140, 5:400], big[:, 8:520], big[::2, 1:2], big[7:8, 3:300], big[:, 571:], big[1:, 442:699]):
        _check_quantized(tsl.tsenor_quantize(x, block), x, block)


def test_quantize_writes_nothing_outside_its_outputs():
    x = _x(37, 45, "bf16", 5)
    buf = torch.full((39, 96), 0x55, dtype=torch.uint8, device="cuda")
    values = buf[1:38].view(torch.float8_e4m3fn)[:, 16:61]
    scales = torch.zeros(tsl.scale_shape(37, 45), dtype=torch.uint8, device="cuda")
    out = tsl.QuantizedMatrix(values, scales)
    assert tsl.tsenor_quantize(x, "row", out=out) is out
    _check_quantized(out, x, "row")
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[1:38, 16:61] = False
    assert bool((buf[rest] == 0x55).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", tsl.BLOCKS)
def test_dequantize(block, dtype):
    x = _x(133, 271, "f32", 6, spread=False)
    q = tsl.tsenor_quantize(x, block)
    want, e = _reference(x, block)
    got = tsl.tsenor_dequantize(q, TYPES[dtype])
    assert torch.equal(got.double(), torch.ldexp(want, e))       # 4 significant bits: exact in both types
    # half a step of e4m3 (2^-4 relative), or of its smallest step 2^-9 below 2^-6
    off = (torch.ldexp(want, e) - x.double()).abs()
    assert bool((off <= torch.maximum(2.0 ** -4 * x.double().abs(), torch.ldexp(torch.full_like(off, 2.0 ** -10), e))).all())


# ---- products ---------------------------------------------------------------------------------

def _operands(form, m, n, k, seed, tile):
    sa, sb = {"nt": ((m, k), (n, k)), "nn": ((m, k), (k, n)), "tn": ((k, m), (k, n))}[form]
    xa, xb = _x(*sa, "f32", seed), _x(*sb, "bf16", seed + 50)
    a = tsl.tsenor_quantize(xa, "column" if form == "tn" else "row")
    b = tsl.tsenor_quantize(xb, "tile" if tile else "row" if form == "nt" else "column")
    return a, b


def _values(q, along_rows):
    rows, cols = q.shape
    if along_rows:
        b, _ = _bytes(q.scales_t, cols, rows)
        b = b.t().repeat_interleave(128, 0)[:rows]
    else:
        b, _ = _bytes(q.scales, rows, cols)
        b = b.repeat_interleave(128, 1)[:, :cols]
    return torch.ldexp(q.values.double(), b - 127)


def _product(a, b, form):
    """(product, sum of the magnitudes) in fp64."""
    va, vb = _values(a, form == "tn"), _values(b, form != "nt")
    va = va.t() if form == "tn" else va
    vb = vb.t() if form == "nt" else vb
    return va @ vb, va.abs() @ vb.abs()


def _check_product(out, want, size, k):
    # products of codes are exact; each of at most k fp32 additions is off by at most 2^-24 of the sum of
    # the magnitudes (64 more for the tensor cores' truncated ones), then the rounding to bf16 by 2^-8
    tol = (k + 64) * 2.0 ** -24 * size
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert bool(((out.double() - want).abs() <= tol).all())


SIZES = [(1, 1, 1), (1, 128, 128), (3, 5, 7), (64, 64, 512), (128, 128, 129), (130, 260, 520), (1, 1000, 640), (17, 96, 33),
         (257, 300, 1111), (700, 1100, 900), (512, 768, 1024), (31, 4100, 2050), (300, 64, 4000), (1, 300, 20000)]


# more tiles than SMs, so that a block walks several; more blocks of 128 than a ring holds
SIZES += [(64, 25000, 300), (2600, 3100, 520), (100, 200, 30000), (1000, 4100, 2000)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("form", tsl.FORMS)
@pytest.mark.parametrize("tile", [False, True])
def test_matmul(form, m, n, k, tile):
    a, b = _operands(form, m, n, k, m + n + k, tile)
    want, size = _product(a, b, form)
    for dtype in TYPES.values():
        out = tsl.tsenor_matmul(a, b, form, dtype=dtype)
        assert out.dtype == dtype and out.shape == (m, n) and out.is_contiguous()
        _check_product(out, want, size, k)
        assert torch.equal(out, tsl.tsenor_matmul(a, b, form, dtype=dtype))


@pytest.mark.parametrize("form", tsl.FORMS)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (33, 95, 200), (300, 515, 700), (520, 1000, 300)])
@pytest.mark.parametrize("dtype", TYPES)
def test_matmul_with_a_mask(form, m, n, k, dtype):
    a, b = _operands(form, m, n, k, 8, False)
    keep = torch.rand((m, n), generator=_gen(11), device="cuda") < 0.5
    if m > 1:
        keep[0] = False
    want, size = _product(a, b, form)
    out = tsl.tsenor_matmul(a, b, form, mask=_words(keep), dtype=TYPES[dtype])
    _check_product(out, torch.where(keep, want, 0.0), torch.where(keep, size, 0.0), k)


@pytest.mark.parametrize("form", tsl.FORMS)
@pytest.mark.parametrize("m,n,k", [(5, 70, 300), (270, 300, 400)])
@pytest.mark.parametrize("dtype", TYPES)
def test_matmul_writes_only_its_output(form, m, n, k, dtype):
    a, b = _operands(form, m, n, k, 12, False)
    want, size = _product(a, b, form)
    for left, width in ((16, n + 40), (3, n + 7)):           # aligned and unaligned rows
        buf = torch.full((m + 2, width), 7.0, dtype=TYPES[dtype], device="cuda")
        out = buf[1:m + 1, left:left + n]
        assert tsl.tsenor_matmul(a, b, form, out=out) is out
        _check_product(out, want, size, k)
        rest = torch.ones_like(buf, dtype=torch.bool)
        rest[1:m + 1, left:left + n] = False
        assert bool((buf[rest] == 7.0).all())


@pytest.mark.parametrize("m,n,k", [(40, 200, 700), (300, 400, 700)])
def test_matmul_nan_stays_in_its_row_and_column(m, n, k):
    xa, xb = _x(m, k, "f32", 1, False), _x(n, k, "f32", 2, False)
    xa[7, 600], xb[11, 3] = float("nan"), float("inf")
    a, b = tsl.tsenor_quantize(xa), tsl.tsenor_quantize(xb)
    out = tsl.tsenor_matmul(a, b)
    bad = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    bad[7], bad[:, 11] = True, True
    assert torch.equal(out.isnan(), bad)


@pytest.mark.parametrize("m,n", [(40, 200), (300, 400)])
def test_matmul_over_a_wide_range_of_scales(m, n):
    k = 640
    xa, xb = _x(m, k, "f32", 1, False), _x(n, k, "f32", 2, False)
    xa *= torch.exp2(torch.randint(-60, 60, (m, 1), generator=_gen(3), device="cuda").float())
    xb *= torch.exp2(torch.randint(-60, 60, (n, 1), generator=_gen(4), device="cuda").float())
    a, b = tsl.tsenor_quantize(xa), tsl.tsenor_quantize(xb)
    want, size = _product(a, b, "nt")
    _check_product(tsl.tsenor_matmul(a, b, dtype=torch.float32), want, size, k)


def test_matmul_operands_that_are_slices():
    x, w = _x(64, 512, "bf16", 1, False), _x(300, 512, "bf16", 2, False)
    q, v = tsl.tsenor_quantize(x), tsl.tsenor_quantize(w, "tile")
    wide = torch.zeros((300, 1024), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    wide[:, 256:768].view(torch.uint8).copy_(v.values.view(torch.uint8))
    other = tsl.QuantizedMatrix(wide[:, 256:768], v.scales, v.scales_t)
    assert torch.equal(tsl.tsenor_matmul(q, other), tsl.tsenor_matmul(q, v))


@pytest.mark.parametrize("form,sa,sb", [("nt", (5, 0), (7, 0)), ("nn", (5, 0), (0, 7)), ("tn", (0, 5), (0, 7))])
def test_matmul_of_an_empty_sum_is_zero(form, sa, sb):
    def empty(rows, cols):
        return tsl.tsenor_quantize(torch.zeros((rows, cols), device="cuda"), "tile")
    a, b = empty(*sa), empty(*sb)
    out = torch.full((5, 7), 3.0, device="cuda")
    tsl.tsenor_matmul(a, b, form, out=out)
    assert bool((out == 0).all())
    assert tsl.tsenor_matmul(empty(0, 9), empty(7, 9)).shape == (0, 7)


def test_offsets_past_32_bits():
    # 70001 x 33024 entries are 2.3e9: the last rows by the large calls and by themselves
    rows, cols = 70001, 33024
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-300:] = _x(300, cols, "bf16", 21, False)
    x[:-300] = 0.5
    q = tsl.tsenor_quantize(x)
    last = tsl.tsenor_quantize(x[-1:])
    assert torch.equal(q.values[-1:].view(torch.uint8), last.values.view(torch.uint8))
    assert torch.equal(_bytes(q.scales, rows, cols)[0][-1:], _bytes(last.scales, 1, cols)[0])
    _, t = tsl.tsenor_quantize_pair(x[:, :130])
    _check_quantized(t, x[:, :130], "column")
    del x
    w = tsl.tsenor_quantize(_x(130, cols, "f32", 22, False), "tile")
    want, size = _product(tsl.QuantizedMatrix(last.values, last.scales), w, "nt")
    _check_product(tsl.tsenor_matmul(q, w, dtype=torch.float32)[-1:], want, size, cols)
    # an output of 70001 x 33024
    a, b = tsl.tsenor_quantize(_x(rows, 130, "f32", 23, False)), tsl.tsenor_quantize(_x(cols, 130, "f32", 24, False))
    out = tsl.tsenor_matmul(a, b)
    va, vb = _values(a, False)[-2:], _values(b, False)
    _check_product(out[-2:], va @ vb.t(), va.abs() @ vb.abs().t(), 130)


def test_binding_refusals():
    x = _x(16, 64, "bf16", 1, False)
    q = tsl.tsenor_quantize(x)
    with pytest.raises(TypeError):
        tsl.tsenor_quantize(x.half())
    with pytest.raises(ValueError):
        tsl.tsenor_quantize(x.t())
    with pytest.raises(ValueError):
        tsl.tsenor_quantize(x, "tile", out=q)                           # no scales_t to write
    with pytest.raises(ValueError):
        tsl.tsenor_quantize(x, "row", mask=torch.zeros((16, 3), dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        tsl.tsenor_quantize(x, "row", mask=torch.zeros((16, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        tsl.tsenor_quantize(x[:1].expand(4, 64))
    with pytest.raises(ValueError):
        tsl.tsenor_matmul(q, tsl.tsenor_quantize(x[:, :32].contiguous()))
    with pytest.raises(ValueError):
        tsl.tsenor_matmul(q, q, "tn")                                   # no scales_t
    with pytest.raises(TypeError):
        tsl.tsenor_matmul(q, q, dtype=torch.float16)
    with pytest.raises(TypeError):
        tsl.tsenor_matmul(q, q, out=torch.zeros((16, 16), device="cuda"), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tsl.tsenor_matmul(q, q, out=torch.zeros((16, 17), device="cuda"))
    narrow = torch.zeros((16, 40), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):                                     # rows start off 16 bytes
        tsl.tsenor_matmul(tsl.QuantizedMatrix(narrow, torch.zeros((1, 1, 512), dtype=torch.uint8, device="cuda")), q)
    with pytest.raises(ValueError):
        tsl.tsenor_matmul(tsl.QuantizedMatrix(q.values, q.scales[:, :, :256]), q)
