"""The limited waits of the products and the distillation kernels on the GPU."""
import ctypes as C
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_mask_search_b200 as tsl  # noqa: E402
from sparse_mask_search_b200 import build  # noqa: E402

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCES = ["matmul.cu", "distill.cu"]


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


# ---- waits that run out ---------------------------------------------------------------------------
#
# A build of the same sources in which a wait gives up as if its polls had run out: at random, one in so many.  Each
# kernel has to end by itself with its copies and products done, count that it gave up, and leave the GPU as it
# was: the calls right behind it are right.

NEVER = (1 << 18, 0)                                     # the library's own limit, and no wait that gives up


@pytest.fixture(scope="module")
def giving_up():
    lib = os.path.join(HERE, "_build", "libgive_up.so")
    sources = [os.path.join(build.HERE, "csrc", f) for f in SOURCES] + [os.path.join(HERE, "give_up.cu")]
    deps = build.sources() + [os.path.join(HERE, "give_up.cu")]
    if not os.path.exists(lib) or os.path.getmtime(lib) < max(os.path.getmtime(s) for s in deps):
        os.makedirs(os.path.dirname(lib), exist_ok=True)
        subprocess.run([build.nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "--threads", "0",
                        "-Xcompiler", "-fPIC", "-shared", "-DTSENOR_GIVE_UP", *sources, "-o", lib], check=True)
    L = C.CDLL(lib)
    ours = tsl.lib()
    for name in ("tsenor_matmul", "tsenor_distill_loss", "tsenor_distill_step"):
        getattr(L, name).argtypes = getattr(ours, name).argtypes
    L.give_up_products.argtypes = L.give_up_distillation.argtypes = [C.c_uint, C.c_uint]
    L.give_up_count.restype = C.c_longlong
    return L


# shares of a tile; one tile to a block; tiles that blocks walk, to rows off 32 bytes too; pairs with one tile, with several, to rows off 32 bytes
PRODUCTS = [("nt", 60, 256, 4096, 256), ("nt", 1, 11008, 4096, 11008), ("nn", 300, 9000, 1100, 9000), ("tn", 1500, 1300, 777, 1301),
            ("tn", 2048, 2900, 1100, 2901), ("nn", 512, 8000, 4096, 8000), ("nt", 2048, 4096, 2048, 4096), ("tn", 2300, 4100, 3300, 4101)]


@pytest.mark.parametrize("form,m,n,k,ldo", PRODUCTS)
@pytest.mark.parametrize("one_in", [1, 3, 20, 200, 3000])
def test_products_that_give_up(giving_up, form, m, n, k, ldo, one_in):
    sa, sb = {"nt": ((m, k), (n, k)), "nn": ((m, k), (k, n)), "tn": ((k, m), (k, n))}[form]
    g = torch.Generator(device="cuda").manual_seed(m + n)
    a = tsl.tsenor_quantize(torch.randn(sa, generator=g, device="cuda"), "tile")
    b = tsl.tsenor_quantize(torch.randn(sb, generator=g, device="cuda"), "tile")
    out = torch.zeros((m, ldo), dtype=torch.bfloat16, device="cuda")
    on_a, on_b = (a.scales_t if form == "tn" else a.scales), (b.scales if form == "nt" else b.scales_t)
    args = (tsl.FORMS[form], a.values.data_ptr(), a.values.stride(0), on_a.data_ptr(), b.values.data_ptr(), b.values.stride(0),
            on_b.data_ptr(), m, n, k, None, out.data_ptr(), tsl.TSENOR_BF16, ldo, torch.cuda.current_stream().cuda_stream)
    want = tsl.tsenor_matmul(a, b, form)
    assert giving_up.give_up_products(200, one_in) == 0 and giving_up.give_up_count() == 0
    gave_up = 0
    for _ in range(12):
        out.zero_()
        assert giving_up.tsenor_matmul(*args) == 0
        behind = tsl.tsenor_matmul(a, b, form)
        count = giving_up.give_up_count()
        assert count >= 0 and torch.equal(behind, want)
        if count == 0:
            assert torch.equal(out[:, :n], want)
        gave_up += count
    assert gave_up > 0 or one_in > 200
    for _ in range(12):                                  # without a pause in between
        assert giving_up.tsenor_matmul(*args) == 0
    behind = tsl.tsenor_matmul(a, b, form)
    assert giving_up.give_up_count() >= 0 and torch.equal(behind, want)
    assert giving_up.give_up_products(*NEVER) == 0
    assert giving_up.tsenor_matmul(*args) == 0
    assert giving_up.give_up_count() == 0 and torch.equal(out[:, :n], want)
    assert tsl.tsenor_error_count() == 0


# slices of a cluster, one row to it and several; rows of one CTA, one and several; fp32 rows of several segments
@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 3, 32000), ("bf16", 400, 131072), ("f32", 100, 40000), ("f32", 147, 3001),
                                              ("f32", 90, 262143), ("bf16", 1, 900)])
@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("one_in", [1, 3, 20, 200, 3000])
def test_distillation_that_gives_up(giving_up, dtype, rows, vocab, step, one_in):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z = torch.randn((rows, vocab), generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    value, index = z.float().topk(7, 1)
    index, value = index.to(torch.int32), value.contiguous()
    index[::5] = -1
    loss, lse, grad = torch.zeros((rows,), device="cuda"), torch.zeros((rows,), device="cuda"), torch.zeros_like(z)
    shared = (z.data_ptr(), int(dtype == "bf16"), rows, vocab, vocab, index.data_ptr(), value.data_ptr(), 7, None, 2.0)
    stream = torch.cuda.current_stream().cuda_stream
    if step:
        outs, ours = (loss, grad), lambda: tsl.tsenor_distill_step(z, index, value, 2.0)
        call = lambda: giving_up.tsenor_distill_step(*shared, None, loss.data_ptr(), grad.data_ptr(), vocab, stream)
    else:
        outs, ours = (loss, lse), lambda: tsl.tsenor_distill_loss(z, index, value, 2.0)
        call = lambda: giving_up.tsenor_distill_loss(*shared, loss.data_ptr(), lse.data_ptr(), stream)
    want = ours()
    same = lambda got: all(torch.equal(x, y) for x, y in zip(got, want))
    assert giving_up.give_up_distillation(200, one_in) == 0 and giving_up.give_up_count() == 0
    gave_up = 0
    for _ in range(8):
        for t in outs:
            t.zero_()
        assert call() == 0
        behind = ours()
        count = giving_up.give_up_count()
        assert count >= 0 and same(behind)
        if count == 0:
            assert same(outs)
        gave_up += count
    # (the loss of many rows and the step of short ones stream them and wait for nothing)
    assert gave_up > 0 or one_in > 3 or not step and rows >= 148
    for _ in range(8):                                   # without a pause in between
        assert call() == 0
    behind = ours()
    assert giving_up.give_up_count() >= 0 and same(behind)
    assert giving_up.give_up_distillation(*NEVER) == 0
    assert call() == 0
    assert giving_up.give_up_count() == 0 and same(outs)
    assert tsl.tsenor_error_count() == 0
