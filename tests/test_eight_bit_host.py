"""The 8-bit and distillation entry points reject bad arguments on the host,
before any CUDA call (no compute is run here)."""
import os
import re

import pytest
import torch

import sparse_mask_search_b200 as tsl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 12                     # an aligned address that is never read: every call here returns before a launch
ARG, SHAPE = -1, -2


def test_limits_of_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "tsenor.h")).read()
    for name, value in (("TOP", tsl.DISTILL_MAX_TOP), ("VOCAB", tsl.DISTILL_MAX_VOCAB)):
        assert int(re.search(rf"#define TSENOR_DISTILL_MAX_{name} (\d+)", text).group(1)) == value
    for prefix, names in (("BLOCK_", tsl.BLOCKS), ("", tsl.FORMS)):
        for key, value in names.items():
            assert re.search(rf"TSENOR_{prefix}{key.upper()} = {value}\b", text), key


@pytest.mark.parametrize("rows,cols", [(0, 5), (5, 0), (1, 1), (128, 512), (129, 513), (4096, 11008)])
def test_scale_bytes(rows, cols):
    a, b, c = tsl.scale_shape(rows, cols)
    want = a * b * c if rows and cols else 0
    assert tsl.lib().tsenor_scale_bytes(rows, cols) == want


def _quantize(**kw):
    a = dict(x=P, dtype=1, rows=8, cols=40, ldx=40, block=2, mask=None, values=P, ldv=48, scales=P, scales_t=P)
    a.update(kw)
    return tsl.lib().tsenor_quantize(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), ARG), (dict(block=3), ARG), (dict(block=-1), ARG), (dict(x=None), ARG), (dict(x=P + 1), ARG),
    (dict(dtype=0, x=P + 2), ARG), (dict(ldx=39), ARG), (dict(values=None), ARG), (dict(values=P + 8), ARG),
    (dict(ldv=40), ARG), (dict(ldv=32), ARG), (dict(mask=P + 2), ARG), (dict(scales=None), ARG),
    (dict(scales_t=None), ARG), (dict(block=0, scales=None), ARG), (dict(block=1, scales_t=None), ARG),
    (dict(scales=P + 4), ARG), (dict(rows=-1), SHAPE), (dict(cols=1 << 31), SHAPE),
    (dict(rows=0, x=None), 0), (dict(cols=0, values=None), 0),
])
def test_quantize_refusals(kw, code):
    assert _quantize(**kw) == code


def _pair(**kw):
    a = dict(x=P, dtype=1, rows=8, cols=40, ldx=40, values=P, ldv=48, scales=P, values_t=2 * P, ldv_t=48, scales_t=P)
    a.update(kw)
    return tsl.lib().tsenor_quantize_pair(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(values_t=P), ARG), (dict(values_t=None), ARG), (dict(ldv_t=40), ARG), (dict(scales=None), ARG),
    (dict(scales_t=None), ARG), (dict(x=None), ARG), (dict(dtype=9), ARG), (dict(rows=1 << 31), SHAPE), (dict(rows=0), 0),
])
def test_quantize_pair_refusals(kw, code):
    assert _pair(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(values=None), ARG), (dict(ldv=39), ARG), (dict(scales=None), ARG), (dict(out=None), ARG), (dict(ldo=39), ARG),
    (dict(dtype=5), ARG), (dict(out=P + 1), ARG), (dict(rows=-1), SHAPE), (dict(rows=0), 0),
])
def test_dequantize_refusals(kw, code):
    a = dict(values=P, rows=8, cols=40, ldv=40, scales=P, along=0, out=P, dtype=1, ldo=40)
    a.update(kw)
    assert tsl.lib().tsenor_dequantize(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(form=3), ARG), (dict(form=-1), ARG), (dict(dtype=2), ARG), (dict(a=None), ARG), (dict(a=P + 8), ARG),
    (dict(lda=40), ARG), (dict(lda=32), ARG), (dict(b=None), ARG), (dict(ldb=72), ARG), (dict(ldb=32), ARG),
    (dict(form=1, ldb=16), ARG), (dict(form=2, lda=0), ARG), (dict(sa=None), ARG), (dict(sb=P + 8), ARG),
    (dict(out=None), ARG), (dict(out=P + 1), ARG), (dict(ldo=23), ARG), (dict(mask=P + 1), ARG),
    (dict(m=-1), SHAPE), (dict(n=1 << 31), SHAPE), (dict(k=-5), SHAPE), (dict(m=0, a=None, out=None), 0), (dict(n=0), 0),
])
def test_matmul_refusals(kw, code):
    a = dict(form=0, a=P, lda=48, sa=P, b=P, ldb=48, sb=P, m=8, n=24, k=40, mask=None, out=P, dtype=1, ldo=24)
    a.update(kw)
    assert tsl.lib().tsenor_matmul(*a.values(), None) == code


BAD_DISTILL = [
    (dict(logits=None), ARG), (dict(logits=P + 1), ARG), (dict(dtype=3), ARG), (dict(ld=99), ARG), (dict(index=None), ARG),
    (dict(top_logits=None), ARG), (dict(index=P + 2), ARG), (dict(teacher_lse=P + 2), ARG), (dict(temperature=0.0), ARG),
    (dict(temperature=-1.0), ARG), (dict(temperature=float("nan")), ARG), (dict(temperature=float("inf")), ARG),
    (dict(rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=262145, ld=262145), SHAPE), (dict(top=-1), SHAPE),
    (dict(top=1025), SHAPE), (dict(rows=0, logits=None), 0),
]


def _shared(**kw):
    a = dict(logits=P, dtype=1, rows=4, vocab=100, ld=100, index=P, top_logits=P, top=3, teacher_lse=None,
             temperature=1.0)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,code", BAD_DISTILL + [(dict(loss=None), ARG), (dict(lse=None), ARG), (dict(loss=P + 2), ARG)])
def test_distill_loss_refusals(kw, code):
    a = _shared() | dict(loss=P, lse=P) | kw
    assert tsl.lib().tsenor_distill_loss(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", BAD_DISTILL + [
    (dict(loss=None), ARG), (dict(grad=None), ARG), (dict(grad=P + 1), ARG), (dict(ldg=99), ARG), (dict(weight=P + 2), ARG),
    (dict(grad=P, ldg=104), ARG)])
def test_distill_step_refusals(kw, code):
    a = _shared() | dict(weight=None, loss=P, grad=2 * P, ldg=100) | kw
    assert tsl.lib().tsenor_distill_step(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", BAD_DISTILL + [(dict(lse=None), ARG), (dict(grad=None), ARG), (dict(ldg=1), ARG)])
def test_distill_grad_refusals(kw, code):
    a = _shared() | dict(lse=P, weight=None, grad=2 * P, ldg=100) | kw
    assert tsl.lib().tsenor_distill_grad(*a.values(), None) == code


def test_binding_refuses_cpu_tensors_and_unknown_names():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        tsl.tsenor_quantize(x)
    with pytest.raises(ValueError):
        tsl.tsenor_quantize_pair(x)
    q = tsl.QuantizedMatrix(torch.zeros(4, 16, dtype=torch.uint8).view(torch.float8_e4m3fn))
    with pytest.raises(ValueError):
        tsl.tsenor_matmul(q, q, "tt")
    with pytest.raises(ValueError):
        tsl.tsenor_matmul(q, q, "nt")
    with pytest.raises(ValueError):
        tsl.tsenor_dequantize(q)
    i, t = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        tsl.tsenor_distill_loss(x, i, t)
    with pytest.raises(ValueError):
        tsl.tsenor_distill_step(x, i, t)
    with pytest.raises(ValueError):
        tsl.tsenor_distill_grad(x, i, t, torch.zeros(4))
