"""The distillation loss and its gradient against their formulas in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_mask_search_b200 as tsl  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _case(rows, vocab, top, dtype, seed, scale=3.0):
    g = _gen(seed)
    z = torch.randn((rows, vocab), generator=g, device="cuda") * scale
    teacher = 0.7 * z + torch.randn((rows, vocab), generator=g, device="cuda") * scale * 0.7
    value, index = teacher.topk(min(top, vocab), 1)
    return z.to(TYPES[dtype]), index.to(torch.int32), value.contiguous(), teacher


def _reference(z, index, top_logits, temp, whole, weight):
    """(loss, lse, grad) in fp64 and how far a fp32 evaluation may be from loss and grad."""
    z, vocab, top = z.double(), z.shape[1], index.shape[1]
    valid = index >= 0
    i = index.long().clamp(min=0)
    t = torch.where(valid, top_logits.double() / temp, -torch.inf)
    none = (t == -torch.inf).all(1, keepdim=True)
    c = whole.double()[:, None] if whole is not None else torch.where(none, 0.0, torch.logsumexp(t, 1, keepdim=True))
    p = torch.where(none, 0.0, (t - c).exp())
    s = z / temp
    lse = torch.logsumexp(s, 1, keepdim=True)
    logp, logq = torch.where(p > 0, t - c, 0.0), torch.where(p > 0, s.gather(1, i) - lse, 0.0)
    loss = temp ** 2 * (p * (logp - logq)).sum(1)
    loss = torch.where(none[:, 0], 0.0, loss)
    w = temp * (weight.double()[:, None] if weight is not None else torch.ones_like(lse))
    total = p.sum(1, keepdim=True)
    q = (s - lse).exp()
    target = torch.zeros_like(s).scatter_add(1, i, p)
    grad = torch.where(none, 0.0, w * (total * q - target))
    # fp32: s, lse, t and c are each off by a few 2^-24 of their size, the sum of the exponentials by the
    # additions of one thread's share (vocab / 256 at most) and the tree, exp by a few steps
    big = torch.where(s.isfinite(), s.abs(), 0.0).amax(1, keepdim=True)
    tbig = torch.where(t.isfinite(), t.abs(), 0.0).amax(1, keepdim=True) + c.abs()
    rq, rp = 2.0 ** -24 * (8 * big + vocab / 256 + 128), 2.0 ** -24 * (8 * tbig + top + 64)
    terms = torch.where(p > 0, p * (logp - logq).abs(), 0.0).sum(1, keepdim=True)
    tol_loss = temp ** 2 * (total * (rq + rp) + terms * (rp + 2.0 ** -24 * top))[:, 0]
    tol_grad = w.abs() * (total * q * (rq + rp) + target * rp)
    return loss, lse[:, 0], grad, tol_loss, tol_grad


def _near(got, want, tol):
    fine = want.isfinite()
    assert torch.equal(got.isfinite(), fine)
    assert bool(((got.double() - want).abs()[fine] <= tol[fine]).all())


def _check(z, index, top_logits, temp=1.0, whole=None, weight=None):
    loss, lse, grad, tol_loss, tol_grad = _reference(z, index, top_logits, temp, whole, weight)
    got, got_lse = tsl.tsenor_distill_loss(z, index, top_logits, temp, whole)
    _near(got, loss, tol_loss)
    _near(got_lse, lse, 2.0 ** -24 * (4 * lse.abs() + z.shape[1] / 256 + 128))
    # the gradient's type rounds by half a step, and its smallest normal's step below that
    half = torch.finfo(z.dtype).eps / 2
    tol_grad = tol_grad + half * grad.abs() + torch.finfo(z.dtype).tiny
    loss2, g2 = tsl.tsenor_distill_step(z, index, top_logits, temp, whole, weight)
    _near(loss2, loss, tol_loss)
    _near(g2, grad, tol_grad)
    g3 = tsl.tsenor_distill_grad(z, index, top_logits, got_lse, temp, whole, weight)
    _near(g3, grad, tol_grad)
    assert g2.dtype == g3.dtype == z.dtype
    again = tsl.tsenor_distill_step(z, index, top_logits, temp, whole, weight)
    assert torch.equal(again[0], loss2) and torch.equal(again[1], g2)
    return loss2, g2


SIZES = [(1, 1, 1), (1, 7, 3), (3, 33, 1), (5, 1000, 20), (7, 32000, 20), (33, 1001, 64), (2, 50021, 256), (9, 4096, 1024),
         (1, 131072, 50), (2, 262144, 64), (300, 257, 8), (600, 2049, 16)]


@pytest.mark.parametrize("rows,vocab,top", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("temp", [1.0, 3.0])
@pytest.mark.parametrize("whole", [False, True])
def test_loss_and_gradient(rows, vocab, top, dtype, temp, whole):
    z, index, value, teacher = _case(rows, vocab, top, dtype, rows + vocab)
    lse = torch.logsumexp(teacher / temp, 1) if whole else None
    weight = torch.rand((rows,), generator=_gen(1), device="cuda")
    _check(z, index, value, temp, lse, weight)
    assert tsl.tsenor_error_count() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [130, 4001, 70000])
def test_rows_with_missing_entries(dtype, vocab):
    z, index, value, _ = _case(6, vocab, 12, dtype, 2)
    index[0] = -1                                # no entry at all: a prompt token
    index[1, 5:] = -1
    index[2, ::2] = -7
    value[3, 2:] = -torch.inf                    # entries of weight 0
    value[4] = -torch.inf                        # no weight at all
    value[0], value[2, ::2] = torch.nan, torch.inf       # what a missing entry holds does not matter
    weight = torch.tensor([1.0, 0.5, 2.0, 1.0, 1.0, 0.0], device="cuda")
    clean = torch.where(index >= 0, value, 0.0)
    loss, grad = _check(z, index, value, 2.0, None, weight)
    loss2, grad2 = tsl.tsenor_distill_step(z, index, clean, 2.0, None, weight)
    assert torch.equal(loss, loss2) and torch.equal(grad, grad2)
    assert bool((grad[[0, 4, 5]] == 0).all()) and loss[0] == 0 and loss[4] == 0 and loss[5] != 0
    assert tsl.tsenor_error_count() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("top", [5, 300])
def test_the_same_index_more_than_once(dtype, top):
    z, index, value, _ = _case(4, 3000, top, dtype, 3)
    index[0] = index[0, 0]
    index[1, 1::2] = index[1, 0]
    index[2, -1] = index[2, 0]
    _check(z, index, value, 1.5)


@pytest.mark.parametrize("dtype", TYPES)
def test_columns_of_probability_zero(dtype):
    z, index, value, _ = _case(4, 1000, 6, dtype, 4)
    z[:, 900:] = -torch.inf                      # a padded vocabulary
    index = torch.where(index >= 900, index - 900, index).contiguous()
    z[1] = -torch.inf
    z[1, 17] = 2.0                               # one column with all of the mass
    index[1] = 17
    _check(z, index, value)
    index[2, 0] = 950                            # the teacher gives weight to a column the student cannot reach
    loss, grad = tsl.tsenor_distill_step(z, index, value)
    assert loss[2] == torch.inf and bool(grad.isfinite().all()) and bool(loss[[0, 1, 3]].isfinite().all())
    _, _, want, _, _ = _reference(z, index, value, 1.0, None, None)
    assert abs(grad[2, 950].double() - want[2, 950]) <= 2.0 ** -7 * abs(want[2, 950])
    assert tsl.tsenor_error_count() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [500, 40000])
def test_failing_rows_are_counted_and_alone(dtype, vocab):
    z, index, value, teacher = _case(9, vocab, 7, dtype, 5)
    whole = torch.logsumexp(teacher, 1)
    good = _check(z, index, value, 1.0, whole)
    z2, i2, v2, w2 = z.clone(), index.clone(), value.clone(), whole.clone()
    z2[1, vocab - 1] = torch.nan
    z2[2, 0] = torch.inf
    z2[3] = -torch.inf
    i2[4, 3] = vocab
    i2[5, 0] = 2 ** 31 - 1
    v2[6, 1] = torch.nan
    w2[7] = torch.inf
    z2[8], i2[8] = torch.nan, -1                 # a row without entries is not read: no failure
    tsl.tsenor_error_count()
    loss, grad = tsl.tsenor_distill_step(z2, i2, v2, teacher_lse=w2)
    assert tsl.tsenor_error_count() == 7
    assert bool(loss[1:8].isnan().all()) and bool((grad[1:] == 0).all()) and loss[8] == 0
    assert loss[0] == good[0][0] and torch.equal(grad[0], good[1][0])
    loss3, lse3 = tsl.tsenor_distill_loss(z2, i2, v2, teacher_lse=w2)
    assert tsl.tsenor_error_count() == 7
    assert bool(loss3[1:8].isnan().all()) and bool(lse3[1:8].isnan().all()) and loss3[8] == 0
    grad3 = tsl.tsenor_distill_grad(z2, i2, v2, lse3, teacher_lse=w2)
    assert bool((grad3[1:] == 0).all())
    assert tsl.tsenor_error_count() == 7


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(5, 1000), (5, 1003), (3, 40001), (200, 515)])
def test_strided_rows_and_the_gradient_in_place(dtype, rows, vocab):
    z, index, value, _ = _case(rows, vocab, 9, dtype, 6)
    for left, width in ((0, vocab), (8, vocab + 24), (3, vocab + 5)):
        buf = torch.full((rows + 2, width), 5.0, dtype=z.dtype, device="cuda")
        inner = buf[1:rows + 1, left:left + vocab]
        inner.copy_(z)
        rest = torch.ones_like(buf, dtype=torch.bool)
        rest[1:rows + 1, left:left + vocab] = False
        loss, grad = _check(inner, index, value, 2.0)
        assert torch.equal(inner, z)
        _, lse = tsl.tsenor_distill_loss(inner, index, value, 2.0)
        grad2 = tsl.tsenor_distill_grad(inner, index, value, lse, 2.0)
        loss3, out = tsl.tsenor_distill_step(inner, index, value, 2.0, grad=inner)
        assert out is inner and torch.equal(loss, loss3) and torch.equal(out, grad)
        assert bool((buf[rest] == 5.0).all())
        inner.copy_(z)
        assert torch.equal(grad2, tsl.tsenor_distill_grad(inner, index, value, lse, 2.0, grad=inner))
        assert bool((buf[rest] == 5.0).all())


@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 600, 33000), ("bf16", 450, 60001), ("f32", 120, 131072), ("f32", 150, 262143),
                                              ("f32", 147, 65003), ("bf16", 500, 110001), ("bf16", 700, 5003),
                                              ("f32", 900, 4099), ("bf16", 450, 5003), ("bf16", 147, 200001)])
@pytest.mark.parametrize("top", [9, 200])
def test_many_rows_of_every_kind(dtype, rows, vocab, top):
    # blocks that walk several rows: with and without entries, failing, without weight, in any order
    z, index, value, _ = _case(rows, vocab, top, dtype, 11)
    kind = torch.randint(0, 8, (rows,), generator=_gen(12), device="cuda")
    index[kind == 0] = -1
    weight = torch.rand((rows,), generator=_gen(13), device="cuda")
    weight[kind == 1] = 0.0
    index[kind == 2, top // 2:] = -1
    loss, lse, grad, tol_loss, tol_grad = _reference(z, index, value, 2.0, None, weight)
    bad = kind == 3
    index[bad, 0] = vocab
    z[bad & (torch.arange(rows, device="cuda") % 2 == 0), vocab // 2] = torch.nan
    tsl.tsenor_error_count()
    got, g = tsl.tsenor_distill_step(z, index, value, 2.0, weight=weight)
    assert tsl.tsenor_error_count() == int(bad.sum())
    assert bool(got[bad].isnan().all()) and bool((g[bad | (kind == 0) | (kind == 1)] == 0).all())
    _near(got[~bad], loss[~bad], tol_loss[~bad])
    tol_grad = tol_grad + torch.finfo(z.dtype).eps / 2 * grad.abs() + torch.finfo(z.dtype).tiny
    _near(g[~bad], grad[~bad], tol_grad[~bad])
    got2, lse2 = tsl.tsenor_distill_loss(z, index, value, 2.0)
    _near(got2[~bad], loss[~bad], tol_loss[~bad])
    _near(lse2[~bad], lse[~bad], 2.0 ** -24 * (4 * lse.abs() + vocab / 256 + 128)[~bad])
    inner = z.clone()
    got3, _ = tsl.tsenor_distill_step(inner, index, value, 2.0, weight=weight, grad=inner)
    assert torch.equal(inner, g) and torch.equal(got3[~bad], got[~bad])
    tsl.tsenor_error_count()


@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 500, 33000), ("bf16", 800, 5003), ("f32", 100, 131072)])
def test_captured_and_replayed(dtype, rows, vocab):
    first, second = (_case(rows, vocab, 20, dtype, s)[:3] for s in (14, 15))
    want = []
    for z, index, value in (first, second):
        loss, lse = tsl.tsenor_distill_loss(z, index, value, 2.0)
        want.append((loss, lse, *tsl.tsenor_distill_step(z, index, value, 2.0), tsl.tsenor_distill_grad(z, index, value, lse, 2.0)))
    held = [t.clone() for t in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, lse = tsl.tsenor_distill_loss(*held, 2.0)
        out = (loss, lse, *tsl.tsenor_distill_step(*held, 2.0), tsl.tsenor_distill_grad(*held, lse, 2.0))
    for case, w in ((second, want[1]), (first, want[0]), (second, want[1])):
        for h, t in zip(held, case):
            h.copy_(t)
        graph.replay()
        for a, b in zip(out, w):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    # loss in fp32 along a random direction: central differences of step h are off by h^2 / 6 times the third
    # derivative and by the loss's own error over h
    z, index, value, _ = _case(3, 50, 6, "f32", 7, scale=1.0)
    temp = 1.7
    d = torch.randn(z.shape, generator=_gen(8), device="cuda")
    _, grad = tsl.tsenor_distill_step(z, index, value, temp)
    h = 2.0 ** -6
    up, _ = tsl.tsenor_distill_loss(z + h * d, index, value, temp)
    down, _ = tsl.tsenor_distill_loss(z - h * d, index, value, temp)
    *_, tol, _ = _reference(z, index, value, temp, None, None)
    # the third derivative is T^2 / T^3 times a third central moment of d, at most (2 max |d|)^3
    third = temp ** 2 * 8 * (d.abs().amax(1).double() / temp) ** 3
    # z + h d is itself rounded: 2^-24 of its size, times the gradient
    moved = ((z.abs() + h * d.abs()) * 2.0 ** -24 * grad.abs()).sum(1).double()
    want = (grad.double() * d.double()).sum(1)
    got = (up.double() - down.double()) / (2 * h)
    assert bool(((got - want).abs() <= third * h * h / 6 + (tol + moved) / h + 2.0 ** -20).all())


@pytest.mark.parametrize("rows,vocab", [(18000, 131072), (500000, 5003)])
def test_offsets_past_32_bits(rows, vocab):
    z = torch.zeros((rows, vocab), dtype=torch.bfloat16, device="cuda")
    tail, index, value, _ = _case(200, vocab, 10, "bf16", 16)
    z[-200:] = tail
    i = torch.zeros((rows, 10), dtype=torch.int32, device="cuda")
    t = torch.zeros((rows, 10), device="cuda")
    i[-200:], t[-200:] = index, value
    loss, lse, grad, tol_loss, tol_grad = _reference(tail, index, value, 2.0, None, None)
    tol_grad = tol_grad + 2.0 ** -8 * grad.abs() + torch.finfo(z.dtype).tiny
    got, got_lse = tsl.tsenor_distill_loss(z, i, t, 2.0)
    _near(got[-200:], loss, tol_loss)
    _near(tsl.tsenor_distill_grad(z, i, t, got_lse, 2.0)[-200:], grad, tol_grad)
    got, g = tsl.tsenor_distill_step(z, i, t, 2.0, grad=z)
    _near(got[-200:], loss, tol_loss)
    _near(g[-200:], grad, tol_grad)
    assert tsl.tsenor_error_count() == 0


def test_no_rows_and_no_entries():
    z = torch.randn((4, 100), device="cuda")
    none = torch.zeros((4, 0), dtype=torch.int32, device="cuda"), torch.zeros((4, 0), device="cuda")
    loss, grad = tsl.tsenor_distill_step(z, *none)
    assert bool((loss == 0).all()) and bool((grad == 0).all())
    loss, grad = tsl.tsenor_distill_step(z[:0], none[0][:0], none[1][:0])
    assert loss.shape == (0,) and grad.shape == (0, 100)


def test_binding_refusals():
    z, index, value, _ = _case(4, 100, 3, "f32", 9)
    for call in (tsl.tsenor_distill_loss, tsl.tsenor_distill_step):
        with pytest.raises(TypeError):
            call(z.half(), index, value)
        with pytest.raises(TypeError):
            call(z, index.long(), value)
        with pytest.raises(TypeError):
            call(z, index, value.bfloat16())
        with pytest.raises(ValueError):
            call(z, index[:3], value)
        with pytest.raises(ValueError):
            call(z, index, value[:, :2])
        with pytest.raises(ValueError):
            call(z, index, value, teacher_lse=torch.zeros((5,), device="cuda"))
        with pytest.raises(tsl.TsenorError):
            call(z, index, value, temperature=0.0)
        with pytest.raises(ValueError):
            call(z, index.cpu(), value)
    with pytest.raises(ValueError):
        tsl.tsenor_distill_grad(z, index, value, torch.zeros((3,), device="cuda"))
    with pytest.raises(TypeError):
        tsl.tsenor_distill_step(z, index, value, grad=z.bfloat16())
    with pytest.raises(ValueError):
        tsl.tsenor_distill_step(z, index, value, grad=z[:3])
    with pytest.raises(ValueError):
        tsl.tsenor_distill_step(z, index, value, weight=torch.ones((3,), device="cuda"))
