"""The new operators together, as a pruned layer is trained: mask, 8-bit copy of the
masked weights, forward product, distillation loss, input and weight gradients, and new
scores for the mask."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_mask_search_b200 as tsl  # noqa: E402

N, M, TAU, ITERS, SWEEPS = 16, 32, 20.0, 50, 2


def _setup(tokens, vocab, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dense = torch.randn((vocab, width), generator=g, device="cuda") * width ** -0.5
    x = torch.randn((tokens, width), generator=g, device="cuda")
    value, index = (x @ dense.t() * 3).topk(16, 1)
    index = index.to(torch.int32)
    index[: tokens // 8] = -1
    return dense.bfloat16(), x.bfloat16(), index, value.contiguous()


def _step(w, x, index, value, mask):
    """One training step of the layer: (loss, dx, dw, and the operands of the two gradient products)."""
    wq = tsl.tsenor_quantize(w, "tile", mask=mask)
    xq, xt = tsl.tsenor_quantize_pair(x)
    logits = tsl.tsenor_matmul(xq, wq, "nt", dtype=torch.float32)
    loss, dz = tsl.tsenor_distill_step(logits, index, value, 2.0, grad=logits)
    zq, zt = tsl.tsenor_quantize_pair(dz)
    dx = tsl.tsenor_matmul(zq, wq, "nn")
    dw = tsl.tsenor_matmul(zt, xt, "tn", mask=mask, dtype=torch.float32)
    return loss, dx, dw, zq.values.view(torch.uint8), zq.scales, zt.values.view(torch.uint8), zt.scales_t


def _bits(mask, cols):
    return ((mask[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).bool().flatten(1)[:, :cols]


def _near(got, a, b, k, keep=None):
    """got = a @ b, summed over k entries in fp32 (and rounded to its type)."""
    want, tol = a @ b, (k + 64) * 2.0 ** -24 * (a.abs() @ b.abs())
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    if keep is not None:
        want, tol = want * keep, tol * keep
    assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("tokens,vocab,width", [(200, 1024, 512), (77, 2048, 256), (1, 512, 128), (513, 640, 1024)])
def test_training_step(tokens, vocab, width):
    w, x, index, value = _setup(tokens, vocab, width, 1)
    mask = tsl.tsenor_mask(w, N, M, TAU, ITERS, SWEEPS)
    temp = 2.0
    loss, dx, dw, *z = _step(w, x, index, value, mask)
    zq = tsl.QuantizedMatrix(z[0].view(torch.float8_e4m3fn), z[1])
    zt = tsl.QuantizedMatrix(z[2].view(torch.float8_e4m3fn), None, z[3])
    keep = _bits(mask, width)
    # the same step in 64 bits from the values that the 8-bit operands stand for
    wv = tsl.tsenor_dequantize(tsl.tsenor_quantize(w, "tile", mask=mask)).double()
    assert bool((wv[~keep] == 0).all())
    xr = tsl.tsenor_dequantize(tsl.tsenor_quantize(x, "row")).double()
    xc = tsl.tsenor_dequantize(tsl.tsenor_quantize(x, "column")).double()
    logits = (xr @ wv.t()).requires_grad_()
    valid = index >= 0
    p = torch.softmax(torch.where(valid, value.double() / temp, -1e30), 1) * valid
    logq = torch.log_softmax(logits / temp, 1).gather(1, index.long().clamp(min=0))
    want = temp ** 2 * (p * (torch.where(p > 0, p, 1.0).log() - logq)).sum(1)
    want.sum().backward()
    # a logit is off by its fp32 sum; the loss moves by at most 2 T times that, besides its own
    # few hundred fp32 steps of T^2 and of itself
    off = (width + 64) * 2.0 ** -24 * (xr.abs() @ wv.abs().t()).amax(1)
    own = 512 * 2.0 ** -24
    assert bool(((loss.double() - want).abs() <= 2 * temp * off + own * (temp ** 2 + want.abs())).all())
    # the gradient T (q - p), then its rounding to e4m3: half a step, 2^-4 of it or 2^-10 of its scale
    q = torch.softmax(logits.detach() / temp, 1)
    target = torch.zeros_like(q).scatter_add(1, index.long().clamp(min=0), p)
    off = temp * (q + target) * (2 * off[:, None] / temp + own)
    ones = torch.full((tokens, vocab), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)   # code of 1
    for part in (zq, zt):
        scale = tsl.tsenor_dequantize(tsl.QuantizedMatrix(ones, part.scales, part.scales_t)).double()
        got = tsl.tsenor_dequantize(part).double()
        tol = off + torch.maximum(2.0 ** -4 * (logits.grad.abs() + off), 2.0 ** -10 * scale)
        assert bool(((got - logits.grad).abs() <= tol).all())
    # the gradient products of those operands
    _near(dx, tsl.tsenor_dequantize(zq).double(), wv, vocab)
    _near(dw, tsl.tsenor_dequantize(zt).double().t(), xc, tokens, keep)
    # gradient scores go back into the solver
    dense_dw = tsl.tsenor_matmul(*(q[1] for q in map(tsl.tsenor_quantize_pair, (logits.grad.float(), x))), "tn",
                                 dtype=torch.float32)
    scores = (w.float() * (w.float() - 0.1 * dense_dw)).abs()
    new = tsl.tsenor_mask_scores(scores, N, M, TAU, ITERS, SWEEPS)
    assert not bool(tsl.tsenor_objective(scores, new, N, M).isnan().any())
    assert tsl.tsenor_error_count() == 0


def test_step_captured_into_a_graph_and_replayed_on_new_inputs():
    first, second = _setup(130, 768, 384, 2), _setup(130, 768, 384, 3)
    mask = tsl.tsenor_mask(first[0], N, M, TAU, ITERS, SWEEPS)
    want = [[t.clone() for t in _step(*s, mask)] for s in (first, second)]
    held = [t.clone() for t in first]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(*held, mask)
    torch.cuda.current_stream().wait_stream(side)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(*held, mask)
    with torch.cuda.graph(other):                    # a second graph of the same calls
        out2 = _step(*held, mask)
    for s, w in ((first, want[0]), (second, want[1]), (first, want[0])):
        for h, t in zip(held, s):
            h.copy_(t)
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(out, out2, w):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_two_streams_at_once_and_a_given_stream():
    jobs = [_setup(300, 1024, 512, s) for s in (4, 5)]
    mask = tsl.tsenor_mask(jobs[0][0], N, M, TAU, ITERS, SWEEPS)
    want = [[t.clone() for t in _step(*j, mask)] for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(3):
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(_step(*j, mask))
    torch.cuda.synchronize()
    for k, out in enumerate(got):
        for a, b in zip(out, want[k % 2]):
            assert torch.equal(a, b)
    w, x, index, value = jobs[0]
    s = streams[0]
    xq = tsl.tsenor_quantize(x, stream=s)
    wq = tsl.tsenor_quantize(w, "tile", mask=mask, stream=s.cuda_stream)
    z = tsl.tsenor_matmul(xq, wq, dtype=torch.float32, stream=s)
    loss, _ = tsl.tsenor_distill_step(z, index, value, 2.0, stream=s)
    s.synchronize()
    assert torch.equal(loss, want[0][0])
