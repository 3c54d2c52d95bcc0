"""Host threads and streams of the 8-bit and distillation calls."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sparse_mask_search_b200 as tsl  # noqa: E402


@pytest.mark.parametrize("call", ["quantize", "matmul", "split", "mask", "plan"])
def test_the_first_call_of_a_host_thread(call):
    x = torch.randn((300, 1024), device="cuda")
    q, w, mask = tsl.tsenor_quantize(x), x[:256].contiguous(), torch.empty((256, 32), dtype=torch.int32, device="cuda")
    one, small, large = tsl.tsenor_quantize(x[:1]), torch.empty((1, 300), device="cuda"), torch.empty((300, 300), device="cuda")
    plan, codes = torch.empty_like(w), tsl.tsenor_quantize(x)
    run = {"quantize": lambda: tsl.tsenor_quantize(x, out=codes).values.float(),
           "matmul": lambda: tsl.tsenor_matmul(q, q, out=large), "split": lambda: tsl.tsenor_matmul(one, q, out=small),
           "mask": lambda: tsl.tsenor_mask(w, 16, 32, 20.0, 10, 1, out=mask),
           "plan": lambda: tsl.tsenor_plan(w, 16, 32, 20.0, 10, out=plan)}[call]
    want = run().clone()
    torch.cuda.synchronize()
    got, errors = [], []

    def first():
        try:
            got.append(run())
        except Exception as e:                          # reported below, in the main thread
            errors.append(e)

    thread = threading.Thread(target=first)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert torch.equal(got[0], want)


def _product(m):
    g = torch.Generator(device="cuda").manual_seed(m)
    a = tsl.tsenor_quantize(torch.randn((m, 2048), generator=g, device="cuda"))
    b = tsl.tsenor_quantize(torch.randn((256, 2048), generator=g, device="cuda"))
    out, stream = torch.empty((m, 256), device="cuda"), torch.cuda.Stream()
    args = (tsl.FORMS["nt"], a.values.data_ptr(), 2048, a.scales.data_ptr(), b.values.data_ptr(), 2048, b.scales.data_ptr(),
            m, 256, 2048, None, out.data_ptr(), tsl.TSENOR_F32, 256, stream.cuda_stream)
    return tsl.lib().tsenor_matmul, args, out, (a, b, stream)


def _step(rows, vocab, top):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    z = torch.randn((rows, vocab), generator=g, device="cuda")
    value, index = z.topk(top, 1)
    index, value, out = index.to(torch.int32), value.contiguous(), torch.empty_like(z)
    loss, stream = torch.empty((rows,), device="cuda"), torch.cuda.Stream()
    args = (z.data_ptr(), tsl.TSENOR_F32, rows, vocab, vocab, index.data_ptr(), value.data_ptr(), top, None, 2.0, None,
            loss.data_ptr(), out.data_ptr(), vocab, stream.cuda_stream)
    return tsl.lib().tsenor_distill_step, args, out, (z, index, value, loss, stream)


@pytest.mark.parametrize("make,sizes", [(_product, [(64,), (8,), (128,)]), (_step, [(2, 262144, 500), (3, 1000, 4)])],
                         ids=["products", "distillation"])
def test_calls_of_different_sizes_from_several_threads(make, sizes):
    # what a launch asks for (its shared memory) belongs to the launch, not to the kernel that the threads share
    jobs = [make(*s) for s in sizes]
    torch.cuda.synchronize()
    want = []
    for call, args, out, _ in jobs:
        assert call(*args) == 0
        torch.cuda.synchronize()
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    failed, gate = [0] * len(jobs), threading.Barrier(len(jobs))

    def run(k):
        call, args, *_ = jobs[k]
        gate.wait()
        for _ in range(20000):
            failed[k] += call(*args) != 0

    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(jobs)
    for (_, _, out, _), w in zip(jobs, want):
        assert torch.equal(out, w)
    assert tsl.tsenor_error_count() == 0


def test_failures_counted_on_one_stream_while_another_reads_the_count():
    # every failure is in one number, none is lost between a read and the reset
    rows, calls = 64, 1500
    z = torch.full((rows, 8), torch.nan, device="cuda")
    index, top = torch.zeros((rows, 1), dtype=torch.int32, device="cuda"), torch.zeros((rows, 1), device="cuda")
    W = torch.full((64, 64), torch.nan, device="cuda")
    tsl.tsenor_error_count()
    torch.cuda.synchronize()
    seen, stop, errors = [], threading.Event(), []

    def read():
        try:
            stream = torch.cuda.Stream()
            while not stop.is_set():
                seen.append(tsl.tsenor_error_count(stream))
        except Exception as e:                          # reported below, in the main thread
            errors.append(e)

    readers = [threading.Thread(target=read) for _ in range(2)]
    for t in readers:
        t.start()
    for _ in range(calls):
        tsl.tsenor_distill_loss(z, index, top)
    for _ in range(10):
        tsl.tsenor_mask(W, 16, 32, 20.0, 5, 1)
    torch.cuda.synchronize()
    stop.set()
    for t in readers:
        t.join()
    assert not errors, errors
    assert sum(seen) + tsl.tsenor_error_count() == rows * calls + 4 * 10
    assert tsl.tsenor_error_count() == 0


def test_stream_zero_is_the_default_stream():
    device = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.stream(torch.cuda.Stream()):
        with tsl._on(device, 0):
            assert torch.cuda.current_stream().cuda_stream == torch.cuda.default_stream().cuda_stream == 0
    x = torch.randn((300, 500), device="cuda")
    want = tsl.tsenor_quantize(x)
    out = tsl.QuantizedMatrix(torch.empty_strided((300, 500), (512, 1), dtype=torch.float8_e4m3fn, device="cuda"),
                              torch.zeros_like(want.scales))
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                       # the default stream is busy: the call waits its turn there
    x.neg_()
    tsl.tsenor_quantize(x, out=out, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out.values.float(), -want.values.float()) and torch.equal(out.scales, want.scales)


@pytest.mark.parametrize("make,size", [(_product, (64,)), (_product, (3000,)), (_step, (3, 1000, 4)), (_step, (2, 262144, 9))])
def test_the_first_call_of_a_host_thread_while_another_captures(make, size):
    call, args, out, _ = make(*size)
    torch.cuda.synchronize()
    assert call(*args) == 0
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    count, status, graph = torch.zeros((1,), device="cuda"), [], torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        count += 1
        thread = threading.Thread(target=lambda: status.append(call(*args)))
        thread.start()
        thread.join()
        count += 1
    graph.replay()
    torch.cuda.synchronize()
    assert status == [0] and float(count) == 2 and torch.equal(out, want)
