"""Several host threads in the 8-bit and distillation calls."""
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
