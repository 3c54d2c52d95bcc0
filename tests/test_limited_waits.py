"""The limited waits of the products and the distillation kernels, and where lanes of a warp meet, read from their sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_mask_search_b200", "csrc")


def _source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def _kernels(name):
    """{kernel: body} of a source."""
    text, found = _source(name), {}
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\(", text):
        depth, at = 0, text.index("{", m.end())
        for i in range(at, len(text)):
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            if depth == 0:
                break
        found[m.group(1)] = text[at:i + 1]
    return found


@pytest.mark.parametrize("name,count", [("quantize.cu", 2), ("matmul.cu", 2), ("distill.cu", 3)])
def test_no_limit_counts_the_time_of_the_kernel_before(name, count):
    # a thread waits for the kernel before without a limit first: in one place for all, or warp 1 in its own branch
    limited = re.compile(r"\b(\w+_bounded|warp_wait\w*|wait_long)\(")
    kernels = _kernels(name)
    assert len(kernels) == count
    for body in kernels.values():
        waits = [m.group(1).strip() for m in re.finditer(r"([^;{}]*)\bprior_done\(\);", body)]
        first = limited.search(body)
        assert first is None or body.index("prior_done();") < first.start()
        if waits != [""]:
            assert waits == ["if (warp != 1)", ""]
            branch = body[re.search(r"else if \(warp == 1\b", body).start():]
            assert branch.index("prior_done();") < limited.search(branch).start()


def test_a_warp_has_one_verdict():
    # lanes that went on after a wait that other lanes gave up would meet aligned instructions without them
    for name in ("matmul.cu", "distill.cu"):
        assert not re.search(r"\bmbar_\w*(bounded|wait|sleep)\b", _source(name))
    text = _source("tensor.h")
    assert len(re.findall(r"\bmbar_try_wait\(|mbarrier\.try_wait", text)) == 3
    functions = [m.start() for m in re.finditer(r"\bbool warp_\w+\(", text)]
    assert len(functions) == 4
    for start in functions:
        body = text[text.index("{", start):]
        body = body[:re.search(r";\s*}\s", body).end()]
        assert re.search(r"return (__all_sync\(0xffffffffu, done\)|warp_wait\([^;]*\));\s*}\s$", body), body


@pytest.mark.parametrize("name", ["matmul.cu", "distill.cu"])
def test_giving_up_is_counted(name):
    # by lane 0, for its warp
    for kernel, body in _kernels(name).items():
        if re.search(r"\bwarp_(wait|sleep|cluster_sleep)\(|\bwait_long\(", body):
            assert re.search(r"if \(stalled && lane == 0\) atomicAdd\(&g_\w+, 1ull\);\s*__syncwarp\(\);", body), kernel


def test_lanes_meet_before_tensor_memory_is_read():
    # the stores between two reads go by lane, some of which may have none
    text = _source("tensor.h")
    reads = [m.start() for m in re.finditer(r"tcgen05\.(ld|wait::ld)", text)]
    assert len(reads) == 2
    for at in reads:
        start = text.rindex("__device__", 0, at)
        assert re.search(r"{\s*__syncwarp\(\);\s*asm volatile\($", text[start:text.rindex("asm volatile(", 0, at) + 13])
