"""Programmatic dependent launch, checked on the sources: a kernel launched with
launch_ex may start while its predecessor drains, and lets its successor start
once it triggers."""
import os
import re

from quantized_state_space_mamba2_b200 import build as B


def read(name):
    with open(os.path.join(B.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


SOURCES = {n: read(n) for n in sorted(os.listdir(B.CSRC)) if n.endswith((".cu", ".cuh"))}


def body(kernel):
    """The text of a __global__ function's body."""
    for text in SOURCES.values():
        for m in re.finditer(r"__global__[^;{]*?\b" + kernel + r"\s*\(", text):
            at = text.index("{", m.end())
            depth, end = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            return text[at:end]
    raise AssertionError(f"{kernel}: no such kernel")


def launched():
    names = set()
    for text in SOURCES.values():
        names |= set(re.findall(r'launch_ex\(\s*"(k_\w+)"', text))
    return sorted(names)


def test_every_kernel_launched_early_waits():
    """A kernel without the wait would run beside its predecessor, and may end
    before it, so that the next kernel's wait does not cover that one either."""
    names = launched()
    assert len(names) >= 20 and "k_fp8_gemm_tc" in names
    assert [n for n in names if "pdl_wait()" not in body(n)] == []


def test_kernels_that_write_a_state_do_not_trigger():
    """k_scan_step loads its state before its wait, so whatever is launched behind
    a kernel that writes states must start after that kernel's end."""
    step = body("k_scan_step")
    assert step.index("a.state + headrow") < step.index("pdl_wait()")
    for name in ("k_scan_step", "k_scan_seq", "k_reorder_rows"):
        assert "pdl_trigger" not in body(name), name
