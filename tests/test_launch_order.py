"""Kernels that may start while the kernel before them still runs (launched by launch_after in smla_host.cuh) wait for
its end before anything else that could touch memory.  Which write a read overtakes is up to the GPU's timing, so
the rule is held on the source (no GPU)."""
import glob
import os
import re

import bench
from sparse_mla_decode_fp8_b200 import build


def _sources():
    return {os.path.basename(f): bench._code_tokens(open(f, encoding="utf-8").read()) for f in glob.glob(os.path.join(build.CSRC, "*.cu"))}


def _body(code, kernel):
    """A kernel's body, from behind its opening brace."""
    m = re.search(r"__global__ void __launch_bounds__\([^)]*\) " + kernel + r"\(", code)
    assert m, kernel
    return code[code.index("{", m.end()) + 1:]


def test_kernels_that_start_early_wait_before_they_read():
    launched = {}
    for name, code in _sources().items():
        for kernel in re.findall(r"launch_after\((\w+),", code):
            launched[kernel] = code
    assert set(launched) == {"span_logits_kernel", "span_scores_kernel", "span_decode_kernel", "join_kernel"}
    for kernel, code in launched.items():
        body = _body(code, kernel)
        before = body[:body.index("wait_for_prior_kernel();")]
        # only shared arrays and numbers made of the thread's and the block's indices: no parameter is looked at
        for statement in filter(None, (s.strip() for s in before.split(";"))):
            assert re.match(r"(__shared__ [\w ]+ |const int )", statement), (kernel, statement)
            assert not re.search(r"\bp\b|->|\w\(", statement.split("=", 1)[-1] if "=" in statement else ""), (kernel, statement)


def test_the_next_kernel_is_let_start_only_behind_the_wait():
    # what the kernel after it may rely on: whatever ran before the first of the two is complete by then
    for code in _sources().values():
        for m in re.finditer(r"let_next_kernel_start\(\);", code):
            start = code.rindex("__global__", 0, m.start())
            assert "wait_for_prior_kernel();" in code[start:m.start()]
