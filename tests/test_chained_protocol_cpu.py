"""Order of a chained tensor-core kernel's set-up (no GPU).

A kernel launched with programmatic serialization may start while the kernel
ahead runs.  What follows for a kernel with bounded waits is checked on the
kernels' source:

  * every bounded wait begins after the wait for the kernel ahead, or its limit
    would count that kernel's time: a thread that all roles meet at the block's
    barrier has waited, or each role waits before its first bounded wait;
  * tensor memory is taken before the kernel behind may start: one that took some
    first and then waited for this kernel would wait for good.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp8_w8a8_quantized_b200", "csrc")
KERNELS = {"mxfp8_gemm.cu": "mxfp8_gemm_kernel", "mxfp4_skinny.cu": "mxfp4_skinny_kernel"}
TOKENS = {"grid_launch_dependents": "launch", "grid_wait_ahead": "wait", "tmem_alloc_pair": "alloc", "tmem_alloc": "alloc",
          "__syncthreads": "barrier", "wait_bounded": "bounded", "sk_wait": "bounded"}


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"/\*.*?\*/|//[^\n]*", "", text, flags=re.S)


def body(name):
    """The kernel's body, comments left out."""
    text = source(name)
    at = text.index("{", text.index(")", text.index(KERNELS[name] + "(")))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]


def tokens(code):
    return [TOKENS[m] for m in re.findall(r"\b(" + "|".join(sorted(TOKENS, key=len, reverse=True)) + r")\s*\(", code)]


@pytest.mark.parametrize("name", KERNELS)
def test_bounded_waits_begin_after_the_kernel_ahead(name):
    code = body(name)
    head, roles = re.split(r"__syncthreads\(\);", code, maxsplit=1)
    assert "bounded" not in tokens(head)
    if "wait" in tokens(head):
        return
    roles = re.split(r"\} else if \(warp == \w+\) \{|    \} else \{\n\s+const float alpha", roles)
    assert len(roles) == 4, "producer, MMA, scale copies, epilogue"
    for role in roles:
        t = tokens(role)
        assert "bounded" in t and "wait" in t[:t.index("bounded")], f"{name}: a role's waits start before the kernel ahead has ended"


@pytest.mark.parametrize("name", KERNELS)
def test_tensor_memory_is_taken_before_the_launch_behind(name):
    t = tokens(body(name))
    assert t.count("launch") == 1 and "launch" in t[:t.index("barrier")]
    assert "alloc" in t[:t.index("launch")], f"{name}: the kernel behind may take tensor memory first"
