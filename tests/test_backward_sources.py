"""Rules of the gradient kernels that no run can show to be broken, read from
their sources (CPU).

A kernel launched while the one before it ends must load what that one wrote
with ordinary loads, behind its wait: __ldg asks for memory that nobody writes
while the kernel runs, and may be moved above the wait.  It also waits on every
way out: what follows it on the stream starts when it is done, not when the one
before it is.
"""
import os
import re

import ssd_scan_gb300

CSRC = os.path.join(os.path.dirname(ssd_scan_gb300.__file__), "csrc")
FILES = ("scan_backward_tc.cu", "scan_backward_simt.cu", "grad_reduce.cu", "conv1d_backward.cu", "norm_backward.cu")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def _block(text, at):
    """The {..} that opens at or behind `at`."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError("unbalanced braces")


def _kernels():
    for name in FILES:
        code = _code(name)
        for m in re.finditer(r"__global__[^{;]*?(\w+_kernel)\(", code):
            yield name, m.group(1), _block(code, m.end())


def test_overlapped_kernels_use_no_read_only_loads():
    overlapped = [(n, k, body) for n, k, body in _kernels() if "griddep_wait()" in body]
    assert {k for _, k, _ in overlapped} == {"scan_bwd_states_tc_kernel", "scan_bwd_tc_kernel", "scan_bwd_carry_kernel",
                                             "scan_bwd_simt_kernel", "scan_bwd_join_kernel", "grad_reduce_kernel"}
    for name, kernel, body in overlapped:
        assert "__ldg" not in body and ".nc." not in body, (name, kernel)
    # the fp32 rows and states of the fp32-pipe kernels go through these
    code = _code("scan_backward_simt.cu")
    for m in re.finditer(r"float4 (?:load4|ld4)\(const float\*", code):
        assert "__ldg" not in _block(code, m.end())


def test_overlapped_kernels_wait_on_every_way_out():
    for name, kernel, body in _kernels():
        if "griddep_wait()" not in body:
            continue
        wait = body.index("griddep_wait()")
        if not re.search(r"\breturn\b", body[:wait]) and not re.search(r"\bif\b", body[:wait]):
            continue  # before anything else
        if kernel == "scan_bwd_tc_kernel":
            # the control warp's run over the heads waits before it reads the states;
            # one that ends before that does so after it
            fail = body.index("if (!ok)", body.index("ok = ctl_run();"))
            assert "griddep_wait()" in _block(body, fail)
        elif kernel == "scan_bwd_states_tc_kernel":
            # every warp that walks, before it waits for anything else
            walk = _block(body, body.index("else", body.index("drain(&s.full")))
            assert "griddep_wait()" in walk and "warp_wait" not in walk[:walk.index("griddep_wait()")]
        else:
            assert not re.search(r"\breturn\b", body[:wait]), (name, kernel)
