"""Kernels that come while the work before them still runs (programmatic dependent launch), by their source: what
they may have read too early shows in no result for as long as it happens to be there already."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kda_delta_rule_token_gb300", "csrc")
# Memory that a call's arguments or its workspace name, read (or written) by an index, or a member array of one.
ACCESS = re.compile(r"\b(?:io|a|g|done|scores|group_of|group_len)(?:\.\w+)*\s*\[|->\w+\s*\[|atomic\w+\((?:&?io|&?a\.|err)")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, kernel):
    """What stands between the braces of a __global__ function."""
    at = re.search(r"__global__[^{;]*\b%s\s*\([^{;]*\{" % kernel, text).end()
    depth, end = 1, at
    while depth:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
    return text[at:end - 1]


def kernels(name):
    return re.findall(r"__global__[^{;]*?\b(kda_\w+)\s*\(", source(name))


FILES = ["beam_select.cu", "beam_reorder.cu", "attn_fork.cu", "attn_shared.cu"]


def test_there_are_such_kernels():
    assert sum(len(kernels(f)) for f in FILES) >= 9


@pytest.mark.parametrize("file,kernel", [(f, k) for f in FILES for k in kernels(f)])
def test_nothing_is_read_before_the_wait(file, kernel):
    before, wait, _ = body(source(file), kernel).partition("griddep_wait();")
    assert wait and not ACCESS.findall(before)


def test_no_loads_of_what_is_constant():
    """Loads that may come from a cache which is not kept in step want memory that no one writes while the kernel
    lives; what a kernel reads that comes early may be written until its wait is over."""
    for file in FILES + ["attn_prefill.cu", "attn_decode.cu", "attn_rows.cuh"]:
        assert not re.search(r"__ldg|\.nc\b", source(file)), file


def test_the_tensor_core_kernel_waits_before_it_reads_the_plan():
    """Its launch behind the few-row kernel does not bring it what the plan, two launches before, wrote."""
    text = body(source("attn_prefill.cu"), "kda_attn_prefill_kernel")
    shared = text[text.index("if (kShared) {"):]
    assert shared.index("griddep_wait();") < shared.index("group_start[")
    assert "a.io" not in text[:text.index("if (kShared) {")].replace("if (!kShared) joins(a.io.workspace)", "")
