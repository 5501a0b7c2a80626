"""What the kernels' sources promise and a run may not show."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_sparse_attention_02_b200", "csrc")


def kernels(path):
    """(name, parameters, body) of each kernel of a source file."""
    src = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^)]*\)\s+)?(\w+)\s*\(", src):
        at, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(src[at], 0)
            at += 1
        params, body, depth = src[m.end():at - 1], src.index("{", at), 1
        end = body + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
        yield m.group(1), params, src[body:end]


@pytest.mark.parametrize("name", sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu"))))
def test_inputs_that_the_kernel_before_may_write_are_not_restrict(name):
    """A kernel that starts while the one before still runs must not promise the compiler that
    its inputs stay unchanged for as long as it runs."""
    waits = 0
    for kernel, params, body in kernels(os.path.join(CSRC, name)):
        if "griddep_wait" not in body:
            continue
        waits += 1
        for p in params.split(","):
            assert not ("const" in p and "__restrict__" in p), f"{kernel}: {p.strip()}"
    assert waits or name not in ("rope.cu", "paged.cu", "prefix.cu", "attn.cu", "topk.cu")


def test_pages_of_a_prefix_are_looked_up_for_a_sequence_that_holds_it():
    """tsa.h: table entries past a sequence's rows are not read.  The prefix pass reads entries of the
    first sequence (a.table) under a test of its length, all others through `table`, the row of a
    sequence that holds the prefix whole."""
    (_, _, body), = kernels(os.path.join(CSRC, "prefix.cu"))
    reads = [line for line in body.splitlines() if re.search(r"a\.table\[", line)]
    assert reads and all("a.lens[0] >= a.prefix_len" in line for line in reads)
    assert body.index("src < 0") < body.index("const int32_t* table = a.table") < body.index("= table[")
