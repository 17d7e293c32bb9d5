"""Every kernel of the 8-bit cache's calls waits for the previous one of its stream before it touches memory: what an earlier kernel
wrote is promised to be visible behind a kernel's own wait only, whatever the kernel between them waited for.
(A missing wait is a race, so it is looked for in the sources and not on a GPU.)"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hybrid_head_sparse_decode_b200", "csrc")


def bodies():
    """(file, kernel, body) of the __global__ functions that those calls launch."""
    for path in sorted(glob.glob(os.path.join(CSRC, "q8_*.cu"))) + [os.path.join(CSRC, f) for f in ("topk.cu", "blocksel.cu")]:
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            head = text.index("{", m.end())
            depth, at = 1, head + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            # (the name: what the parameter list follows)
            name = [n for n in re.findall(r"(\w+)\s*\(", text[m.end():head]) if n != "__launch_bounds__"][0]
            yield os.path.basename(path), name, text[head:at]


KERNELS = [(f, n, b) for f, n, b in bodies() if "pdl_launch_dependents" in b]


def test_the_sources_were_read():
    names = {n for _, n, _ in KERNELS}
    assert {"q8_append_kernel", "q8_sets_kernel", "q8_attn_kernel", "q8_merge_kernel", "topk_combine_kernel"} <= names


@pytest.mark.parametrize("file,name,body", KERNELS, ids=[n for _, n, _ in KERNELS])
def test_the_wait_is_unconditional_and_comes_first(file, name, body):
    lines = [x.strip() for x in body.splitlines()]
    waits = [i for i, x in enumerate(lines) if "pdl_wait()" in x]
    assert waits and lines[waits[0]] == "pdl_wait();", "the first wait stands on its own"
    before = "\n".join(lines[:waits[0]])
    # nothing that memory of an earlier kernel holds is read or written before it
    assert not re.search(r"p\.\w+\[|\*\w*p\.\w+|flag_error", before), before
