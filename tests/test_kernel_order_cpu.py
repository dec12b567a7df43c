"""Orders inside the kernels that a run shows only when it hangs, read from their sources.

A kernel that lets its programmatic dependents launch before it holds its tensor memory can hang: a
dependent placed on the same SM may allocate the columns first and then wait for this grid, whose
allocation waits for the dependent's columns.  A shuffle that takes the lanes that happen to be active
for its own is undefined once they have diverged."""
from __future__ import annotations

import glob
import os
import re

import pytest

from int8_quantized_02_b200 import build as build_mod

RELEASE = re.compile(r"griddepcontrol\.launch_dependents|pdl_wait_then_release\(")


def functions(path):
    """(name, body) of each function of a source file, comments left out."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
    for m in re.finditer(r"(\w+)\s*\([^;{}()]*(?:\([^()]*\)[^;{}()]*)*\)\s*(?:const\s*)?\{", text):
        if m.group(1) in ("if", "for", "while", "switch"):
            continue
        depth, at = 1, m.end()
        while depth and at < len(text):
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), text[m.end():at]


KERNELS = [(os.path.basename(p), name, body) for p in sorted(glob.glob(os.path.join(build_mod.CSRC, "*.cu")))
           for name, body in functions(p) if re.search(r"\btmem_alloc(_pair)?\(", body)]


def test_every_kernel_with_tensor_memory_is_read():
    assert {k[1] for k in KERNELS} == {"gemm_body", "llmint8_decode_kernel", "mxfp4_pair_kernel",
                                       "mxfp4_band_kernel"}


@pytest.mark.parametrize("name,body", [k[1:] for k in KERNELS], ids=[k[1] for k in KERNELS])
def test_dependents_launch_after_the_allocation(name, body):
    if name == "llmint8_decode_kernel":       # the quantizer's CTAs allocate nothing and return
        body = body[body.index("quantize_x("):]
    alloc = max(m.start() for m in re.finditer(r"\btmem_alloc(_pair)?\(", body))
    for m in RELEASE.finditer(body):
        assert alloc < m.start(), "dependents may launch before the allocation"
        between = body[alloc:m.start()]       # the same block, or behind a barrier
        assert "}" not in between or "__syncthreads()" in between, \
            "another warp may let them launch before the allocating one is done"


def test_shuffles_name_their_lanes():
    for p in glob.glob(os.path.join(build_mod.CSRC, "*.cu*")):
        assert "__activemask" not in open(p).read(), os.path.basename(p)
