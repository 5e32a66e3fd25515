"""Where the kernels of csrc/mxfp4.hip and csrc/layer_norm.hip pass data through
LDS and wait for it themselves, the source states the order between accesses,
waits and barriers: the wait builtins count as touching no memory, the compiler
knows nothing of the other lanes, and no result shows an order that it
happened to keep."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "blockwise_bit_codebook_amd", "csrc")
FENCE = '__builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");'


def body(file, name):
    """A function's text, from its name to the closing brace in column 0."""
    source = open(os.path.join(CSRC, file)).read()
    at = re.search(rf"\b{name}\([^;{{]*\)\s*{{", source).start()
    return source[at:source.index("\n}\n", at)]


def statements(text):
    """Those of a function, without comments."""
    lines = (line.split("//")[0].strip() for line in text[text.index("{") + 1:].splitlines())
    return [line for line in lines if line]


def test_a_barrier_that_leaves_loads_in_flight():
    # accesses before it are done: fence, wait, barrier; those after it come after the second fence
    assert statements(body("matrix.h", "barrier_in_flight")) == [
        FENCE, "__builtin_amdgcn_s_waitcnt(0xC07F);", "__builtin_amdgcn_s_barrier();", FENCE]
