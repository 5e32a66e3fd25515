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


def test_what_states_the_order_within_a_wave():
    assert statements(body("mxfp4.hip", "wave_order")) == [FENCE, "__builtin_amdgcn_wave_barrier();"]


def test_partial_steps_of_few_rows_and_tokens():
    for name, read in (("mx_few_rows_kernel", "read(e);"), ("mx_tokens_kernel", "read(e, steps);")):
        text = body("mxfp4.hip", name)
        at = text.index(read)
        assert text[:at].rstrip().endswith("wave_order();"), name         # pieces stored, then read by other lanes
        sums = text.index("sum_place(l16, q, TN * q + j)")
        assert "wave_order();" in text[at:sums], name                      # operands read, then gone over by the sums


def test_tiles_leave_through_a_region_of_the_wave():
    text = body("mxfp4.hip", "store_tile")
    stored, read = text.index("= d;"), text.index("if (packed)")
    assert "wave_order();" in text[stored:read]
    assert re.search(r"if \(i0 \+ kPass < TM\) wave_order\(\);", text[read:])


def test_the_ring_waits_before_its_barriers():
    # a step's operands have arrived, its predecessor's have been read: both before the next loads are issued
    text = body("mxfp4.hip", "mx_ring_kernel")
    waits = re.findall(r"landed<[^;]*>\(\);\s*(\w+)\(\);", text)
    assert waits == ["barrier_in_flight", "barrier_in_flight"]
    step = text[text.index("auto step ="):]
    assert step.index("landed<") < step.index("barrier_in_flight") < step.index("put_scales(") < step.index("fetch_one(n, f, now)")
