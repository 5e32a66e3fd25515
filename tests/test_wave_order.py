"""Where lanes of one wave exchange data through LDS without a barrier,
csrc/int8.hip states the order between the accesses: the compiler knows
nothing of the other lanes, and no result shows an order that it happened to
keep."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = open(os.path.join(ROOT, "blockwise_bit_codebook_amd", "csrc", "int8.hip")).read()


def body(name):
    """A function's text, from its name to the closing brace in column 0."""
    at = re.search(rf"\b{name}\([^;{{]*\)\s*{{", SOURCE).start()
    return SOURCE[at:SOURCE.index("\n}\n", at)]


def test_partial_steps_of_few_rows_and_tokens():
    for name, read in (("int8_few_rows_kernel", "read(e);"), ("int8_tokens_kernel", "read(e, steps);")):
        text = body(name)
        at = text.index(read)
        assert text[:at].rstrip().endswith("wave_order();"), name        # pieces stored, then read by other lanes
        sums = text.index("sum_place(l16, q, TN * q + j)")
        assert "wave_order();" in text[at:sums], name                     # operands read, then gone over by the sums


def test_tiles_leave_through_a_region_of_the_wave():
    text = body("store_tile")
    stored, read = text.index("= d;"), text.index("if (packed)")
    assert "wave_order();" in text[stored:read]
    assert re.search(r"if \(i0 \+ kPass < TM\) wave_order\(\);", text[read:])


def test_what_states_the_order():
    text = body("wave_order")
    assert '__builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront")' in text and "__builtin_amdgcn_wave_barrier()" in text
