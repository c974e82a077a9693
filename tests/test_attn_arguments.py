"""Arguments of the attention entry points at the ends of their ranges, on the CPU: every call here ends before any
HIP call."""
import ctypes
import os

import pytest

import gated_delta_rule_08_amd as gdr

OK, NULL, SHAPE = 0, -1, -2
BIG = 2 ** 31 - 1
P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(8)]  # fake, aligned addresses


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdr.library_path()):
        from gated_delta_rule_08_amd import build
        build.build()
    return gdr.load_library()


def test_a_loose_bound_of_the_queries_is_no_error(lib):
    """max_q is any upper bound: what it says beyond total_q sizes nothing."""
    def call(mq, tq=8, q=None, N=2):
        return lib.gdr_attn_prefill_varlen(1, N, tq, 8, mq, 32, 8, 64, 0, 0, 1.0, q, *P[1:7], None)

    for mq in (8, 9, 1 << 24, 1 << 29, BIG):
        assert call(mq) == NULL, mq  # past the sizes, at the missing q
        assert call(mq, tq=0) == OK, mq
    assert call(-1) == SHAPE and call(BIG, tq=BIG) == SHAPE
