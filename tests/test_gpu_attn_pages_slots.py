"""Slots of the page plan at the end of int32."""
import pytest
import torch

import gated_delta_rule_08_amd as gdr
from gpu_util import announce, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page", [1, 2, 64, 65536])
@pytest.mark.parametrize("add", [3, 5000])
def test_slots_beyond_int32(page, add):
    """A slot that an int does not hold is -1, in the plan's own launch (few tokens) and in the second."""
    announce("slots beyond int32 %d %d" % (page, add))
    last = (2 ** 31 - 1) // page  # the last page whose slots fit
    width = -(-(add + 2) // page) + 1
    free = [last, last + 1, 2 ** 31 - 1, last - 1, 0, 7]
    free = [min(x, 2 ** 31 - 1) for x in free] * (width + 1)
    lengths, want = [1, 0, 2], [add, 1, add]
    held = [min(last + 1, 2 ** 31 - 1), 0, last]
    table = [[h] + [-1] * (width - 1) for h in held]
    table_d, cu, slots = ints(table), ints([0] * 4), ints([-77] * (2 * add + 9))
    added, out, left = ints([0] * 3), ints([0] * 3), ints([0])
    gdr.gdr_attn_plan_pages(ints(lengths), ints(want), ints(free), ints([len(free)]), table_d, page, cu, added, out, left, slots)
    torch.cuda.synchronize()
    stack, expect = list(free), []
    for n in range(3):
        for p in range(lengths[n], lengths[n] + want[n]):
            if p % page == 0:
                table[n][p // page] = stack.pop()
            slot = table[n][p // page] * page + p % page
            expect.append(slot if 0 <= slot < 2 ** 31 else -1)
    assert added.tolist() == want and table_d.tolist() == table
    assert slots[:len(expect)].tolist() == expect and (slots[len(expect):] == -77).all()
    assert -1 in expect or page == 1
    assert max(expect) == 2 ** 31 - 1 or page != 1


def test_as_many_requests_as_an_int_holds():
    """2^31 - 2 of them: the rounds of 1024 end there.  (9 GB a tensor.)"""
    announce("plan of 2^31 - 2 requests")
    N = 2 ** 31 - 2
    lengths, add = (torch.zeros(N, dtype=torch.int32, device="cuda") for _ in range(2))
    at = [0, 1023, 1024, 2 ** 30, 2 ** 30 + 1, N - 1026, N - 1025, N - 2, N - 1]
    for i in at:
        add[i] = 1
    add[5], add[N - 5] = 2, 2  # outgrow their rows
    table = torch.full((N, 1), -5, dtype=torch.int32, device="cuda")
    cu = torch.full((N + 1,), -5, dtype=torch.int32, device="cuda")
    slots, left = ints([-77] * 6000), ints([0])
    gdr.gdr_attn_plan_pages(lengths, add, ints(list(range(100, 120))), ints([20]), table, 1, cu, add, lengths, left, slots)
    torch.cuda.synchronize()
    assert left.tolist() == [20 - len(at)] and int(cu[N]) == len(at) and int(cu[0]) == 0
    assert int((add != 0).sum()) == len(at) and int((lengths != 0).sum()) == len(at) and int((table != -5).sum()) == len(at)
    for x, i in enumerate(at):
        assert (int(cu[i]), int(cu[i + 1]), int(table[i, 0]), int(lengths[i]), int(add[i])) == (x, x + 1, 119 - x, 1, 1)
    assert slots[:len(at)].tolist() == [119 - x for x in range(len(at))] and (slots[len(at):] == -77).all()
