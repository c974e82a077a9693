"""The page plan of a serving step against a request-by-request walk on the host."""
import random

import pytest
import torch

import gated_delta_rule_08_amd as gdr
from gpu_util import announce, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def walk(lengths, add, free, n_free, table, page, max_tokens):
    """(table, cu, added, lengths_out, n_free_out, slots) of the definition."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    free = list(free[:max(0, min(n_free, len(free)))])
    cu, slots, added, serving = [0], [], [], True
    for n, (have, want) in enumerate(zip(lengths, add)):
        fine = have >= 0 and want >= 0 and have + want <= width * page
        need = -(-(have + want) // page) - -(-have // page) if fine else 0
        if fine and serving and (need > len(free) or len(slots) + want > max_tokens):
            serving = False
        got = want if fine and serving else 0
        for p in range(have, have + got):
            if p % page == 0:
                table[n][p // page] = free.pop()
            at = table[n][p // page]
            slots.append(at * page + p % page if at >= 0 else -1)
        added.append(got)
        cu.append(len(slots))
    return table, cu, added, [a + b for a, b in zip(lengths, added)], len(free), slots


def run(lengths, add, free, n_free, width, page, max_tokens=None, with_slots=True, in_place=False, table=None):
    N = len(lengths)
    if table is None:
        table = [[1000 * n + i if i * page < max(0, h) else -1 - i for i in range(width)] for n, h in enumerate(lengths)]
    ref = walk(lengths, add, free, n_free, table, page, 2 ** 31 - 1 if max_tokens is None else max_tokens)
    dev = lambda xs: torch.tensor(xs, dtype=torch.int32, device="cuda")  # noqa: E731
    t = dev(table).view(N, width)
    ld, ad, fd, nf = dev(lengths), dev(add), dev(free), dev([n_free])
    cu = torch.full((N + 1,), 77, dtype=torch.int32, device="cuda")
    lo, go, no = (ld, ad, nf) if in_place else (torch.full_like(ld, 77), torch.full_like(ad, 77), torch.full_like(nf, 77))
    slots = None
    if with_slots:
        slots = torch.full((len(ref[5]) + 5 if max_tokens is None else max_tokens,), -77, dtype=torch.int32, device="cuda")
    gdr.gdr_attn_plan_pages(ld, ad, fd, nf, t, page, cu, go, lo, no, slots, max_tokens=None if with_slots else max_tokens)
    torch.cuda.synchronize()
    assert cu.tolist() == ref[1] and go.tolist() == ref[2] and lo.tolist() == ref[3] and no.tolist() == [ref[4]]
    assert t.tolist() == ref[0]
    assert fd.tolist() == list(free)
    if with_slots:
        assert slots[:len(ref[5])].tolist() == ref[5] and (slots[len(ref[5]):] == -77).all()
    return ref


@pytest.mark.parametrize("page", [1, 2, 16, 64, 1024])
def test_random(page):
    announce("pages random %d" % page)
    r = random.Random(page)
    for case in range(12):
        N = r.choice([1, 2, 5, 63, 64, 65, 300])
        width = r.choice([1, 3, 17])
        lengths = [r.randint(0, width * page) for _ in range(N)]
        add = [min(r.choice([0, 1, 1, r.randint(0, 3 * page)]), width * page - n) for n in lengths]
        need = sum(-(-(n + a) // page) - -(-n // page) for n, a in zip(lengths, add))
        n_free = r.choice([need, need + 3, need // 2, 0])
        free = [10 ** 6 + 7 * i for i in range(n_free + r.randint(0, 4))]
        tokens = r.choice([None, None, sum(add), sum(add) // 2, 0])
        run(lengths, add, free, n_free, width, page, tokens, with_slots=r.random() < 0.7, in_place=r.random() < 0.5)


@pytest.mark.parametrize("N", [1023, 1024, 1025, 2500])
def test_many_requests(N):
    """More requests than one round of the sums takes; the stack ends in the first, a middle and the last round."""
    announce("pages many %d" % N)
    r = random.Random(N)
    lengths = [r.randint(0, 60) for _ in range(N)]
    add = [r.choice([1, 1, 1, 20, 0]) for _ in range(N)]
    need = sum(-(-(n + a) // 16) - -(-n // 16) for n, a in zip(lengths, add))
    for n_free in (need, need // 2, need - 1, 3):
        run(lengths, add, [5 * i for i in range(n_free)], n_free, 8, 16)
    run(lengths, add, [5 * i for i in range(need)], need, 8, 16, max_tokens=sum(add) // 3, in_place=True)


def test_bad_requests():
    """Negative lengths and additions, and rows outgrown, add nothing and hold no one up; a stack count out of range."""
    announce("pages bad requests")
    big = 2 ** 31 - 1
    lengths, add = [5, -1, 20, 64, big, 0, 63, 10], [3, 4, -1, 1, big, 65, 1, 2]
    for n_free in (-5, 0, 3, 9, 100, big, -2 ** 31):
        run(lengths, add, list(range(100, 109)), n_free, 4, 16)
    # entries of the table that are no pages have no slots
    run([20, 5], [3, 20], [7, -4, 9], 3, 4, 16, table=[[3, -9, -1, -1], [8, -1, -1, -1]])


def test_no_requests_and_no_tokens():
    announce("pages none")
    run([], [], [4, 5], 2, 3, 16)
    run([], [], [], 0, 0, 16)
    run([0, 3], [0, 0], [4, 5], 2, 3, 16)
    run([0, 0], [0, 2], [], 0, 0, 16)  # rows without entries


def test_prompts_of_thousands():
    announce("pages prompts")
    r = random.Random(1)
    lengths = [r.randint(0, 5000) for _ in range(70)]
    add = [r.randint(1, 9000) for _ in range(70)]
    need = sum(-(-(n + a) // 32) - -(-n // 32) for n, a in zip(lengths, add))
    run(lengths, add, [3 * i for i in range(need + 1)], need + 1, 450, 32)
    run(lengths, add, [3 * i for i in range(need)], need - 500, 450, 32)


def test_one_request_takes_every_token():
    announce("pages one request")
    run([0], [200001], list(range(12501)), 12501, 12501, 16)
    run([15], [200001], list(range(12501)), 12501, 12501, 16)
