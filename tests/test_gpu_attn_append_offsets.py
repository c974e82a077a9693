"""The append to the pages with offsets that are out of order or out of range: what it may write, and nothing else."""
import random

import pytest
import torch

import gated_delta_rule_08_amd as gdr
from gpu_util import announce, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def append(cu, lens, table, total, pages, page, Hkv, d):
    """The pages after an append of tokens t = 1, 2, .. (k = t, v = -t) to pages full of 0.5."""
    t = torch.arange(1, total + 1, dtype=torch.float32, device="cuda").reshape(-1, 1, 1).expand(total, Hkv, d).contiguous()
    k_pages, v_pages = (torch.full((pages, Hkv, page, d), 0.5, device="cuda") for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    gdr.gdr_attn_append(t, -t, i32(cu), i32(lens), k_pages, v_pages, i32(table))
    k, v = k_pages.cpu(), v_pages.cpu()
    assert torch.equal(torch.where(k == 0.5, k, -k), v)  # the same places in both
    assert torch.equal(k, k[:, :1, :, :1].expand_as(k))  # a token's row is one token's in every head and channel
    return k[:, 0, :, 0]


def places(cu, lens, table, total, pages, page):
    """{(page, slot): token + 1} of every token in every sequence whose range holds it."""
    out = {}
    for s, n in enumerate(lens):
        for t in range(max(0, cu[s]), min(total, cu[s + 1])) if cu[s] >= 0 and n >= 0 else ():
            pos = n + t - cu[s]
            if pos // page < len(table[s]) and 0 <= table[s][pos // page] < pages:
                out[table[s][pos // page], pos % page] = t + 1
    return out


def test_nothing_has_a_place():
    """Reversed, empty and negative ranges, and ranges of sequences without a page or with a negative length."""
    announce("attn append, nothing has a place")
    table, lens = [[0, 1], [2, -1], [3, 99], [4, 5]], [8, 8, 8, -3]
    for cu in ([-9] * 5, [5, 2, 60, 60, 60], [60, 60, 60, 60, 60], [40, 30, 20, 10, 0], [-5, 40, 40, 40, 40]):
        assert (append(cu, lens, table, 40, 6, 8, 1, 64) == 0.5).all(), cu


def test_sequences_in_order_among_odd_ranges():
    """Offsets in order are exact, also where the last ones pass the packed total or the first is not 0."""
    announce("attn append, odd ranges in order")
    table, lens = [[0, 1], [2, 3], [6, 7], [4, 5]], [3, 0, 8, 1]
    for cu in ([0, 10, 10, 20, 30], [4, 5, 9, 9, 500], [0, 0, 0, 0, 13], [0, 13, 90, 90, 100]):
        got, want = append(cu, lens, table, 30, 8, 8, 2, 64), places(cu, lens, table, 30, 8, 8)
        assert {(p, s): int(got[p, s]) for p, s in (got != 0.5).nonzero().tolist()} == want, cu


@pytest.mark.parametrize("seed", range(12))
def test_offsets_out_of_order(seed):
    """Each slot holds what was there or the token that a range which holds it puts there."""
    announce("attn append, out of order %d" % seed)
    rng = random.Random(seed)
    N, total, page, width = rng.choice([4, 7, 90]), 300, 16, 5
    order = list(range(N * width + 3))
    rng.shuffle(order)
    table = [order[s * width:(s + 1) * width] for s in range(N)]
    lens = [rng.randint(0, 40) for _ in range(N)]
    cu = [rng.randint(-20, total + 60) for _ in range(N + 1)]
    if seed % 2:  # in order but for a few
        cu.sort()
        for _ in range(2):
            cu[rng.randrange(N + 1)] = rng.randint(0, total)
    got, may = append(cu, lens, table, total, N * width + 3, page, 1, 64), places(cu, lens, table, total, N * width + 3, page)
    for p, s in (got != 0.5).nonzero().tolist():
        assert may.get((p, s)) == int(got[p, s]), (cu, p, s)
