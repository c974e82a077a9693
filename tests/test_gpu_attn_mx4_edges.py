"""The 4-bit cache where its kernels can go wrong and test_gpu_attn_mx4.py does not lead: see each test."""
import math

import pytest
import torch

import gated_delta_rule_08_amd as gdr
from attn_ref import check
from gpu_util import announce, ensure_built
from mx4_ref import Mx4Cache, attend

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(seed, dt, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dt])


def ints(xs):
    return torch.tensor(xs, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_decode_of_a_query_that_is_not_finite(dt, sign, bad):
    """NaN where it sees a key, whatever the signs of the keys there; 0 where it sees none; the other rows as they are."""
    announce("mx4 decode non-finite query %s %d %s" % (dt, sign, bad))
    lengths = [0, 1, 40, 700, 1500]
    for Hq, Hkv, d in ((4, 2, 128), (8, 1, 64), (16, 1, 128)):  # 4, 2 and 1 copies of the rows
        c = Mx4Cache(lengths, [0] * 5, Hkv, d, 64)
        for b, n in enumerate(lengths):
            k = make(10 + b, dt, n, Hkv, d)
            k[..., 7] = sign * (1 + k[..., 7].abs())  # the scores' infinities all of one sign
            c.put(b, 0, k, make(50 + b, dt, n, Hkv, d))
        q = make(1, dt, 5, 1, Hq, d)
        q[:, 0, 1, 7] = bad
        for scale in (0.1, -0.1):
            o = torch.full_like(q, 7.0).cuda()
            gdr.gdr_attn_decode_mx4(q.cuda(), *c.device(), ints(lengths), o, scale=scale)
            torch.cuda.synchronize()
            o = o.cpu()
            assert (o[0] == 0).all() and torch.isnan(o[1:, 0, 1]).all(), (Hq, scale)
            for b, n in enumerate(lengths):
                k, v = c.get(b, 0, n)
                ref, bound = attend(q[b].nan_to_num(0.0, 0.0, 0.0), k, v, n, 0, 0, scale, DT[dt])
                keep = torch.arange(Hq) != 1
                check("o[%d]" % b, o[b][:, keep], ref[:, keep], bound[:, keep])


# ---------------------------------------------------------------- append and read


def offsets(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32).cuda()


def append_and_read(dt, held, counts, Hkv, d, page, extra=0):
    """The append byte by byte, then everything the cache holds read back; `extra` tokens of no sequence at the end."""
    c = Mx4Cache(held, counts, Hkv, d, page)
    for b, n in enumerate(held):
        if n:
            c.put(b, 0, make(1000 + b, dt, n, Hkv, d), make(5000 + b, dt, n, Hkv, d))
    total = sum(counts)
    k, v = make(1, dt, total + extra, Hkv, d), make(2, dt, total + extra, Hkv, d)
    dev = c.device()
    gdr.gdr_attn_append_mx4(k.cuda(), v.cuda(), offsets(counts), ints(held), *dev)
    torch.cuda.synchronize()
    at = 0
    for b, n in enumerate(counts):
        if n:
            c.put(b, held[b], k[at:at + n], v[at:at + n])
        at += n
    for name, x, y in zip(("k_codes", "k_scales", "v_codes", "v_scales"), dev[:4], c.packed()):
        assert torch.equal(x.cpu(), y), name
    # from the middle of each sequence on
    first = [(h + n) // 3 for h, n in zip(held, counts)]
    there = [h + n - f for h, n, f in zip(held, counts, first)]
    total = sum(there)
    ko, vo = (torch.full((total + extra, Hkv, d), 9.0, dtype=DT[dt], device="cuda") for _ in range(2))
    gdr.gdr_attn_read_mx4(*dev, offsets(there), ko, vo, first=ints(first))
    torch.cuda.synchronize()
    ko, vo, at = ko.double().cpu(), vo.double().cpu(), 0
    for b, n in enumerate(there):
        if n:
            rk, rv = c.get(b, first[b], n)
            assert torch.equal(ko[at:at + n], rk) and torch.equal(vo[at:at + n], rv), b
        at += n
    assert (ko[at:] == 9).all() and (vo[at:] == 9).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_sequences_without_tokens(dt):
    """Idle sequences between the others, from none to thousands, in front and behind."""
    announce("mx4 sequences without tokens %s" % dt)
    counts = []
    for idle, n in ((0, 1), (1, 2), (3, 1), (4, 33), (5, 1), (6, 7), (63, 1), (64, 40), (1000, 3), (2500, 100), (2, 1)):
        counts += [0] * idle + [n]
    append_and_read(dt, [(7 * b) % 40 if b % 50 == 0 else 0 for b in range(len(counts))], counts, 2, 64, 32, extra=5)
    append_and_read(dt, [0] * 3000, [0] * 1700 + [1, 1, 1] + [0] * 1297, 1, 128, 32)
    append_and_read(dt, [0, 5, 0, 0], [0, 0, 0, 9], 1, 128, 32)


def test_many_sequences_without_tokens_take_no_time():
    """A million idle sequences between two tokens are not walked one by one (some 200 ms; the call takes 0.02)."""
    announce("mx4 a million idle sequences")
    N, Hkv, d, page = 1000002, 1, 64, 32
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = u8(2, Hkv, page, d // 2), u8(2, Hkv, page, d // 32), u8(2, Hkv, 1, d, 16), u8(2, Hkv, page, d // 32)
    table = torch.zeros(N, 1, dtype=torch.int32, device="cuda")
    table[-1] = 1
    cu = torch.ones(N + 1, dtype=torch.int32, device="cuda")
    cu[0], cu[-1] = 0, 2
    k, lens = make(1, "f32", 2, Hkv, d).cuda(), torch.zeros(N, dtype=torch.int32, device="cuda")
    out = [torch.zeros_like(k) for _ in range(2)]
    best = math.inf
    for _ in range(5):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        gdr.gdr_attn_append_mx4(k, k, cu, lens, *cache, table)
        gdr.gdr_attn_read_mx4(*cache, table, cu, *out)
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end))
    assert torch.equal(out[0], out[1]) and (out[0] != 0).any(-1).all()
    assert best < 5, "%.2f ms" % best


def ragged(total, parts, seed):
    """`parts` lengths that add up to total: some 0 or 1, the others far apart."""
    g = torch.Generator().manual_seed(seed)
    cut = [0] + sorted(torch.randint(0, total + 1, (parts - 3,), generator=g).tolist()) + [total]
    counts = [b - a for a, b in zip(cut, cut[1:])]
    big = max(range(len(counts)), key=counts.__getitem__)
    counts[big] -= 1
    return counts[:2] + [0] + counts[2:] + [1]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("total,parts,Hkv,d,page", [
    (2047, 14, 8, 128, 64), (2048, 14, 8, 128, 64), (2049, 14, 8, 128, 64), (2601, 9, 8, 128, 32),  # 16384 tokens x heads
    (8191, 20, 3, 64, 32), (8193, 20, 3, 64, 128), (4097, 3, 5, 128, 1024),  # two heads of 64 to a wave
    (2700, 120, 8, 128, 32), (3001, 420, 6, 128, 32),  # shorter sequences: ranges of 8 and of 2
])
def test_long_batches(dt, total, parts, Hkv, d, page):
    """Append and read of as many tokens as take ranges of 32, on both sides of where they begin."""
    announce("mx4 long batches %s %s" % (dt, (total, parts, Hkv, d, page)))
    counts = ragged(total, parts, total)
    assert sum(counts) == total
    held = [(37 * b) % 95 if b % 4 else 32 * (b % 3) for b in range(len(counts))]
    append_and_read(dt, held, counts, Hkv, d, page, extra=37 if total % 2 else 0)


def test_one_long_prompt():
    announce("mx4 one long prompt")
    for held, n in ((0, 5000), (17, 5003)):
        append_and_read("bf16", [held], [n], 4, 128, 64)


def guarded(x, space):
    """x in the middle of a larger allocation of sentinels: (the view, the allocation)."""
    pool = torch.full((x.numel() + 2 * space,), 0xA5, dtype=torch.uint8, device="cuda")
    view = pool[space:space + x.numel()].view(x.shape)
    view.copy_(x)
    return view, pool


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Hkv,d,page", [(2, 64, 32), (3, 128, 64)])
def test_append_writes_nowhere_else(dt, Hkv, d, page):
    """Offsets out of order or beyond the tokens, bad lengths and bad pages: nothing before, between or behind the caches, and
    no page that is in no row of the table."""
    announce("mx4 append writes nowhere else %s %s" % (dt, (Hkv, d, page)))
    N, space = 6, 1 << 16
    c = Mx4Cache([100] * N, [60] * N, Hkv, d, page, spare=5)
    used = set(c.table.view(-1).tolist())
    spare = [p for p in range(c.kc.shape[0]) if p not in used]
    assert len(spare) == 5
    total = 300
    k, v = make(1, dt, total, Hkv, d).cuda(), make(2, dt, total, Hkv, d).cuda()
    top = 2 ** 31 - 1
    pages = c.kc.shape[0]
    for cu in ([-5, 90, 30, top, 60, 20, -9], [0, 50, 100, 150, 200, 250, top], [299, 0, 299, 0, 299, 0, 299],
               [-2 ** 31, -1, 5, 300, 301, 10 ** 9, top], [0, 50, 100, 150, 200, 250, 300]):
        for lens in ([0] * N, [100, -1, top, 159, -2 ** 31, 10 ** 6], [160, 128, 159, 31, 33, 1]):
            for spoil in (False, True):
                table = c.table.clone()
                if spoil:
                    table[1, 0], table[2, -1], table[4, 1], table[5, 0] = pages, -1, top, -2 ** 31
                views, pools = zip(*(guarded(x, space) for x in c.packed()))
                gdr.gdr_attn_append_mx4(k, v, ints(cu), ints(lens), *views, table.cuda())
                torch.cuda.synchronize()
                for view, pool, before in zip(views, pools, c.packed()):
                    assert (pool[:space] == 0xA5).all() and (pool[-space:] == 0xA5).all(), (cu, lens)
                    assert torch.equal(view[spare].cpu(), before[spare]), (cu, lens)
    assert not torch.equal(views[0].cpu(), c.packed()[0])  # the last offsets are in order: most of it is written


# ---------------------------------------------------------------- decode: a wave for each unit


@pytest.mark.parametrize("B,Tq,Hq,Hkv,d,page,window,sinks,longest", [
    (513, 1, 16, 2, 64, 32, 0, 0, 200), (515, 1, 16, 2, 128, 32, 0, 0, 600),    # 8 rows: two copies
    (513, 2, 8, 2, 128, 64, 0, 0, 1000), (345, 1, 21, 3, 64, 64, 150, 2, 900),   # 8 and 7
    (1025, 1, 16, 1, 128, 32, 0, 0, 300), (343, 5, 12, 3, 128, 32, 0, 0, 100),   # 16 and 20: one copy, a second tile
    (513, 1, 17, 1, 128, 64, 300, 5, 700), (515, 9, 2, 1, 64, 32, 0, 0, 130),    # 17 and 18
])
def test_decode_many_short_units(B, Tq, Hq, Hkv, d, page, window, sinks, longest):
    """bf16 with more than four rows to a unit, over 1023 units of up to 1024 keys: a wave to each, the last workgroup not full."""
    announce("mx4 decode many short units %s" % ((B, Tq, Hq, Hkv, d, page, window, sinks, longest),))
    units = B * Hkv * -(-Tq * Hq // Hkv // 16)
    assert units >= 1024 and units % 4
    edges = [0, 1, 31, 32, 33, 127, 128, 129, longest]
    lengths = edges + [1 + 37 * b % min(200, longest) for b in range(B - len(edges))]
    decode_and_check("bf16", lengths, Tq, Hq, Hkv, d, page, window, sinks, every=7)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("G", [7, 8, 16, 20])
def test_decode_short_tables(dt, G):
    """Tables of up to 128 keys, or a window that leaves as few: the same form for few units too."""
    announce("mx4 decode short tables %s %d" % (dt, G))
    decode_and_check(dt, [0, 1, 32, 127, 128], 1, 2 * G, 2, 128, 32, 0, 0)
    decode_and_check(dt, [0, 1, 32, 127, 128], 1, G, 1, 64, 128, 0, 0)
    decode_and_check(dt, [5, 300, 97, 1000, 64], 1, G, 1, 128, 64, 90, 33)


def decode_and_check(dt, lengths, Tq, Hq, Hkv, d, page, window, sinks, every=1):
    c = Mx4Cache(lengths, [0] * len(lengths), Hkv, d, page)
    for b, n in enumerate(lengths):
        c.put(b, 0, make(10 + b, dt, n, Hkv, d), make(5000 + b, dt, n, Hkv, d))
    q = make(1, dt, len(lengths), Tq, Hq, d)
    o = torch.full_like(q, 7.0).cuda()
    gdr.gdr_attn_decode_mx4(q.cuda(), *c.device(), ints(lengths), o, window=window, sinks=sinks)
    torch.cuda.synchronize()
    o = o.cpu()
    for b in list(range(9)) + list(range(9, len(lengths), every)) + [len(lengths) - 1]:
        if b < len(lengths):
            k, v = c.get(b, 0, lengths[b])
            ref, bound = attend(q[b], k, v, lengths[b], window, sinks, d ** -0.5, DT[dt])
            check("o[%d]" % b, o[b], ref, bound)
