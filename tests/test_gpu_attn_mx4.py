"""The 4-bit cache on the GPU: append, read back and the decode step against the format's definition in 64 bits."""
import math

import pytest
import torch

import gated_delta_rule_08_amd as gdr
from attn_ref import check
from gpu_util import announce, ensure_built
from mx4_ref import VALUES, Mx4Cache, attend, quantise, value

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


def offsets(counts):
    return ints([sum(counts[:i]) for i in range(len(counts) + 1)])


def same_cache(got, c):
    for name, x, y in zip(("k_codes", "k_scales", "v_codes", "v_scales"), got, c.packed()):
        x = x.cpu()
        assert torch.equal(x, y), "%s: %d bytes differ" % (name, int((x != y).sum()))


# ---------------------------------------------------------------- append


def run_append(dt, held, counts, Hkv, d, page, k=None, v=None):
    c = Mx4Cache(held, counts, Hkv, d, page)
    for b, n in enumerate(held):
        c.put(b, 0, make(10 + b, dt, n, Hkv, d), make(50 + b, dt, n, Hkv, d))
    total = sum(counts)
    k = make(1, dt, total, Hkv, d) if k is None else k
    v = make(2, dt, total, Hkv, d) if v is None else v
    dev = c.device()
    gdr.gdr_attn_append_mx4(k.cuda(), v.cuda(), offsets(counts), ints(held), *dev)
    torch.cuda.synchronize()
    at = 0
    for b, n in enumerate(counts):
        c.put(b, held[b], k[at:at + n], v[at:at + n])
        at += n
    same_cache(dev[:4], c)
    return c, dev


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Hkv,d,page", [(1, 64, 32), (2, 128, 64), (3, 64, 256), (8, 128, 32)])
def test_append(dt, Hkv, d, page):
    announce("mx4 append %s %s" % (dt, (Hkv, d, page)))
    run_append(dt, [0, 1, 31, 32, 33, 5, 64, 0, 30, 7], [1, 1, 1, 2, 63, 0, 32, 100, 2, 29], Hkv, d, page)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_append_one_token_each(dt):
    """The step between a decode step and the next: one token for every sequence."""
    announce("mx4 append one each %s" % dt)
    run_append(dt, [(13 * b) % 71 for b in range(130)], [1] * 130, 2, 64, 32)


def test_append_of_every_rounding():
    """Values on, beside and between the codes' midpoints, at every limit of the scale."""
    announce("mx4 append roundings")
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    near = sorted({x for m in mids + VALUES + [6.5, 7.0] for x in (m, math.nextafter(m, 0), math.nextafter(m, 9))})
    near = torch.tensor(near, dtype=torch.float64).float()
    rows = []
    for e in (0, -3, 5, -100, -124, -126, -130, -149, 100, 120, 125):
        for top in (4.0, 6.0, 7.0, 7.0000005, 7.5, 3.5, 3.500001):
            x = torch.ldexp(near, torch.tensor(float(e)))
            x = torch.cat([x, -x])[torch.randperm(2 * len(near), generator=torch.Generator().manual_seed(len(rows)))]
            for part in x.split(31):
                row = torch.full((32,), 0.0)
                row[:len(part)] = part
                row[31] = math.ldexp(top, e) if e + 3 < 128 else 3.4e38
                rows.append(row)
    rows += [torch.zeros(32), -torch.zeros(32), torch.full((32,), 3.4028234663852886e38), torch.full((32,), 2.0 ** -149)]
    rows += [rows[i % 4] for i in range(-len(rows) % 4)]
    x = torch.stack(rows)
    assert torch.isfinite(x).all()
    x = x.reshape(-1, 2, 64)
    run_append("f32", [3], [x.shape[0]], 2, 64, 32, x, x.flip(0).contiguous())
    y = x.bfloat16()
    y[~torch.isfinite(y)] = 1.0
    run_append("bf16", [3], [y.shape[0]], 2, 64, 32, y, y.flip(0).contiguous())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_append_non_finite(dt):
    announce("mx4 append non-finite %s" % dt)
    k, v = make(1, dt, 40, 2, 128), make(2, dt, 40, 2, 128)
    k[3, 0, 5], k[7, 1, 127], k[39, 0, 64] = math.inf, -math.inf, math.nan
    v[0, 0, 0], v[31, 1, 33], v[32, 1, 100] = math.nan, math.inf, -math.inf
    c, _ = run_append(dt, [5], [40], 2, 128, 32, k, v)
    assert int((c.ks == 255).sum()) > 3


def test_append_bad_places():
    """Tokens without a place are not written: bad lengths, pages, offsets; tokens of no sequence."""
    announce("mx4 append bad places")
    Hkv, d, page = 2, 64, 32
    held, counts = [0, 10, 40, 0, 5, 0], [40, 40, 40, 8, 8, 8]
    c = Mx4Cache(held, counts, Hkv, d, page)
    for b, n in enumerate(held):
        c.put(b, 0, make(10 + b, "bf16", n, Hkv, d), make(50 + b, "bf16", n, Hkv, d))
    total = 4 + sum(counts) + 9
    k, v = make(1, "bf16", total, Hkv, d), make(2, "bf16", total, Hkv, d)
    dev = c.device()
    table = dev[4].clone()
    table[0, 1] = c.kc.shape[0]  # sequence 0: its second page lies outside the pool
    table[2, :] = -7
    lens = ints([0, 10, 40, -1, 2 ** 31 - 4, 0])
    cu = [4]
    for n in counts:
        cu.append(cu[-1] + n)
    gdr.gdr_attn_append_mx4(k.cuda(), v.cuda(), ints(cu), lens, *dev[:4], table)
    torch.cuda.synchronize()
    c.put(0, 0, k[4:36], v[4:36])
    c.put(1, 10, k[44:84], v[44:84])
    c.put(5, 0, k[cu[5]:cu[6]], v[cu[5]:cu[6]])
    same_cache(dev[:4], c)
    before = [x.clone() for x in dev[:4]]
    # offsets out of order and beyond the tokens: bounded reads, and no write behind the pages
    gdr.gdr_attn_append_mx4(k.cuda(), v.cuda(), ints([-5, 90, 30, 2 ** 31 - 1, 60, 20, -9]), ints([0] * 6), *dev)
    torch.cuda.synchronize()
    assert [x.shape for x in before] == [x.shape for x in dev[:4]]


# ---------------------------------------------------------------- read


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Hkv,d,page", [(1, 64, 32), (2, 128, 64), (3, 64, 256), (5, 128, 32)])
def test_read(dt, Hkv, d, page):
    announce("mx4 read %s %s" % (dt, (Hkv, d, page)))
    held = [0, 1, 31, 32, 33, 100, 257, 64]
    c = Mx4Cache(held, [0] * len(held), Hkv, d, page)
    for b, n in enumerate(held):
        k, v = make(10 + b, dt, n, Hkv, d), make(50 + b, dt, n, Hkv, d)
        k *= torch.ldexp(torch.ones(()), torch.randint(-100, 100, (n, Hkv, 1), generator=torch.Generator().manual_seed(b))).to(k.dtype)
        c.put(b, 0, k, v)
    for first in (None, [0, 1, 3, 32, 32, 65, 31, 17]):
        counts = held if first is None else [n - f for n, f in zip(held, first)]
        total = sum(counts) + 3
        k, v = (torch.full((total, Hkv, d), 9.0, dtype=DT[dt], device="cuda") for _ in range(2))
        gdr.gdr_attn_read_mx4(*c.device(), offsets(counts), k, v, first=None if first is None else ints(first))
        torch.cuda.synchronize()
        at = 0
        for b, n in enumerate(counts):
            rk, rv = c.get(b, 0 if first is None else first[b], n)
            assert torch.equal(k[at:at + n].double().cpu(), rk) and torch.equal(v[at:at + n].double().cpu(), rv), b
            at += n
        assert (k[at:] == 9).all() and (v[at:] == 9).all()


def test_read_nan_and_bad_places():
    announce("mx4 read bad places")
    c = Mx4Cache([70, 40], [0, 0], 2, 64, 32)
    k = make(1, "f32", 70, 2, 64)
    k[3, 1, 40] = math.inf
    c.put(0, 0, k, k)
    c.put(1, 0, k[:40], k[:40])
    dev = c.device()
    table = dev[4].clone()
    table[0, 1], table[1, 0] = -1, 99
    ko, vo = (torch.full((110, 2, 64), 9.0, device="cuda") for _ in range(2))
    gdr.gdr_attn_read_mx4(*dev[:4], table, ints([0, 70, 110]), ko, vo, first=ints([0, 0]))
    torch.cuda.synchronize()
    rk, rv = c.get(0, 0, 70)
    for x, r in ((ko, rk), (vo, rv)):
        x = x.cpu()
        assert torch.equal(x[:32].double().nan_to_num(77.0), r[:32].nan_to_num(77.0)) and torch.isnan(x[3, 1, 32:]).all()
        assert torch.equal(x[64:70].double(), r[64:70])
        assert (x[32:64] == 9).all() and (x[70:102] == 9).all() and not (x[102:] == 9).any()
    ko.fill_(9.0)
    gdr.gdr_attn_read_mx4(*dev, ints([0, 5, 10]), ko, vo, first=ints([-1, 2 ** 31 - 3]))
    torch.cuda.synchronize()
    assert (ko == 9).all()


# ---------------------------------------------------------------- decode


def run_decode(dt, lengths, Tq, Hq, Hkv, d, page, window, sinks, scale=None, big=False):
    c = Mx4Cache(lengths, [0] * len(lengths), Hkv, d, page)
    for b, n in enumerate(lengths):
        c.put(b, 0, make(10 + b, dt, n, Hkv, d) * (8 if big else 1), make(50 + b, dt, n, Hkv, d))
    B = len(lengths)
    q = make(1, dt, B, Tq, Hq, d)
    o = torch.full_like(q, 7.0).cuda()
    gdr.gdr_attn_decode_mx4(q.cuda(), *c.device(), ints(lengths), o, window=window, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    worst = 0.0
    for b, n in enumerate(lengths):
        k, v = c.get(b, 0, n)
        ref, bound = attend(q[b], k, v, n, window, sinks, d ** -0.5 if scale is None else scale, DT[dt])
        worst = max(worst, check("o[%d]" % b, o[b], ref, bound))
    return worst


LENGTHS = [0, 1, 2, 31, 32, 33, 95, 127, 128, 129, 160, 300]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Tq,Hq,Hkv,d,page,window,sinks", [
    (1, 1, 1, 64, 32, 0, 0), (1, 8, 2, 128, 32, 0, 0), (1, 6, 2, 64, 64, 0, 0), (1, 32, 1, 128, 64, 0, 0),
    (1, 17, 1, 64, 32, 40, 3), (1, 4, 4, 128, 128, 1, 0), (1, 8, 2, 64, 128, 50, 70), (1, 5, 5, 128, 32, 33, 1),
    (3, 8, 2, 128, 64, 0, 0), (5, 6, 2, 64, 32, 37, 2), (8, 4, 1, 64, 32, 100, 33), (64, 2, 2, 128, 32, 0, 0),
    (17, 1, 1, 64, 64, 16, 1),
])
def test_decode(dt, Tq, Hq, Hkv, d, page, window, sinks):
    announce("mx4 decode %s %s" % (dt, (Tq, Hq, Hkv, d, page, window, sinks)))
    assert gdr.gdr_attn_decode_mx4_workspace_bytes(DT[dt], 12, Tq, Hq, Hkv, d, page, -(-300 // page), window, sinks) == 0
    run_decode(dt, LENGTHS, Tq, Hq, Hkv, d, page, window, sinks)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Tq,Hq,Hkv,d,page,window,sinks", [
    (1, 1, 1, 128, 32, 0, 0), (1, 8, 2, 128, 64, 0, 0), (1, 6, 2, 64, 32, 700, 5), (2, 20, 1, 128, 64, 0, 0),
    (1, 17, 1, 64, 32, 520, 300), (4, 5, 5, 128, 32, 1000, 1), (1, 36, 2, 64, 256, 0, 0), (7, 6, 3, 64, 32, 600, 64),
])
def test_decode_long_tables(dt, Tq, Hq, Hkv, d, page, window, sinks):
    """Tables with room for long sequences: shares of the batch's blocks, joined where they meet."""
    announce("mx4 decode long tables %s %s" % (dt, (Tq, Hq, Hkv, d, page, window, sinks)))
    lengths = [0, 1, 127, 128, 129, 300, 640, 5, 1900]
    assert gdr.gdr_attn_decode_mx4_workspace_bytes(DT[dt], 9, Tq, Hq, Hkv, d, page, -(-1900 // page), window, sinks) > 0
    run_decode(dt, lengths, Tq, Hq, Hkv, d, page, window, sinks)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Tq,Hq,Hkv,d,page,window,sinks", [
    (1, 1, 1, 128, 64, 0, 0), (1, 8, 2, 64, 32, 0, 0), (1, 14, 2, 128, 32, 4100, 33), (2, 20, 1, 64, 128, 0, 0),
])
def test_decode_dealt(dt, Tq, Hq, Hkv, d, page, window, sinks):
    """Tables with room for more keys than a unit takes by itself however many units there are."""
    announce("mx4 decode dealt %s %s" % (dt, (Tq, Hq, Hkv, d, page, window, sinks)))
    run_decode(dt, [0, 1, 127, 128, 4999, 129, 513, 1, 2500], Tq, Hq, Hkv, d, page, window, sinks)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,Tq,Hq,Hkv,d,page,window,sinks,longest", [
    (147, 1, 7, 7, 128, 32, 0, 0, 300), (129, 1, 16, 8, 64, 32, 0, 0, 1024), (65, 3, 16, 16, 128, 64, 0, 0, 700),
    (131, 1, 16, 8, 64, 32, 500, 3, 1500),
])
def test_decode_many_short(dt, B, Tq, Hq, Hkv, d, page, window, sinks, longest):
    """A wave for each of many short units, the last workgroup not full."""
    announce("mx4 decode many short %s %s" % (dt, (B, Tq, Hq, Hkv, d, page, window, sinks, longest)))
    edges = [0, 1, 31, 32, 33, 127, 128, 129, longest]
    run_decode(dt, edges + [1 + 37 * b % 200 for b in range(B - len(edges))], Tq, Hq, Hkv, d, page, window, sinks)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_decode_scales(dt, scale):
    announce("mx4 decode scale %s %s" % (dt, scale))
    run_decode(dt, [1, 40, 700], 2, 4, 2, 64, 64, 0, 0, scale=scale)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_decode_skips_and_hides(dt):
    """Bad lengths are skipped; pages outside the pool are hidden, all of a sequence's among them."""
    announce("mx4 decode skips %s" % dt)
    Hq, Hkv, d, page = 4, 2, 128, 32
    lengths = [100, 100, 100, 100, 600, 64]
    c = Mx4Cache(lengths, [0] * 6, Hkv, d, page)
    for b, n in enumerate(lengths):
        c.put(b, 0, make(10 + b, dt, n, Hkv, d), make(50 + b, dt, n, Hkv, d))
    q = make(1, dt, 6, 2, Hq, d)
    o = torch.full_like(q, 7.0).cuda()
    dev = c.device()
    table = dev[4].clone()
    table[2, 1], table[3, :], table[4, 3] = -1, 10 ** 6, c.kc.shape[0]
    lens = ints([-1, c.table.shape[1] * page + 1, 100, 100, 600, 64])
    gdr.gdr_attn_decode_mx4(q.cuda(), *dev[:4], table, lens, o)
    torch.cuda.synchronize()
    assert (o[:2] == 7).all() and (o[3] == 0).all()
    for b, hidden in ((2, range(32, 64)), (4, range(96, 128)), (5, ())):
        n = lengths[b]
        k, v = c.get(b, 0, n)
        keep = torch.tensor([j for j in range(n) if j not in hidden])
        # the hidden pages lie before both queries: the others keep their order
        ref, bound = attend(q[b], k[keep], v[keep], len(keep), 0, 0, d ** -0.5, DT[dt])
        check("o[%d]" % b, o[b], ref, bound)
    for bad in (2 ** 31 - 1, 2 ** 31 - 64, -2 ** 31):
        o.fill_(7.0)
        gdr.gdr_attn_decode_mx4(q.cuda(), *dev[:4], table, ints([bad] * 6), o)
        torch.cuda.synchronize()
        assert (o == 7).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [200, 1500])
def test_decode_non_finite(dt, n):
    """A block that stands for NaN reaches the rows and channels that see it, and no others."""
    announce("mx4 decode non-finite %s %d" % (dt, n))
    Hq, Hkv, d, page, Tq, window = 4, 2, 64, 32, 2, 100
    c = Mx4Cache([n] * 4, [0] * 4, Hkv, d, page)
    q = make(1, dt, 4, Tq, Hq, d)
    for b in range(4):
        k, v = make(10 + b, dt, n, Hkv, d), make(50 + b, dt, n, Hkv, d)
        if b == 0:
            k[n - 30, 0, 3] = math.nan  # seen by both queries
        if b == 1:
            v[n - 30, 1, 40] = math.inf  # channels 32 .. 63 of head 1
        if b == 2:  # hidden from both
            k[n - 150, 0, 3], v[n - 150, 1, 3] = math.inf, math.nan
        if b == 3:  # the last position: hidden from the first query only
            k[n - 1, 0, 3], v[n - 1, 1, 3] = math.nan, math.nan
        c.put(b, 0, k, v)
    o = torch.full_like(q, 7.0).cuda()
    gdr.gdr_attn_decode_mx4(q.cuda(), *c.device(), ints([n] * 4), o, window=window)
    torch.cuda.synchronize()
    o = o.cpu()
    nan = torch.zeros(4, Tq, Hq, d, dtype=torch.bool)
    nan[0, :, :2] = True
    nan[1, :, 2:, 32:] = True
    nan[3, 1, :2] = True
    nan[3, 1, 2:, :32] = True
    assert torch.equal(torch.isnan(o), nan)
    for b in range(4):
        k, v = c.get(b, 0, n)
        ref, bound = attend(q[b], k.nan_to_num(0.0), v.nan_to_num(0.0), n, window, 0, d ** -0.5, DT[dt])
        keep = ~nan[b]
        check("o[%d]" % b, torch.where(keep, o[b], torch.zeros(())), torch.where(keep, ref, torch.zeros(()).double()),
              torch.where(keep, bound, torch.zeros(()).double()))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("byte", [0, 252, 253, 254, 255])
@pytest.mark.parametrize("code", [0, 7, 15])
def test_decode_hidden_bytes_have_no_influence(dt, byte, code):
    """Whatever lies in the slots behind a sequence, in scales that no append writes too (253 and 254 times a code
    leave the range of bf16), the output is that of a cleared cache, bit by bit."""
    announce("mx4 decode hidden bytes %s %d %d" % (dt, byte, code))
    lengths = [1, 5, 33, 70, 130]
    for Hq, Hkv, d in ((4, 2, 128), (8, 1, 64), (16, 1, 128)):  # 4, 2 and 1 copies of the rows
        c = Mx4Cache(lengths, [0] * 5, Hkv, d, 64)
        outs = []
        for scale, fill in ((byte, code), (1, 0)):
            c.ks.fill_(scale), c.vs.fill_(scale), c.kc.fill_(fill), c.vc.fill_(fill)
            for b, n in enumerate(lengths):
                c.put(b, 0, make(10 + b, dt, n, Hkv, d), make(50 + b, dt, n, Hkv, d))
            q = make(1, dt, 5, 1, Hq, d).cuda()
            outs.append(torch.full_like(q, 7.0))
            gdr.gdr_attn_decode_mx4(q, *c.device(), ints(lengths), outs[-1])
            torch.cuda.synchronize()
        assert torch.isfinite(outs[1]).all() and torch.equal(outs[0], outs[1])


def test_decode_a_nan_far_below_the_maximum_is_seen():
    """A NaN value whose weight underflows, in another wave's or another workgroup's part."""
    announce("mx4 decode underflow")
    Hq, Hkv, d, page = 2, 1, 64, 32
    for n, at in ((520, 3), (6000, 5)):
        c = Mx4Cache([n], [0], Hkv, d, page)
        k, v = torch.full((n, 1, d), -4.0), make(5, "f32", n, 1, d)
        k[n - 1] = 4.0
        v[at, 0, 1] = math.nan
        c.put(0, 0, k, v)
        q = torch.full((1, 1, Hq, d), 4.0)
        o = torch.zeros_like(q).cuda()
        gdr.gdr_attn_decode_mx4(q.cuda(), *c.device(), ints([n]), o, scale=1.0)
        torch.cuda.synchronize()
        assert torch.isnan(o[..., :32]).all() and torch.isfinite(o[..., 32:]).all()
    q[0, 0, 1, 7] = math.inf
    gdr.gdr_attn_decode_mx4(q.cuda(), *c.device(), ints([n]), o, scale=1.0)
    torch.cuda.synchronize()
    assert torch.isnan(o[0, 0, 1]).all() and torch.isfinite(o[0, 0, 0, 32:]).all()


def test_decode_many_sequences():
    """More sequences than one scan of the lengths takes, some of them skipped; repeated calls agree bit by bit."""
    announce("mx4 decode many sequences")
    n, page, Hq, Hkv, d = 700, 32, 4, 2, 64
    lengths = [(37 * b) % 90 if b % 5 else 0 for b in range(n)]
    lengths[3], lengths[400], lengths[699] = 800, 1300, 600
    c = Mx4Cache(lengths, [0] * n, Hkv, d, page)
    for b, m in enumerate(lengths):
        c.put(b, 0, make(10 + b, "bf16", m, Hkv, d), make(1000 + b, "bf16", m, Hkv, d))
    q = make(1, "bf16", n, Hq, d)
    bad = [0, 1, 255, 256, 511, 650]
    lens = list(lengths)
    for b in bad:
        lens[b] = -3 if b % 2 else 10 ** 6
    dev, lens_d, qd = c.device(), ints(lens), q.cuda()
    outs = []
    for _ in range(3):
        o = torch.full_like(qd, 7.0)
        gdr.gdr_attn_decode_mx4(qd, *dev, lens_d, o)
        torch.cuda.synchronize()
        outs.append(o.cpu())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for b, m in enumerate(lengths):
        if b in bad:
            assert (outs[0][b] == 7).all()
            continue
        k, v = c.get(b, 0, m)
        ref, bound = attend(q[b:b + 1], k, v, m, 0, 0, d ** -0.5, torch.bfloat16)
        check("o[%d]" % b, outs[0][b:b + 1], ref, bound)


def test_value_of_every_code():
    """The read of every code at scales from the smallest to the largest."""
    announce("mx4 codes")
    c = Mx4Cache([128], [0], 1, 64, 32)
    g = torch.Generator().manual_seed(3)
    c.kc = torch.randint(0, 16, c.kc.shape, generator=g, dtype=torch.uint8)
    c.vc = torch.randint(0, 16, c.vc.shape, generator=g, dtype=torch.uint8)
    c.ks = torch.randint(1, 253, c.ks.shape, generator=g, dtype=torch.uint8)
    c.vs = torch.randint(1, 253, c.vs.shape, generator=g, dtype=torch.uint8)
    c.ks.view(-1)[::7], c.vs.view(-1)[::5], c.ks.view(-1)[1::9] = 1, 252, 252
    for dt in DT.values():
        k, v = (torch.zeros(128, 1, 64, dtype=dt, device="cuda") for _ in range(2))
        gdr.gdr_attn_read_mx4(*c.device(), ints([0, 128]), k, v)
        torch.cuda.synchronize()
        rk, rv = c.get(0, 0, 128)
        assert torch.equal(k.double().cpu(), rk) and torch.equal(v.double().cpu(), rv)
    codes, scales = quantise(rk)
    assert torch.equal(value(codes, scales), rk)
