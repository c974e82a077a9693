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
