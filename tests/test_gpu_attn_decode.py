"""Paged decode attention and the append to the pages against the float64 definition."""
import pytest
import torch

import gated_delta_rule_08_amd as gdr
from attn_ref import attend, check
from gpu_util import announce, ensure_built

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(seed, dt, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dt])


class Cache:
    """A paged cache on the CPU: NaN wherever no token is, pages in random order."""

    def __init__(self, dt, lengths, room, Hkv, d, page, seed=0):
        self.page, self.lengths = page, list(lengths)
        need = [-(-(n + r) // page) for n, r in zip(lengths, room)]
        order = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(seed)).tolist()
        width = max(1, max(need, default=1))
        self.table = torch.full((len(lengths), width), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
            order = order[n:]
        self.k = torch.full((sum(need) + 2, Hkv, page, d), float("nan"), dtype=DT[dt])
        self.v = self.k.clone()
        self.tokens = [(make(100 + b, dt, n, Hkv, d), make(200 + b, dt, n, Hkv, d)) for b, n in enumerate(lengths)]
        for b in range(len(lengths)):
            self.put(b, 0, *self.tokens[b])

    def put(self, b, at, k, v):
        for i in range(k.shape[0]):
            p = int(self.table[b, (at + i) // self.page])
            self.k[p, :, (at + i) % self.page] = k[i]
            self.v[p, :, (at + i) % self.page] = v[i]

    def device(self):
        return (self.k.cuda(), self.v.cuda(), self.table.cuda(), torch.tensor(self.lengths, dtype=torch.int32).cuda())


def same(a, b):
    """Bitwise (NaN where NaN)."""
    view = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.cpu().contiguous().view(view), b.cpu().contiguous().view(view))


def run_decode(dt, lengths, Hq, Hkv, d, page, window, sinks, scale=None, tail=0):
    c = Cache(dt, lengths, [1 + tail] * len(lengths), Hkv, d, page)
    B = len(lengths)
    q, k, v = make(1, dt, B, Hq, d), make(2, dt, B, Hkv, d), make(3, dt, B, Hkv, d)
    kp, vp, table, lens = c.device()
    o = torch.full_like(q, 7.0).cuda()
    gdr.gdr_attn_decode(q.cuda(), k.cuda(), v.cuda(), kp, vp, table, lens, o, window=window, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    for b, n in enumerate(lengths):
        c.put(b, n, k[b:b + 1], v[b:b + 1])
        full = [torch.cat([t, x[b:b + 1]]) for t, x in zip(c.tokens[b], (k, v))]
        ref = attend(q[b:b + 1], *full, window, sinks, d ** -0.5 if scale is None else scale, DT[dt])
        check("o[%d]" % b, o[b:b + 1], *ref["o"])
    assert same(kp, c.k) and same(vp, c.v)
    return o


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d,page,window,sinks", [
    (1, 1, 64, 1, 0, 0), (8, 2, 128, 16, 0, 0), (6, 2, 64, 4, 0, 0), (32, 1, 128, 64, 0, 0), (17, 1, 64, 32, 40, 3),
    (4, 4, 128, 16, 1, 0), (8, 2, 64, 128, 50, 70), (5, 5, 128, 2, 33, 1), (16, 2, 64, 256, 1000, 4),
])
def test_decode(dt, Hq, Hkv, d, page, window, sinks):
    announce("attn decode %s %s" % (dt, (Hq, Hkv, d, page, window, sinks)))
    run_decode(dt, [0, 1, 15, 16, 31, 33, 127, 128, 300], Hq, Hkv, d, page, window, sinks)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,d,page,window,sinks", [
    (1, 1, 128, 1, 0, 0), (8, 2, 128, 16, 0, 0), (6, 2, 64, 4, 700, 5), (40, 1, 128, 64, 0, 0), (17, 1, 64, 32, 520, 300),
    (4, 4, 128, 16, 600, 0), (5, 5, 128, 2, 1000, 1), (36, 2, 64, 256, 0, 0),
])
def test_decode_long_tables(dt, Hq, Hkv, d, page, window, sinks):
    """Tables with room for long sequences: the shares of the batch's key blocks, joined where they meet."""
    announce("attn decode long tables %s %s" % (dt, (Hq, Hkv, d, page, window, sinks)))
    assert gdr.gdr_attn_decode_workspace_bytes(DT[dt], 9, Hq, Hkv, d, page, -(-900 // page), window, sinks) > 0
    run_decode(dt, [0, 1, 127, 128, 129, 300, 640, 5, 899], Hq, Hkv, d, page, window, sinks)


def test_decode_many_sequences():
    """More sequences than one scan of the lengths takes, among them empty, out of range and without a page."""
    announce("attn decode many sequences")
    n, page, Hq, Hkv, d = 700, 16, 4, 2, 64
    lengths = [(37 * b) % 90 if b % 5 else 0 for b in range(n)]
    lengths[3], lengths[400], lengths[699] = 800, 1300, 600
    c = Cache("bf16", lengths, [1] * n, Hkv, d, page)
    q, k, v = make(1, "bf16", n, Hq, d), make(2, "bf16", n, Hkv, d), make(3, "bf16", n, Hkv, d)
    kp, vp, table, lens = c.device()
    bad = [0, 1, 255, 256, 257, 511, 512, 650]
    for i, b in enumerate(bad):
        if i % 3 == 0:
            lens[b] = -1 - b
        elif i % 3 == 1:
            lens[b] = table.shape[1] * page + b
        else:
            table[b, lengths[b] // page] = -1
    o = torch.full_like(q, 7.0).cuda()
    gdr.gdr_attn_decode(q.cuda(), k.cuda(), v.cuda(), kp, vp, table, lens, o)
    torch.cuda.synchronize()
    for b, m in enumerate(lengths):
        if b in bad:
            assert (o[b] == 7).all()
            continue
        c.put(b, m, k[b:b + 1], v[b:b + 1])
        full = [torch.cat([t, x[b:b + 1]]) for t, x in zip(c.tokens[b], (k, v))]
        check("o[%d]" % b, o[b:b + 1], *attend(q[b:b + 1], *full, 0, 0, 0.125, torch.bfloat16)["o"])
    assert same(kp, c.k) and same(vp, c.v)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_decode_many_heads_and_many_parts(dt):
    """A long sequence, cut into dozens of parts, among short ones with enough heads that each is joined by one wave."""
    announce("attn decode many heads and parts %s" % dt)
    run_decode(dt, [30000] + [b % 7 for b in range(40)], 32, 4, 64, 256, 0, 0)


def test_cache_beyond_4_gib():
    """Page tensors of 8.6 GB each, the sequence's pages at their far end and at their front."""
    announce("attn cache beyond 4 GiB")
    pages, Hkv, Hq, page, d, n = 1 << 17, 2, 4, 128, 128, 700
    kp = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    table = torch.tensor([[pages - 1, 0, pages - 2, pages // 2 + 3, 1, pages - 7, -1]], dtype=torch.int32, device="cuda")
    k, v, q = make(1, "bf16", n + 1, Hkv, d), make(2, "bf16", n + 1, Hkv, d), make(3, "bf16", 1, Hq, d)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdr.gdr_attn_append(k[:n].cuda(), v[:n].cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda"), lens, kp, vp, table)
    lens += n
    o = torch.empty_like(q).cuda()
    gdr.gdr_attn_decode(q.cuda(), k[n:].cuda(), v[n:].cuda(), kp, vp, table, lens, o)
    check("o", o, *attend(q, k, v, 0, 0, d ** -0.5, torch.bfloat16)["o"])
    assert same(kp[pages - 7, :, n % page], k[n]) and same(vp[pages - 2, :, 5], v[2 * page + 5])


def test_append_many_sequences():
    """Units of one workgroup from many sequences, empty ones between them."""
    announce("attn append many sequences")
    page, Hkv, d = 4, 1, 64
    new = [(i * 7) % 5 for i in range(200)]
    lengths = [(i * 3) % 11 for i in range(200)]
    c = Cache("bf16", lengths, new, Hkv, d, page)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    k, v = make(1, "bf16", cu[-1], Hkv, d), make(2, "bf16", cu[-1], Hkv, d)
    kp, vp, table, lens = c.device()
    gdr.gdr_attn_append(k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), lens, kp, vp, table)
    for b, n in enumerate(new):
        c.put(b, lengths[b], k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]])
    assert same(kp, c.k) and same(vp, c.v)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 200)])
def test_decode_split_over_the_length(dt, window, sinks):
    """Long and short sequences in one call: most are cut into parts and joined, short ones are not."""
    announce("attn decode split %s %d" % (dt, window))
    assert gdr.gdr_attn_decode_workspace_bytes(DT[dt], 5, 4, 2, 64, 16, 4000 // 16 + 1, window, sinks) > 0
    run_decode(dt, [4000, 0, 129, 2049, 513], 4, 2, 64, 16, window, sinks)


@pytest.mark.parametrize("scale", [0.0, -0.5, 3.0])
def test_decode_scale(scale):
    announce("attn decode scale %g" % scale)
    run_decode("f32", [100, 900], 4, 2, 64, 16, 0, 0, scale=scale)


def test_bad_tables_are_refused_by_the_kernel():
    """Sequences with a bad length or page write nothing; an invalid page further back hides its positions."""
    announce("attn decode bad table")
    lengths, page, Hq, Hkv, d = [40, 40, 40, 40, 40, 40], 16, 4, 2, 64
    c = Cache("f32", lengths, [1] * 6, Hkv, d, page)
    q, k, v = make(1, "f32", 6, Hq, d), make(2, "f32", 6, Hkv, d), make(3, "f32", 6, Hkv, d)
    kp, vp, table, lens = c.device()
    lens[0], lens[1] = -1, 48                      # negative; no room in the 3-page row
    table[2, 2], table[3, 2] = -1, kp.shape[0]     # the new position's page
    table[4, 0] = kp.shape[0] + 5                  # positions 0..15
    o = torch.full_like(q, 7.0).cuda()
    gdr.gdr_attn_decode(q.cuda(), k.cuda(), v.cuda(), kp, vp, table, lens, o)
    torch.cuda.synchronize()
    assert (o[:4] == 7).all()
    for b, first in ((4, 16), (5, 0)):
        c.put(b, 40, k[b:b + 1], v[b:b + 1])
        full = [torch.cat([t, x[b:b + 1]])[first:] for t, x in zip(c.tokens[b], (k, v))]
        check("o", o[b:b + 1], *attend(q[b:b + 1], *full, 0, 0, 0.125, torch.float32)["o"])
    assert same(kp, c.k) and same(vp, c.v)


@pytest.mark.parametrize("dt,d,page", [("bf16", 128, 16), ("f32", 64, 8)])
def test_append(dt, d, page):
    announce("attn append %s" % dt)
    Hkv, lengths, new = 3, [0, 5, 16, 31, 7], [40, 0, 1, 20, 17]
    c = Cache(dt, lengths, new, Hkv, d, page)
    cu = [3]
    for n in new:
        cu.append(cu[-1] + n)
    k, v = make(1, dt, cu[-1] + 6, Hkv, d), make(2, dt, cu[-1] + 6, Hkv, d)
    kp, vp, table, lens = c.device()
    gdr.gdr_attn_append(k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), lens, kp, vp, table)
    for b, n in enumerate(new):
        c.put(b, lengths[b], k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]])
    assert same(kp, c.k) and same(vp, c.v)


def test_append_leaves_out_what_has_no_place():
    announce("attn append, no place")
    page, Hkv, d = 8, 1, 64
    c = Cache("f32", [8, 8, 8, 8], [8, 8, 8, 8], Hkv, d, page)
    k, v = make(1, "f32", 40, Hkv, d), make(2, "f32", 40, Hkv, d)
    kp, vp, table, lens = c.device()
    table[1, 1], table[2, 1], lens[3] = -1, kp.shape[0], -3
    cu = torch.tensor([0, 12, 20, 30, 40], dtype=torch.int32).cuda()  # 12 tokens: 4 beyond the table row
    gdr.gdr_attn_append(k.cuda(), v.cuda(), cu, lens, kp, vp, table)
    c.put(0, 8, k[:8], v[:8])
    assert same(kp, c.k) and same(vp, c.v)
    for bad in ([0, 50, 20, 30, 40], [5, 2, 60, 60, 60], [-9, -9, -9, -9, -9]):
        gdr.gdr_attn_append(k.cuda(), v.cuda(), torch.tensor(bad, dtype=torch.int32).cuda(), lens, kp, vp, table)
    torch.cuda.synchronize()


@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 3)])
def test_prompt_then_tokens(window, sinks):
    """As a server uses them: prefill a batch of prompts, append their keys, decode token by token; every
    token's output is the last row of a prefill of the whole sequence."""
    announce("attn prompt then tokens %d" % window)
    dt, Hq, Hkv, d, page, steps = "bf16", 8, 2, 128, 16, 5
    lens = [33, 1, 70]
    total = [n + steps for n in lens]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    full = [(make(10 + b, dt, n, Hq, d), make(20 + b, dt, n, Hkv, d), make(30 + b, dt, n, Hkv, d)) for b, n in enumerate(total)]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, v = (torch.cat([full[b][i][:n] for b, n in enumerate(lens)]).cuda() for i in range(3))
    o = torch.empty_like(q)
    gdr.gdr_attn_prefill_varlen(q, k, v, dev(cu), dev(cu), o, max_seqlen_q=70, window=window, sinks=sinks)
    c = Cache(dt, [0, 0, 0], total, Hkv, d, page)
    kp, vp, table, held = c.device()
    gdr.gdr_attn_append(k, v, dev(cu), held, kp, vp, table)
    held += dev(lens)
    for t in range(steps):
        q1, k1, v1 = (torch.stack([full[b][i][n + t] for b, n in enumerate(lens)]).cuda() for i in range(3))
        o1 = torch.empty_like(q1)
        gdr.gdr_attn_decode(q1, k1, v1, kp, vp, table, held, o1, window=window, sinks=sinks)
        held += 1
        for b, n in enumerate(lens):
            x = [y[:n + t + 1] for y in full[b]]
            ref = attend(*x, window, sinks, d ** -0.5, DT[dt])["o"]
            check("token", o1[b], ref[0][-1], ref[1][-1])
    for b, n in enumerate(lens):
        check("prompt", o[cu[b]:cu[b + 1]], *attend(*(y[:n] for y in full[b]), window, sinks, d ** -0.5, DT[dt])["o"])


def test_decode_captured():
    """A captured step replayed while lengths advance between the replays, against eager steps; bitwise."""
    announce("attn decode graph")
    B, Hq, Hkv, d, page, L = 2, 8, 2, 128, 16, 3000
    c = Cache("bf16", [L, 20], [8, 8], Hkv, d, page)
    kp, vp, table, lens = c.device()
    ke, ve, le = kp.clone(), vp.clone(), lens.clone()
    q, k, v = make(1, "bf16", B, Hq, d).cuda(), make(2, "bf16", B, Hkv, d).cuda(), make(3, "bf16", B, Hkv, d).cuda()
    o, oe = torch.empty_like(q), torch.empty_like(q)
    n = gdr.gdr_attn_decode_workspace_bytes(q.dtype, B, Hq, Hkv, d, page, table.shape[1])
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # position lens is written again by the first replay
        gdr.gdr_attn_decode(q, k, v, kp, vp, table, lens, o, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr.gdr_attn_decode(q, k, v, kp, vp, table, lens, o, workspace=ws)
    for t in range(4):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        gdr.gdr_attn_decode(q, k, v, ke, ve, table, le, oe)
        assert torch.equal(o, oe) and same(kp, ke) and same(vp, ve)
        lens += 1
        le += 1
