"""The operators around the attention layers together, as a layer uses them: serving steps (page plan, norm and rotation,
append, read, prefill, decode), eager and captured, on other streams, over caches beyond 4 GiB; and a training step.

Each stage is checked with its own bound on the inputs it had: what the stage before wrote."""
import math

import pytest
import torch

import gated_delta_rule_08_amd as gdr
from attn_ref import attend as attend_full
from attn_ref import check
from gpu_util import announce, ensure_built
from mx4_ref import Mx4Cache, attend, quantise, value
from test_gpu_attn_rope import reference as rope_reference

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(seed, dt, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dt)


def ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


class Server:
    """A layer's serving state on the GPU: page table, free pages, lengths, a 4-bit cache."""

    def __init__(self, dt, N, Hq, Hkv, d, page, width, pages, window=0, sinks=0):
        self.dt, self.N, self.Hq, self.Hkv, self.d, self.page = DT[dt], N, Hq, Hkv, d, page
        self.window, self.sinks = window, sinks
        u8 = lambda *s: torch.full(s, 255, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.cache = u8(pages, Hkv, page, d // 2), u8(pages, Hkv, page, d // 32), u8(pages, Hkv, page // 32, d, 16), u8(pages, Hkv, page, d // 32)
        self.table = torch.full((N, width), -1, dtype=torch.int32, device="cuda")
        self.free, self.n_free = ints(torch.randperm(pages, generator=torch.Generator().manual_seed(1)).tolist()), ints([pages])
        self.lengths, self.before = ints([0] * N), ints([0] * N)
        self.cu, self.added = ints([0] * (N + 1)), ints([0] * N)
        self.freq = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().cuda()
        self.w_q, self.w_k = (1 + 0.2 * make(s, torch.float32, d) for s in (91, 92))
        self.wq, self.wk = self.w_q.cuda(), self.w_k.cuda()

    def plan(self, add, slots=None):
        self.before.copy_(self.lengths)
        gdr.gdr_attn_plan_pages(self.lengths, add, self.free, self.n_free, self.table, self.page, self.cu, self.added, self.lengths,
                                self.n_free, slots)

    def rotate_and_append(self, qkv, positions, q, k, v):
        x = qkv.view(-1, self.Hq + 2 * self.Hkv, self.d)
        gdr.gdr_attn_norm_rope(x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], positions, self.freq, q, k, w_q=self.wq, w_k=self.wk)
        v.copy_(x[:, self.Hq + self.Hkv:])
        gdr.gdr_attn_append_mx4(k, v, self.cu, self.before, *self.cache, self.table)


@pytest.mark.parametrize("dt,Hq,Hkv,d,page,window,sinks", [
    ("f32", 4, 2, 64, 32, 0, 0), ("bf16", 8, 2, 128, 64, 0, 0), ("bf16", 6, 3, 64, 32, 50, 3), ("bf16", 5, 5, 128, 128, 0, 0)])
def test_serving_steps(dt, Hq, Hkv, d, page, window, sinks):
    """Prompts of uneven lengths, their next parts on the context read back, then single tokens and drafts."""
    announce("serving steps %s" % ((dt, Hq, Hkv, d, page, window, sinks),))
    N, T = 4, DT[dt]
    s = Server(dt, N, Hq, Hkv, d, page, 12 * 32 // page + 1, 60, window, sinks)
    held = [0] * N
    seen = [(torch.zeros(0, Hkv, d).double(), torch.zeros(0, Hkv, d).double()) for _ in range(N)]  # values in the cache
    for step, add in enumerate([[70, 1, 33, 64], [31, 40, 0, 5], [1, 1, 1, 1], [3, 3, 3, 3], [1, 0, 1, 1]]):
        total = sum(add)
        slots = torch.full((total + 3,), -9, dtype=torch.int32, device="cuda")
        s.plan(ints(add), slots)
        qkv = make(10 + step, T, total, (Hq + 2 * Hkv) * d)
        pos = torch.tensor([h + i for h, a in zip(held, add) for i in range(a)], dtype=torch.int32)
        q, k, v = (torch.full((total, h, d), 7.0, dtype=T, device="cuda") for h in (Hq, Hkv, Hkv))
        s.rotate_and_append(qkv.cuda(), pos.cuda(), q, k, v)
        torch.cuda.synchronize()
        x = qkv.view(total, -1, d)
        t = pos[:, None].double() * s.freq.cpu().double()
        check("q", q, *rope_reference(x[:, :Hq], s.w_q, t, False, True, 1e-6)["out"])
        check("k", k, *rope_reference(x[:, Hq:Hq + Hkv], s.w_k, t, False, True, 1e-6)["out"])
        # the plan: every token has a place of its own, where the table has its page
        table, at = s.table.cpu(), 0
        place = [int(table[n, (held[n] + i) // page]) * page + (held[n] + i) % page for n in range(N) for i in range(add[n])]
        assert slots[:total].tolist() == place and (slots[total:] == -9).all()
        assert s.lengths.tolist() == [h + a for h, a in zip(held, add)]
        used = table[table >= 0]
        assert len(set(used.tolist())) == len(used) == 60 - int(s.n_free)
        for n, a in enumerate(add):
            new = [value(*quantise(y[at:at + a].float().cpu())) for y in (k, v)]
            seen[n] = tuple(torch.cat([old, y]) for old, y in zip(seen[n], new))
            at += a
        held = [h + a for h, a in zip(held, add)]
        if step < 2:  # the prompts' parts attend to the context read back
            cu_k = ints([sum(held[:n]) for n in range(N + 1)])
            ko, vo = (torch.zeros(sum(held), Hkv, d, dtype=T, device="cuda") for _ in range(2))
            gdr.gdr_attn_read_mx4(*s.cache, s.table, cu_k, ko, vo)
            o = torch.full_like(q, 7.0)
            gdr.gdr_attn_prefill_varlen(q, ko, vo, s.cu, cu_k, o, window=window, sinks=sinks)
            torch.cuda.synchronize()
            at = 0
            for n, a in enumerate(add):
                lo = sum(held[:n])
                assert torch.equal(ko[lo:lo + held[n]].double().cpu(), seen[n][0])
                assert torch.equal(vo[lo:lo + held[n]].double().cpu(), seen[n][1])
                ref = attend_full(q[at:at + a].cpu(), seen[n][0], seen[n][1], window, sinks, d ** -0.5, T)
                check("prefill[%d]" % n, o[at:at + a], *ref["o"])
                at += a
        else:  # the same number of tokens each, where one adds none its last is asked again
            Tq = max(add)
            at = [sum(add[:n]) for n in range(N)]
            qd = torch.stack([q[at[n]:at[n] + a] if a else q[:Tq] for n, a in enumerate(add)])
            o = torch.full_like(qd, 7.0)
            gdr.gdr_attn_decode_mx4(qd, *s.cache, s.table, s.lengths, o, window=window, sinks=sinks)
            torch.cuda.synchronize()
            for n in range(N):
                ref, bound = attend(qd[n].cpu(), *seen[n], held[n], window, sinks, d ** -0.5, T)
                check("decode[%d]" % n, o[n], ref, bound)


def test_captured_steps():
    """A decode step captured whole and replayed, the plan's state advancing in place, against the same steps run eagerly;
    other work and synchronizations lie between the replays, and two graphs are kept of the same step."""
    announce("captured serving steps")
    N, Hq, Hkv, d, page = 5, 8, 2, 128, 32
    prompt = [40, 1, 70, 33, 600]

    def server():
        s = Server("bf16", N, Hq, Hkv, d, page, 24, 120)
        s.plan(ints(prompt))
        total = sum(prompt)
        q, k, v = (torch.empty(total, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
        pos = torch.tensor([i for n in prompt for i in range(n)], dtype=torch.int32, device="cuda")
        s.rotate_and_append(make(3, torch.bfloat16, total, (Hq + 2 * Hkv) * d).cuda(), pos, q, k, v)
        s.qkv = torch.zeros(N, (Hq + 2 * Hkv) * d, dtype=torch.bfloat16, device="cuda")
        s.one = ints([1] * N)
        s.q, s.k, s.v, s.o = (torch.empty(N, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv, Hq))
        s.slots = torch.zeros(N, dtype=torch.int32, device="cuda")
        return s

    def step(s):
        s.plan(s.one, s.slots)
        s.rotate_and_append(s.qkv, s.before, s.q, s.k, s.v)
        gdr.gdr_attn_decode_mx4(s.q, *s.cache, s.table, s.lengths, s.o)

    eager, a = server(), server()
    assert gdr.gdr_attn_decode_mx4_workspace_bytes(torch.bfloat16, N, 1, Hq, Hkv, d, page, 24) > 0
    keep = [x.clone() for x in (*a.cache, a.table, a.lengths, a.n_free)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            step(a)
    for x, y in zip((*a.cache, a.table, a.lengths, a.n_free), keep):  # as before the warm-up
        x.copy_(y)
    noise = torch.randn(512, 512, device="cuda")
    for i in range(40):  # crosses page ends
        x = make(100 + i, torch.bfloat16, N, (Hq + 2 * Hkv) * d).cuda()
        for s in (eager, a):
            s.qkv.copy_(x)
        step(eager)
        graphs[i % 2].replay()
        if i % 3 == 0:
            torch.cuda.synchronize()
        noise = noise @ noise / 30
        for name in ("o", "q", "k", "lengths", "n_free", "table", "slots", "cu", "added"):
            assert torch.equal(getattr(eager, name), getattr(a, name)), (i, name)
        for x, y in zip(eager.cache, a.cache):
            assert torch.equal(x, y), i


def test_captured_training():
    """Forward and backward of the rotation in a graph, its workspace made inside, against eager results."""
    announce("captured rotation")
    T, Hq, Hkv, d = 300, 4, 2, 64
    q, k, gq, gk = (torch.zeros(T, h, d, device="cuda") for h in (Hq, Hkv, Hq, Hkv))
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), (0.5 ** torch.arange(32.0)).cuda()
    w = torch.ones(d, device="cuda")
    outs = [torch.empty_like(x) for x in (q, k, q, k, w, w)]

    def run(o):
        gdr.gdr_attn_norm_rope(q, k, pos, freq, o[0], o[1], w_q=w, w_k=w)
        gdr.gdr_attn_norm_rope_backward(q, k, pos, freq, gq, gk, o[2], o[3], w_q=w, w_k=w, grad_w_q=o[4], grad_w_k=o[5])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(outs)
    for i in range(5):
        for j, x in enumerate((q, k, gq, gk)):
            x.copy_(make(10 * i + j, torch.float32, *x.shape))
        graph.replay()
        want = [torch.empty_like(x) for x in outs]
        run(want)
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_another_stream(handle):
    """Every call on a stream that is not the current one, behind the work there that makes its inputs."""
    announce("serving on another stream %s" % handle)
    N, Hq, Hkv, d, page, n = 3, 4, 2, 64, 32, 700
    work = torch.randn(4096, 4096, device="cuda")
    out = torch.empty_like(work)
    torch.mm(work, work, out=out)
    s = torch.cuda.Stream()
    to = s.cuda_stream if handle else s
    results = []
    for late in (False, True):
        a = Server("bf16", N, Hq, Hkv, d, page, 24, 80)
        total = N * n
        qkv = make(5, torch.bfloat16, total, Hq + 2 * Hkv, d).cuda()
        pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(N)
        add, x, p = ints([0] * N), torch.zeros_like(qkv), torch.zeros_like(pos)
        q, k, v = (torch.zeros(total, h, d, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
        kr, vr, o = torch.zeros_like(k), torch.zeros_like(v), torch.zeros(N, Hq, d, dtype=torch.bfloat16, device="cuda")
        gq, gk, dq, dk, dw = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(q), torch.zeros_like(k), torch.zeros(d, device="cuda")
        grads = make(6, torch.bfloat16, total, Hq, d).cuda(), make(7, torch.bfloat16, total, Hkv, d).cuda()
        want = ints([n] * N)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            if late:
                for _ in range(20):
                    torch.mm(work, work, out=out)
            add.copy_(want), x.copy_(qkv), p.copy_(pos), gq.copy_(grads[0]), gk.copy_(grads[1])
        gdr.gdr_attn_plan_pages(a.lengths, add, a.free, a.n_free, a.table, page, a.cu, a.added, a.lengths, a.n_free, stream=to)
        gdr.gdr_attn_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], p, a.freq, q, k, stream=to)
        gdr.gdr_attn_append_mx4(k, k, a.cu, a.before, *a.cache, a.table, stream=to)
        gdr.gdr_attn_read_mx4(*a.cache, a.table, a.cu, kr, vr, stream=to)
        with torch.cuda.stream(s):
            last = q.view(N, n, Hq, d)[:, -1].contiguous()
        gdr.gdr_attn_decode_mx4(last, *a.cache, a.table, a.lengths, o, stream=to)
        gdr.gdr_attn_norm_rope_backward(x[:, :Hq], x[:, Hq:Hq + Hkv], p, a.freq, gq, gk, dq, dk, w_q=a.wq, grad_w_q=dw, stream=to)
        s.synchronize()
        results.append((a.table, a.lengths, q, k, kr, vr, o, dq, dk, dw))
    for i, (x, y) in enumerate(zip(*results)):
        assert torch.equal(x, y), i
    assert float(results[0][6].abs().max()) > 0 and float(results[0][9].abs().max()) > 0


def test_two_streams_at_once():
    """Calls in flight on two streams, each with buffers of its own, give what they give one after another."""
    announce("serving on two streams")
    Hq, Hkv, d, page, n = 8, 2, 128, 64, 3000
    cases = []
    for i in range(2):
        c = Mx4Cache([n, n // 3 + i], [0, 0], Hkv, d, page, seed=i)
        c.kc.random_(0, 16, generator=torch.Generator().manual_seed(i)), c.vc.random_(0, 16, generator=torch.Generator().manual_seed(9 + i))
        c.ks.fill_(126 + i), c.vs.fill_(125)
        cases.append((make(20 + i, torch.bfloat16, 2, Hq, d).cuda(), c.device(), ints(c.lengths)))
    want = []
    for q, cache, lengths in cases:
        o = torch.empty_like(q)
        gdr.gdr_attn_decode_mx4(q, *cache, lengths, o)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[torch.empty_like(q) for _ in range(20)] for q, _, _ in cases]
    for r in range(20):
        for i, (q, cache, lengths) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                gdr.gdr_attn_decode_mx4(q, *cache, lengths, got[i][r])
    torch.cuda.synchronize()
    for i in range(2):
        for r in range(20):
            assert torch.equal(got[i][r], want[i]), (i, r)


def test_caches_beyond_4_gib():
    """Pages whose bytes lie beyond 2^32 (codes and dense rows alike): append, read and decode there."""
    announce("mx4 beyond 4 GiB")
    Hkv, d, page, pages, n = 8, 128, 256, 36000, 700
    kc = torch.zeros(pages, Hkv, page, d // 2, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(pages, Hkv, page // 32, d, 16, dtype=torch.uint8, device="cuda")
    ks, vs = (torch.ones(pages, Hkv, page, d // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    assert kc.numel() > 2 ** 32
    table = ints([[pages - 1, pages - 2, pages - 3, 5], [17, pages // 2, pages - 9, pages - 5]])
    k, v, q = make(1, torch.bfloat16, 2 * n, Hkv, d), make(2, torch.bfloat16, 2 * n, Hkv, d), make(3, torch.bfloat16, 2, Hkv, d)
    cu = ints([0, n, 2 * n])
    gdr.gdr_attn_append_mx4(k.cuda(), v.cuda(), cu, ints([0, 0]), kc, ks, vc, vs, table)
    ko, vo = (torch.zeros(2 * n, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gdr.gdr_attn_read_mx4(kc, ks, vc, vs, table, cu, ko, vo)
    o = torch.zeros(2, Hkv, d, dtype=torch.bfloat16, device="cuda")
    gdr.gdr_attn_decode_mx4(q.cuda(), kc, ks, vc, vs, table, ints([n, n]), o)
    torch.cuda.synchronize()
    rk, rv = (value(*quantise(x.float())) for x in (k, v))
    assert torch.equal(ko.double().cpu(), rk) and torch.equal(vo.double().cpu(), rv)
    for b in range(2):
        ref, bound = attend(q[b:b + 1], rk[b * n:(b + 1) * n], rv[b * n:(b + 1) * n], n, 0, 0, d ** -0.5, torch.bfloat16)
        check("o[%d]" % b, o[b:b + 1], ref, bound)


def test_rotation_beyond_4_gib():
    """Tokens whose rows lie beyond 2^32 bytes, in a fused projection and in the outputs."""
    announce("rope beyond 4 GiB")
    T, Hq, Hkv, d = 70000, 256, 4, 128
    qkv = torch.zeros(T, Hq + Hkv, d, dtype=torch.bfloat16, device="cuda")
    tail = make(1, torch.bfloat16, 50, Hq + Hkv, d)
    qkv[-50:] = tail.cuda()
    qkv[:50] = tail.cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    pos[-50:] = pos[:50]
    freq = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float().cuda()
    q, k = qkv[:, :Hq], qkv[:, Hq:]
    qo, ko = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, Hkv, d, dtype=torch.bfloat16, device="cuda")
    gdr.gdr_attn_norm_rope(q, k, pos, freq, qo, ko)
    wide = torch.zeros_like(qkv)
    gdr.gdr_attn_norm_rope_backward(q, k, pos, freq, qo, ko, wide[:, :Hq], wide[:, Hq:])
    torch.cuda.synchronize()
    assert qo.numel() * 2 > 2 ** 32
    for x in (qo, ko, wide):
        assert torch.equal(x[:50], x[-50:])
    t = pos[:50, None].double().cpu() * freq.cpu().double()
    ref = rope_reference(tail[:, :Hq], None, t, False, True, 1e-6, qo[:50].cpu())
    check("q", qo[-50:], *ref["out"])
    check("grad_q", wide[-50:, :Hq], *ref["grad"])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_training_step(dt):
    """Norm, rotation and attention forward, then back to the projection and the weights, stage by stage."""
    announce("training step %s" % dt)
    B, T, Hq, Hkv, d, window, sinks = 1, 90, 4, 2, 64, 40, 2
    typ = DT[dt]
    qkv = make(1, typ, B, T, Hq + 2 * Hkv, d)
    dev = qkv.cuda()
    q, k = dev[:, :, :Hq], dev[:, :, Hq:Hq + Hkv]
    v = dev[:, :, Hq + Hkv:].contiguous()
    pos = torch.arange(T, dtype=torch.int32).reshape(B, T)
    freq = (10000.0 ** (-torch.arange(0, d, 2).double() / d)).float()
    wq, wk = 1 + 0.3 * make(2, torch.float32, d), 1 + 0.3 * make(3, torch.float32, d)
    go = make(4, typ, B, T, Hq, d)
    qr, kr = (torch.empty(B, T, h, d, dtype=typ, device="cuda") for h in (Hq, Hkv))
    gdr.gdr_attn_norm_rope(q, k, pos.cuda(), freq.cuda(), qr, kr, w_q=wq.cuda(), w_k=wk.cuda())
    o, lse = torch.empty_like(qr), torch.empty(B, T, Hq, device="cuda")
    gdr.gdr_attn_prefill(qr, kr, v, o, lse, window=window, sinks=sinks)
    dqr, dkr, dv = torch.empty_like(qr), torch.empty_like(kr), torch.empty_like(v)
    gdr.gdr_attn_backward(qr, kr, v, o, lse, go.cuda(), dqr, dkr, dv, window=window, sinks=sinks)
    grad = torch.full_like(dev, 7.0)
    dwq, dwk = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    gdr.gdr_attn_norm_rope_backward(q, k, pos.cuda(), freq.cuda(), dqr, dkr, grad[:, :, :Hq], grad[:, :, Hq:Hq + Hkv], w_q=wq.cuda(),
                                    w_k=wk.cuda(), grad_w_q=dwq, grad_w_k=dwk)
    grad[:, :, Hq + Hkv:] = dv
    torch.cuda.synchronize()
    att = attend_full(qr[0].cpu(), kr[0].cpu(), v[0].cpu(), window, sinks, d ** -0.5, typ, go[0])
    for name, x in (("o", o), ("grad_q", dqr), ("grad_k", dkr), ("grad_v", dv)):
        check(name, x[0], *att[name])
    t = pos[..., None].double() * freq.double()
    for name, x, w, out, g, dx, dw in (("q", qkv[:, :, :Hq], wq, qr, dqr, grad[:, :, :Hq], dwq),
                                       ("k", qkv[:, :, Hq:Hq + Hkv], wk, kr, dkr, grad[:, :, Hq:Hq + Hkv], dwk)):
        ref = rope_reference(x, w, t, False, True, 1e-6, g.cpu())
        check(name, out, *ref["out"])
        check("grad " + name, dx, *ref["grad"])
        check("grad_w " + name, dw, *ref["grad_w"])


def test_refusals_on_the_device():
    """Refused by the library, not by the binding: nothing is written."""
    announce("serving refusals")
    q = torch.ones(4, 2, 64, device="cuda")
    pos, freq = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(4, device="cuda")
    out = torch.full_like(q, 7.0)
    with pytest.raises(gdr.GdrError):
        gdr.gdr_attn_norm_rope(q, q, pos, freq, out, out.clone())  # 8 rotated channels
    wide = torch.ones(4, 4, 64, device="cuda")
    with pytest.raises(gdr.GdrError):  # in place where the tokens lie apart
        gdr._check(gdr.load_library().gdr_attn_norm_rope(0, 2, 4, 2, 0, 64, 0, 0.0, 256, 0, wide.data_ptr(), None, None, None, None,
                                                         None, wide.data_ptr(), None, None))
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    cache = u8(3, 2, 16, 32), u8(3, 2, 16, 2), u8(3, 2, 0, 64, 16), u8(3, 2, 16, 2)
    with pytest.raises(gdr.GdrError):  # pages of 16
        gdr.gdr_attn_decode_mx4(q, *cache, torch.zeros(4, 3, dtype=torch.int32, device="cuda"), pos, out)
    with pytest.raises(ValueError, match="one device|GPU"):
        gdr.gdr_attn_decode_mx4(q.cpu(), *cache, torch.zeros(4, 3, dtype=torch.int32, device="cuda"), pos, out)
    torch.cuda.synchronize()
    assert (out == 7).all() and math.isclose(float(wide.sum()), wide.numel())
