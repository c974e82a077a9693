"""Windowed attention prefill (dense and packed) and its backward against the float64 definition."""
import itertools
import math

import pytest
import torch

import gated_delta_rule_08_amd as gdr
from attn_ref import attend, check, visible
from gpu_util import announce, ensure_built

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(seed, dt, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dt])


def forward(q, k, v, window, sinks, scale):
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    gdr.gdr_attn_prefill(q, k, v, o, lse, window=window, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    return o, lse


# B, Tq, Tk, Hq, Hkv, d, window, sinks: one token, around the 32-, 64- and 128-row tiles, grouped heads (also 3 and 5,
# so that a tile starts inside a query's group), windows that end inside a tile, sinks around a tile, queries at the end
# of longer keys, and more queries than keys (empty rows)
CASES = [
    (1, 1, 1, 1, 1, 64, 0, 0),
    (2, 2, 2, 2, 1, 128, 0, 0),
    (1, 31, 31, 3, 1, 64, 0, 0),
    (2, 33, 33, 4, 4, 128, 0, 0),
    (1, 64, 64, 8, 2, 128, 0, 0),
    (1, 65, 65, 5, 1, 64, 1, 0),
    (1, 130, 130, 4, 2, 128, 40, 0),
    (1, 130, 130, 4, 2, 64, 64, 4),
    (1, 257, 257, 6, 2, 128, 33, 70),
    (2, 200, 200, 2, 2, 64, 1, 1),
    (1, 300, 300, 8, 1, 128, 100, 3),
    (8, 70, 70, 4, 2, 64, 32, 2),
    (1, 1, 300, 8, 2, 128, 0, 0),
    (1, 17, 400, 4, 1, 64, 90, 5),
    (2, 100, 163, 6, 3, 128, 0, 0),
    (1, 50, 20, 4, 2, 64, 0, 0),
    (1, 150, 90, 2, 1, 128, 30, 2),
    (1, 20, 0, 2, 1, 64, 0, 0),
    (1, 97, 97, 2, 1, 128, 1000, 4),
    (1, 700, 700, 2, 1, 64, 128, 150),
    (1, 640, 640, 8, 2, 64, 50, 4),
    (1, 40, 40, 40, 1, 128, 7, 1),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_forward_and_backward(case, dt):
    B, Tq, Tk, Hq, Hkv, d, window, sinks = case
    announce("attn prefill + backward %s %s" % (dt, case))
    q, k, v, go = make(1, dt, B, Tq, Hq, d), make(2, dt, B, Tk, Hkv, d), make(3, dt, B, Tk, Hkv, d), make(4, dt, B, Tq, Hq, d)
    scale = d ** -0.5
    o, lse = forward(q, k, v, window, sinks, scale)
    dq, dk, dv = (torch.full_like(x, 7.0).cuda() for x in (q, k, v))
    gdr.gdr_attn_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, go.cuda(), dq, dk, dv, window=window, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    for b in range(B):
        ref = attend(q[b], k[b], v[b], window, sinks, scale, DT[dt], go[b])
        for name, got in (("o", o), ("lse", lse), ("grad_q", dq), ("grad_k", dk), ("grad_v", dv)):
            check(name, got[b], *ref[name])


# Enough heads that every workgroup takes 128 rows or keys: full causal (the first keys' row lists sliced or not) and
# windows (sink keys' rows in segments), head counts that are and are not a multiple of 8, groups that do and do not
# divide 32, one and several rounds of workgroups
MANY = [
    (33, 150, 150, 16, 8, 64, 0, 0),
    (33, 150, 150, 16, 8, 128, 40, 3),
    (24, 300, 300, 12, 12, 128, 0, 0),
    (40, 97, 160, 24, 8, 128, 64, 70),
    (26, 129, 129, 15, 5, 64, 100, 2),
    (300, 33, 33, 1, 1, 64, 0, 0),
    (260, 40, 20, 2, 1, 128, 0, 0),
    (260, 64, 200, 2, 1, 64, 130, 131),
    (8, 700, 700, 32, 4, 64, 0, 0),
    (64, 260, 260, 7, 7, 128, 33, 1),
    # few key blocks under a window: the sinks' blocks cut into many slices, the others into one, or two
    (1, 3000, 3000, 1, 1, 64, 20, 4),
    (1, 2500, 2600, 2, 1, 128, 200, 150),
    (2, 900, 900, 12, 2, 64, 300, 40),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "x".join(map(str, c)))
def test_many_heads(case, dt):
    B, Tq, Tk, Hq, Hkv, d, window, sinks = case
    announce("attn many heads %s %s" % (dt, case))
    q, k, v, go = make(1, dt, B, Tq, Hq, d), make(2, dt, B, Tk, Hkv, d), make(3, dt, B, Tk, Hkv, d), make(4, dt, B, Tq, Hq, d)
    o, lse = forward(q, k, v, window, sinks, 0.1)
    dq, dk, dv = (torch.full_like(x, 7.0).cuda() for x in (q, k, v))
    gdr.gdr_attn_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, go.cuda(), dq, dk, dv, window=window, sinks=sinks, scale=0.1)
    torch.cuda.synchronize()
    for t in (o, lse, dq, dk, dv):  # every row was written
        assert not (t.reshape(-1, t.shape[-1]) == 7).all(-1).any()
    for b in sorted({0, min(1, B - 1), B // 2, B - 1}):
        ref = attend(q[b], k[b], v[b], window, sinks, 0.1, DT[dt], go[b])
        for name, got in (("o", o), ("lse", lse), ("grad_q", dq), ("grad_k", dk), ("grad_v", dv)):
            check(name, got[b], *ref[name])


def test_tensors_beyond_4_gib():
    """Keys and values of 4.7 GB each, the queries at their end: sinks at the front, the window at the far end."""
    announce("attn beyond 4 GiB")
    Tk, Tq, H, d, window, sinks = 71000, 40, 256, 128, 100, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros(1, Tk, H, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    seen = list(range(sinks)) + list(range(Tk - Tq - window, Tk))
    for t in (k, v):
        t[:, :sinks] = torch.randn(1, sinks, H, d, generator=g, device="cuda")
        t[:, Tk - Tq - window:] = torch.randn(1, Tq + window, H, d, generator=g, device="cuda")
        t[:, sinks + 1] = float("nan")  # seen by no query
    q, go = (torch.randn(1, Tq, H, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    o, lse = torch.empty_like(q), torch.empty(1, Tq, H, device="cuda")
    gdr.gdr_attn_prefill(q, k, v, o, lse, window=window, sinks=sinks)
    dq, dk, dv = torch.empty_like(q), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    gdr.gdr_attn_backward(q, k, v, o, lse, go, dq, dk, dv, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert not dk[:, sinks:Tk - Tq - window].any() and not dv[:, sinks:Tk - Tq - window].any()
    for h in (0, 1, 77, 255):
        # the keys in between are never seen, so the reference may leave them out
        x = [t[0, seen][:, h:h + 1].cpu() for t in (k, v)]
        ref = attend(q[0, :, h:h + 1].cpu(), *x, window, sinks, d ** -0.5, torch.bfloat16, go[0, :, h:h + 1].cpu())
        for name, got in (("o", o[0]), ("lse", lse[0]), ("grad_q", dq[0])):
            check(name, got[:, h:h + 1], *ref[name])
        for name, got in (("grad_k", dk), ("grad_v", dv)):
            check(name, got[0, seen][:, h:h + 1], *ref[name])


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scale(scale):
    announce("attn scale %g" % scale)
    q, k, v, go = (make(i, "f32", 1, 90, 2, 64) for i in range(4))
    o, lse = forward(q, k, v, 40, 2, scale)
    dq, dk, dv = (torch.empty_like(x).cuda() for x in (q, k, v))
    gdr.gdr_attn_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, go.cuda(), dq, dk, dv, window=40, sinks=2, scale=scale)
    ref = attend(q[0], k[0], v[0], 40, 2, scale, torch.float32, go[0])
    for name, got in (("o", o), ("lse", lse), ("grad_q", dq), ("grad_k", dk), ("grad_v", dv)):
        check(name, got[0], *ref[name])


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 64)])
def test_large_scores(dt, d):
    """Scores of several hundred: the running maximum keeps every exponent in range."""
    announce("attn large scores %s" % dt)
    q, k, v = make(1, dt, 1, 200, 2, d) * 8, make(2, dt, 1, 200, 2, d) * 8, make(3, dt, 1, 200, 2, d)
    o, lse = forward(q, k, v, 0, 0, 1.0)
    ref = attend(q[0], k[0], v[0], 0, 0, 1.0, DT[dt])
    check("o", o[0], *ref["o"])
    check("lse", lse[0], *ref["lse"])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("B,d", [(1, 64), (140, 64), (1, 128), (140, 128)])
def test_non_finite_values_stay_with_the_rows_that_see_them(dt, what, B, d):
    """A non-finite key, value, query or gradient row reaches exactly the outputs its definition gives it."""
    announce("attn non-finite %s %s %d %d" % (dt, what, B, d))
    T, Hq, Hkv, window, sinks, at = 150, 4, 2, 30, 2, 77
    x = float(what)
    q, k, v, go = make(1, dt, B, T, Hq, d), make(2, dt, B, T, Hkv, d), make(3, dt, B, T, Hkv, d), make(4, dt, B, T, Hq, d)
    o0, lse0 = forward(q, k, v, window, sinks, 0.125)
    keys = [i for i in range(T) if at <= i < at + window]  # the queries that see key `at`
    rest = [i for i in range(T) if i not in keys]
    for t in (k, v):
        bad = t.clone()
        bad[:, at, 1] = x
        o, lse = forward(q, bad if t is k else k, bad if t is v else v, window, sinks, 0.125)
        assert torch.isfinite(o[:, rest].float()).all() and torch.isfinite(o[:, :, :2].float()).all()
        tol = 2 ** -7 if dt == "bf16" else 1e-5  # a wave that starts again rounds its weights otherwise
        assert torch.allclose(o[:, rest].float(), o0[:, rest].float(), rtol=tol, atol=tol)
        assert torch.allclose(lse[:, rest], lse0[:, rest], rtol=1e-5, atol=1e-5)
        if t is v or what == "nan":
            assert not torch.isfinite(o[:, keys, 2:].float()).any()
    bad = q.clone()
    bad[:, at, 2] = x
    o, lse = forward(bad, k, v, window, sinks, 0.125)
    mine = torch.zeros(T, Hq, dtype=torch.bool)
    mine[at, 2] = True
    assert torch.isfinite(o[0][~mine].float()).all() and torch.isnan(o[0][mine].float()).all()
    # gradients: a non-finite grad_o row reaches its own query and the keys it sees
    badg = go.clone()
    badg[:, at, 2] = x
    dq, dk, dv = (torch.empty_like(t).cuda() for t in (q, k, v))
    gdr.gdr_attn_backward(q.cuda(), k.cuda(), v.cuda(), o0, lse0, badg.cuda(), dq, dk, dv, window=window, sinks=sinks, scale=0.125)
    ref = attend(q[0], k[0], v[0], window, sinks, 0.125, DT[dt], go[0])
    seen = [j for j in range(T) if j <= at and (j > at - window or j < sinks)]
    hidden = [j for j in range(T) if j not in seen]
    assert not torch.isfinite(dv[0, seen, 1].float()).any()
    for name, got in (("grad_k", dk), ("grad_v", dv)):
        check(name, got[0, hidden], ref[name][0][hidden], ref[name][1][hidden])
        check(name, got[0, :, :1], ref[name][0][:, :1], ref[name][1][:, :1])
    check("grad_q", dq[0][~mine], ref["grad_q"][0][~mine], ref["grad_q"][1][~mine])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,d", [(1, 64), (140, 128)])
def test_single_non_finite_elements(dt, B, d):
    """Infinities of both signs and NaN in single elements of v and grad_o: every sum over visible pairs has the value
    float64 gives it, element by element (an infinity, a NaN, or a number within its bound)."""
    announce("attn single non-finite elements %s %d %d" % (dt, B, d))
    T, window, sinks, scale = 150, 30, 2, 0.125
    x = [make(i, dt, B, T, 1, d) for i in range(4)]
    q, k, v, go = x
    clean = [t[0, :, 0].double() for t in x]
    spots = [(1, 3, "inf"), (70, 4, "inf"), (75, 4, "-inf"), (75, 5, "nan"), (90, 6, "-inf"), (149, 7, "nan"), (20, 8, "inf")]
    bad = v.clone()
    for j, ch, what in spots:
        bad[:, j, 0, ch] = float(what)

    def sums(see, w, t):  # sum over the visible pairs of w_ij t_j, hidden ones left out
        return torch.stack([(w[i][see[i]].unsqueeze(-1) * t[see[i]]).sum(0) for i in range(see.shape[0])])

    def compare(name, got, ref, bound):
        got, ref = got[:, 0].double().cpu(), ref
        odd = ~torch.isfinite(ref)
        assert torch.equal(torch.isnan(got), torch.isnan(ref)) and torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)]), name
        assert ((got - ref).masked_fill(odd, 0).abs() <= bound.masked_fill(odd, 1)).all(), name

    see = visible(T, T, window, sinks)
    ref = attend(q[0], k[0], v[0], window, sinks, scale, DT[dt], go[0])
    p = torch.softmax((clean[0] @ clean[1].t() * scale).masked_fill(~see, -math.inf), -1)
    o0, lse = forward(q, k, v, window, sinks, scale)
    o, lse1 = forward(q, k, bad, window, sinks, scale)
    check("lse", lse1[0], *ref["lse"])
    # a sum that has lost no terms has the clean sum's bound; the other channels are the clean ones
    compare("o", o[0], sums(see, p, bad[0, :, 0].double()), ref["o"][1][:, 0])
    badg = go.clone()
    for j, ch, what in spots:
        badg[:, j, 0, ch] = float(what)
    dq, dk, dv = (torch.empty_like(t).cuda() for t in (q, k, v))
    gdr.gdr_attn_backward(q.cuda(), k.cuda(), v.cuda(), o0, lse, badg.cuda(), dq, dk, dv, window=window, sinks=sinks, scale=scale)
    compare("grad_v", dv[0], sums(see.t(), p.t(), badg[0, :, 0].double()), ref["grad_v"][1][:, 0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_packed_sequences(dt):
    """Lengths 0, 1 and around the tiles, each with keys before its queries; rows of no sequence stay."""
    announce("attn packed %s" % dt)
    lens, past, Hq, Hkv, d, window, sinks = [5, 0, 1, 64, 129, 32, 200], [0, 3, 70, 0, 9, 200, 1], 6, 2, 64, 50, 3
    cu_q = [2] + [2 + n for n in itertools.accumulate(lens)]
    cu_k = [1] + [1 + n for n in itertools.accumulate(a + b for a, b in zip(lens, past))]
    q = make(1, dt, cu_q[-1] + 5, Hq, d)
    k, v = make(2, dt, cu_k[-1] + 4, Hkv, d), make(3, dt, cu_k[-1] + 4, Hkv, d)
    k[0] = v[0] = k[-4:] = v[-4:] = float("nan")  # keys of no sequence
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for bound in (None, 200, 1000):
        o = torch.full_like(q, 7.0).cuda()
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        gdr.gdr_attn_prefill_varlen(q.cuda(), k.cuda(), v.cuda(), dev(cu_q), dev(cu_k), o, lse, max_seqlen_q=bound,
                                    window=window, sinks=sinks)
        assert (o[:2] == 7).all() and (o[-5:] == 7).all() and (lse[:2] == 7).all() and (lse[-5:] == 7).all()
        for n in range(len(lens)):
            a, b, c, e = cu_q[n], cu_q[n + 1], cu_k[n], cu_k[n + 1]
            ref = attend(q[a:b], k[c:e], v[c:e], window, sinks, d ** -0.5, DT[dt])
            check("o", o[a:b], *ref["o"])
            check("lse", lse[a:b], *ref["lse"])


def test_packed_sequence_with_bad_offsets_is_skipped():
    announce("attn packed, bad offsets")
    q, k = make(1, "bf16", 60, 2, 64).cuda(), make(2, "bf16", 60, 1, 64).cuda()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good = torch.empty_like(q)
    gdr.gdr_attn_prefill_varlen(q, k, k, dev([0, 20, 40, 60]), dev([0, 20, 40, 60]), good, max_seqlen_q=20)
    for cu_q, cu_k, ok in (([0, 20, 40, 61], [0, 20, 40, 60], [1, 1, 0]), ([0, 20, 10, 60], [0, 20, 40, 60], [1, 0, 0]),
                           ([-5, 20, 40, 60], [0, 20, 40, 60], [0, 1, 1]), ([0, 20, 40, 60], [0, 20, 40, 70], [1, 1, 0]),
                           ([0, 20, 40, 60], [0, 20, 15, 60], [1, 0, 0]), ([0, 20, 40, 60], [-1, 20, 40, 60], [0, 1, 1])):
        o = torch.full_like(q, 7.0)
        gdr.gdr_attn_prefill_varlen(q, k, k, dev(cu_q), dev(cu_k), o, max_seqlen_q=20)
        for n in range(3):
            part, same = o[20 * n:20 * n + 20], good[20 * n:20 * n + 20]
            if ok[n]:
                assert torch.equal(part, same), (cu_q, cu_k, n)
            elif cu_q == [0, 20, 40, 60] and cu_k == [0, 20, 15, 60] and n == 2:
                continue  # 20 queries at the end of 45 keys: well formed, other keys
            else:
                assert (part == 7).all(), (cu_q, cu_k, n)


def test_repeatable_and_captured():
    """Bitwise repeatable; a captured call replays to the same results with eager work between the replays."""
    announce("attn graph")
    B, T, Hq, Hkv, d, window, sinks = 1, 600, 8, 2, 128, 130, 4
    mk = lambda s, H: make(s, "bf16", B, T, H, d).cuda()  # noqa: E731
    q, k, v, go = mk(1, Hq), mk(2, Hkv), mk(3, Hkv), mk(4, Hq)
    o, lse = torch.empty_like(q), torch.empty(B, T, Hq, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(gdr.gdr_attn_backward_workspace_bytes(q.dtype, B, T, T, Hq, Hkv, d, window, sinks), dtype=torch.uint8,
                     device="cuda")

    def step(workspace):
        gdr.gdr_attn_prefill(q, k, v, o, lse, window=window, sinks=sinks)
        gdr.gdr_attn_backward(q, k, v, o, lse, go, dq, dk, dv, window=window, sinks=sinks, workspace=workspace)

    step(None)
    first = [t.clone() for t in (o, lse, dq, dk, dv)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ws)
    for _ in range(3):
        for t in (o, lse, dq, dk, dv):
            t.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, (o, lse, dq, dk, dv)):
            assert torch.equal(a, b)
        torch.randn(1000, device="cuda").sum().item()


def test_side_stream_and_automatic_workspace():
    announce("attn side stream")
    q, k, go = (make(i, "bf16", 1, 300, 4, 64).cuda() for i in range(3))
    o, lse = torch.empty_like(q), torch.empty(1, 300, 4, device="cuda")
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    gdr.gdr_attn_prefill(q, k, k, o, lse, window=20, sinks=1, stream=s)
    gdr.gdr_attn_backward(q, k, k, o, lse, go, dq, dk, dv, window=20, sinks=1, stream=s)
    junk = [torch.full((1 << 18,), 3.0, device="cuda") for _ in range(8)]
    s.synchronize()
    ref = attend(q[0].cpu(), k[0].cpu(), k[0].cpu(), 20, 1, 0.125, torch.bfloat16, go[0].cpu())
    for name, got in (("o", o), ("grad_q", dq), ("grad_k", dk), ("grad_v", dv)):
        check(name, got[0], *ref[name])
    del junk


@pytest.mark.parametrize("B,window,sinks", [(1, 0, 0), (60, 0, 0), (1, 1, 0), (60, 1, 0)])
def test_a_single_visible_key_has_no_score_gradient(B, window, sinks):
    """Softmax of one score is constant: dS = P (dP - delta) with delta = P dP is P dP (1 - P), and P is off from 1 by
    the error of the score (a sum of d products, its scaling, 2^-24 each) and of the exponential and logarithm."""
    announce("attn single key %d %d" % (B, window))
    T, H, d, scale = 40, 4, 128, 0.1
    q, k, v, go = (make(i, "bf16", B, T, H, d) for i in range(4))
    o, lse = forward(q, k, v, window, sinks, scale)
    dq, dk, dv = (torch.empty_like(t).cuda() for t in (q, k, v))
    gdr.gdr_attn_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, go.cuda(), dq, dk, dv, window=window, sinks=sinks, scale=scale)
    rows = slice(0, T if window == 1 else 1)
    q, k, v, go = (t[:, rows].double() for t in (q, k, v, go))
    off = (d + 4) * 2 ** -24 * scale * (q * k).abs().sum(-1, keepdim=True) + 32 * 2 ** -24 * (1 + scale * (q * k).sum(-1, keepdim=True).abs())
    bound = 1.01 * scale * k.abs() * (go * v).abs().sum(-1, keepdim=True) * (off + 2 * d * 2 ** -24)
    assert (dq[:, rows].double().cpu().abs() <= bound).all()


def test_two_streams_at_once():
    """Training steps of different sizes on two streams, enqueued in turn: bitwise what each gives alone."""
    announce("attn two streams")
    cases = [(1, 700, 8, 2, 128, 130, 4), (2, 333, 6, 6, 64, 0, 0)]
    x = [[make(i, "bf16", B, T, H, d).cuda() for i, H in enumerate((Hq, Hkv, Hkv, Hq))] for B, T, Hq, Hkv, d, _, _ in cases]

    def step(case, x, stream):
        B, T, Hq, Hkv, d, window, sinks = case
        q, k, v, go = x
        o, lse = torch.empty_like(q), torch.empty(B, T, Hq, device="cuda")
        dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
        gdr.gdr_attn_prefill(q, k, v, o, lse, window=window, sinks=sinks, stream=stream)
        gdr.gdr_attn_backward(q, k, v, o, lse, go, dq, dk, dv, window=window, sinks=sinks, stream=stream)
        return o, lse, dq, dk, dv

    alone = [step(c, t, None) for c, t in zip(cases, x)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    runs = []
    for _ in range(5):
        for c, t, s in zip(cases, x, streams):
            with torch.cuda.stream(s):
                runs.append((alone[cases.index(c)], step(c, t, None)))
    torch.cuda.synchronize()
    for want, got in runs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals_on_the_device():
    announce("attn refusals")
    q, k = make(1, "bf16", 2, 40, 4, 64).cuda(), make(2, "bf16", 2, 40, 2, 64).cuda()
    o, lse = torch.full_like(q, 7.0), torch.full((2, 40, 4), 7.0, device="cuda")
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    for bad in ((turned, k, k, o), (q, k, k, turned), (q[:, ::2], k, k, o[:, ::2])):
        with pytest.raises(ValueError, match="contiguous"):
            gdr.gdr_attn_prefill(*bad, lse if bad[0].shape == q.shape else None)
    with pytest.raises(ValueError, match="GPU"):
        gdr.gdr_attn_prefill(q, k, k.cpu(), o)
    shifted = torch.zeros(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape)
    with pytest.raises(gdr.GdrError):  # not 16-byte aligned
        gdr.gdr_attn_prefill(shifted, k, k, o)
    need = gdr.gdr_attn_backward_workspace_bytes(q.dtype, 2, 40, 40, 4, 2, 64)
    with pytest.raises(gdr.GdrError):
        gdr.gdr_attn_backward(q, k, k, q, lse, q, o, torch.empty_like(k), torch.empty_like(k),
                              workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert (o == 7).all() and (lse == 7).all()


def test_gradient_against_differences():
    """A directional derivative of sum(grad_o * o) by central differences of the fp32 forward.

    Step h = 2^-6: the third-order term is at most h^2 of the third derivative, the forward's rounding
    (sums of 2^-24 relative) divided by 2h; both well below 1e-2 of the derivative here.
    """
    announce("attn gradient against differences")
    B, T, Hq, Hkv, d, window, sinks, h = 1, 60, 4, 2, 64, 20, 2, 2.0 ** -6
    q, k, v, go = (make(i, "f32", B, T, H, d) for i, H in ((1, Hq), (2, Hkv), (3, Hkv), (4, Hq)))
    o, lse = forward(q, k, v, window, sinks, 0.125)
    grads = [torch.empty_like(t).cuda() for t in (q, k, v)]
    gdr.gdr_attn_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, go.cuda(), *grads, window=window, sinks=sinks, scale=0.125)
    for i in range(3):
        step = make(10 + i, "f32", *(q, k, v)[i].shape)
        val = []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = x[i] + sign * h * step
            val.append(float((forward(*x, window, sinks, 0.125)[0].double().cpu() * go.double()).sum()))
        want = (val[0] - val[1]) / (2 * h)
        got = float((grads[i].double().cpu() * step.double()).sum())
        size = float(grads[i].double().norm() * step.double().norm())
        assert abs(got - want) <= 1e-2 * max(abs(want), size * 1e-2), (i, got, want)
