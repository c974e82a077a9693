"""Attention at the ends of what its arguments allow: scores of -infinity, large scores, pages shared by sequences."""
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


def step(q, k, v, go, window, sinks, scale):
    x = [t.cuda() for t in (q, k, v, go)]
    o, lse = torch.full_like(x[0], 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    gdr.gdr_attn_prefill(*x[:3], o, lse, window=window, sinks=sinks, scale=scale)
    grads = [torch.full_like(t, 7.0) for t in x[:3]]
    gdr.gdr_attn_backward(*x[:3], o, lse, x[3], *grads, window=window, sinks=sinks, scale=scale)
    return (o, lse, *grads)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,d", [(1, 70, 64), (1, 500, 128), (150, 70, 128)])
def test_rows_whose_scores_all_overflow_to_minus_infinity(dt, B, T, d):
    """Such a row has no weight: o = 0, lse = -infinity, and no gradient flows through it; other rows are as ever."""
    announce("attn scores of -infinity %s %d %d %d" % (dt, B, T, d))
    H, first = 2, T // 2
    q, k, v, go = (make(i, dt, B, T, H, d) for i in range(4))
    k = k.abs()
    # head 0: half the queries as large as its keys, of the other sign, so that every product with a key overflows
    q[:, first:, 0], k[:, :, 0] = -2.0 ** 70, 2.0 ** 70
    o, lse, dq, dk, dv = step(q, k, v, go, 0, 0, 1.0)
    assert (o[:, first:, 0] == 0).all() and (lse[:, first:, 0] == -float("inf")).all()
    assert (dq[:, first:, 0] == 0).all()
    assert (dk[:, first:, 0] == 0).all() and (dv[:, first:, 0] == 0).all()  # keys that only these rows see
    for b in (0, B - 1):
        ref = attend(q[b, :, 1:], k[b, :, 1:], v[b, :, 1:], 0, 0, 1.0, DT[dt], go[b, :, 1:])
        for name, got in (("o", o), ("lse", lse), ("grad_q", dq), ("grad_k", dk), ("grad_v", dv)):
            check(name, got[b, :, 1:], *ref[name])


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 64), ("f32", 128)])
def test_gradients_at_large_scores(dt, d):
    """Scores of several hundred, where the log-sum-exp carries the largest rounding."""
    announce("attn gradients at large scores %s %d" % (dt, d))
    q, k, v, go = make(1, dt, 1, 200, 2, d) * 8, make(2, dt, 1, 200, 2, d) * 8, make(3, dt, 1, 200, 2, d), make(4, dt, 1, 200, 2, d)
    got = step(q, k, v, go, 50, 3, 1.0)
    ref = attend(q[0], k[0], v[0], 50, 3, 1.0, DT[dt], go[0])
    for name, t in zip(("o", "lse", "grad_q", "grad_k", "grad_v"), got):
        check(name, t[0], *ref[name])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("pages", [12, 80])  # one workgroup to a head; key blocks dealt out and joined
def test_sequences_that_share_full_pages(dt, pages):
    """A prefix appended once, its full pages in several sequences' tables; one table names a page twice."""
    announce("attn shared pages %s %d" % (dt, pages))
    page, Hq, Hkv, d, B = 16, 8, 2, 64, 4
    prefix = 5 * page
    k, v = make(1, dt, prefix, Hkv, d), make(2, dt, prefix, Hkv, d)
    kp, vp = (torch.full((12, Hkv, page, d), float("nan"), dtype=DT[dt], device="cuda") for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    row = lambda *x: list(x) + [-1] * (pages - len(x))  # noqa: E731
    gdr.gdr_attn_append(k.cuda(), v.cuda(), i32([0, prefix]), i32([0]), kp, vp, i32([row(0, 1, 2, 3, 4)]))
    seqs = [[0, 1, 2, 3, 4], [0, 1, 2], [0, 1, 2, 3, 4], [2, 2, 0]]  # their full pages; then one of their own
    table = i32([row(*s, 5 + b) for b, s in enumerate(seqs)])
    held = [len(s) * page for s in seqs]
    own = [[torch.empty(0, Hkv, d, dtype=DT[dt])] * 2 for _ in range(B)]
    for t in range(3):
        q, k1, v1 = make(10 + t, dt, B, Hq, d), make(20 + t, dt, B, Hkv, d), make(30 + t, dt, B, Hkv, d)
        o = torch.empty(B, Hq, d, dtype=DT[dt], device="cuda")
        gdr.gdr_attn_decode(q.cuda(), k1.cuda(), v1.cuda(), kp, vp, table, i32([n + t for n in held]), o)
        for b, s in enumerate(seqs):
            own[b] = [torch.cat([a, x[b:b + 1]]) for a, x in zip(own[b], (k1, v1))]
            full = [torch.cat([x[p * page:(p + 1) * page] for p in s] + [own[b][i]]) for i, x in enumerate((k, v))]
            check("o", o[b:b + 1], *attend(q[b:b + 1], *full, 0, 0, d ** -0.5, DT[dt])["o"])
