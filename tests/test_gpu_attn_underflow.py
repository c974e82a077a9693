"""Non-finite values that meet weights too small for fp32: a weight of 0 does not hide them."""
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


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,d", [(1, 64), (1, 128), (300, 64), (300, 128)])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_gradients_of_rows_whose_output_is_not_finite(dt, B, d, what):
    """Key `at` has all the weight of the rows that see it (a score of 400 against about 1) and a non-finite value.
    Their delta is not finite, so neither is any of their score gradients, in whatever step of the walk they come
    and however small the weight: grad_k of every key that one of these rows sees, and of no other."""
    announce("attn underflow, gradients %s %d %d %s" % (dt, B, d, what))
    T, window, at = 100, 5, 33  # the keys before it that the same rows see are another wave's
    q = torch.ones(B, T, 1, d, dtype=DT[dt])
    k, v, go = (make(i, dt, B, T, 1, d) for i in range(3))
    k *= 0.125
    k[:, at] = 400 / d  # a score of 400
    bad = v.clone()
    bad[:, at] = float(what)
    x = [t.cuda() for t in (q, k, bad, go)]
    o, lse = torch.empty_like(x[0]), torch.empty(B, T, 1, device="cuda")
    gdr.gdr_attn_prefill(*x[:3], o, lse, window=window, scale=1.0)
    dq, dk, dv = (torch.full_like(t, 7.0) for t in x[:3])
    gdr.gdr_attn_backward(*x[:3], o, lse, x[3], dq, dk, dv, window=window, scale=1.0)
    rows, keys = range(at, at + window), range(at - window + 1, at + window)
    for b in sorted({0, B // 2, B - 1}):
        ref = attend(q[b], k[b], v[b], window, 0, 1.0, DT[dt], go[b])  # finite values: the weights do not see them
        clean = [i for i in range(T) if i not in rows]
        check("o", o[b, clean], ref["o"][0][clean], ref["o"][1][clean])
        check("grad_q", dq[b, clean], ref["grad_q"][0][clean], ref["grad_q"][1][clean])
        assert torch.isnan(dq[b, list(rows)].float()).all()
        other = [j for j in range(T) if j not in keys]
        check("grad_k", dk[b, other], ref["grad_k"][0][other], ref["grad_k"][1][other])
        assert torch.isnan(dk[b, list(keys)].float()).all()
        check("grad_v", dv[b], *ref["grad_v"])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("pages", [8, 64])  # one workgroup to a head; key blocks dealt out and joined
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_decode_values_whose_weight_underflows(dt, d, pages, what):
    """One key has all the weight (a score of 400 against about 1) and another, of the same or another wave's keys,
    before or after it, a non-finite value: the output is not finite in that value's channel and as ever in the others."""
    announce("attn underflow, decode %s %d %d %s" % (dt, d, pages, what))
    page, Hq, Hkv, n = 16, 4, 2, 127
    assert (gdr.gdr_attn_decode_workspace_bytes(DT[dt], 8, Hq, Hkv, d, page, pages) > 0) == (pages == 64)
    spots = [(3, 5), (3, 40), (3, 126), (70, 2), (70, 75), (70, 100), (120, 1), (120, 127)]  # (heavy key, odd value)
    B = len(spots)
    q = torch.ones(B, Hq, d, dtype=DT[dt])
    k, v = make(1, dt, B, n + 1, Hkv, d) * 0.125, make(2, dt, B, n + 1, Hkv, d)
    for b, (heavy, _) in enumerate(spots):
        k[b, heavy] = 400 / d
    bad = v.clone()
    for b, (_, odd) in enumerate(spots):
        bad[b, odd, :, 9] = float(what)
    table = torch.full((B, pages), -1, dtype=torch.int32)
    table[:, :8] = torch.randperm(8 * B, generator=torch.Generator().manual_seed(1)).reshape(B, 8).int()
    kp, vp = (torch.zeros(8 * B, Hkv, page, d, dtype=DT[dt]) for _ in range(2))
    for b in range(B):
        for pool, t in ((kp, k), (vp, bad)):
            pool[table[b, :8].long()] = t[b].reshape(8, page, Hkv, d).transpose(1, 2)
    lens = torch.full((B,), n, dtype=torch.int32)
    o = torch.full((B, Hq, d), 7.0, dtype=DT[dt], device="cuda")
    gdr.gdr_attn_decode(q.cuda(), k[:, n].contiguous().cuda(), bad[:, n].contiguous().cuda(), kp.cuda(), vp.cuda(), table.cuda(),
                        lens.cuda(), o, scale=1.0)
    rest = [c for c in range(d) if c != 9]
    for b in range(B):
        ref = attend(q[b:b + 1], k[b], v[b], 0, 0, 1.0, DT[dt])["o"]
        check("o", o[b:b + 1, :, rest], ref[0][..., rest], ref[1][..., rest])
        assert not torch.isfinite(o[b, :, 9].float()).any(), spots[b]
