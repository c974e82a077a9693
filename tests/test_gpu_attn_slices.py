"""The attention backward where rows are cut into slices or segments, against the float64 definition."""
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


# B, Tq, Tk, Hq, Hkv, d, window, sinks: lists that shrink key by key (full causal), that begin late (queries at the end
# of longer keys) or are missing for the first keys (a window far behind them), sinks in some blocks or in all, groups
# that make lists many times longer than the keys, blocks with one key
CASES = [
    (1, 1500, 1500, 8, 1, 64, 0, 0),
    (2, 640, 640, 6, 2, 128, 0, 0),
    (1, 500, 2300, 8, 1, 64, 0, 0),
    (1, 900, 700, 6, 1, 128, 0, 0),
    (1, 300, 2000, 16, 1, 64, 250, 0),
    (1, 700, 1025, 12, 2, 128, 300, 140),
    (1, 1100, 1100, 4, 1, 64, 700, 1000),
    (1, 129, 129, 32, 1, 128, 0, 0),
    (3, 385, 385, 10, 1, 64, 130, 129),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_slices(case, dt):
    B, Tq, Tk, Hq, Hkv, d, window, sinks = case
    announce("attn slices %s %s" % (dt, case))
    q, k, v, go = make(1, dt, B, Tq, Hq, d), make(2, dt, B, Tk, Hkv, d), make(3, dt, B, Tk, Hkv, d), make(4, dt, B, Tq, Hq, d)
    x = [t.cuda() for t in (q, k, v, go)]
    o, lse = torch.empty_like(x[0]), torch.empty(B, Tq, Hq, device="cuda")
    gdr.gdr_attn_prefill(*x[:3], o, lse, window=window, sinks=sinks)
    need = gdr.gdr_attn_backward_workspace_bytes(DT[dt], B, Tq, Tk, Hq, Hkv, d, window, sinks)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")  # NaN where nothing is written
    grads = [torch.full_like(t, 7.0) for t in x[:3]]
    gdr.gdr_attn_backward(*x[:3], o, lse, x[3], *grads, window=window, sinks=sinks, workspace=ws[:need])
    assert (ws[need:] == 255).all()
    for b in range(B):
        ref = attend(q[b], k[b], v[b], window, sinks, d ** -0.5, DT[dt], go[b])
        for name, got in zip(("grad_q", "grad_k", "grad_v"), grads):
            check(name, got[b], *ref[name])
