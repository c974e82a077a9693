"""Attention calls on a stream that is not the current one, whose inputs are that stream's own work."""
import pytest
import torch

import gated_delta_rule_08_amd as gdr
from attn_ref import attend, check
from gpu_util import announce, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_offsets_written_on_the_calls_stream(handle):
    """The queries' offsets arrive on the call's stream behind other work there, and no bound is given: it is
    read from them in the order of that stream."""
    announce("attn offsets on another stream %s" % handle)
    lens, Hq, Hkv, d = [70, 1, 200], 4, 2, 64
    cu = torch.tensor([0, 70, 71, 271], dtype=torch.int32)
    q, k, v = make(1, 271, Hq, d), make(2, 271, Hkv, d), make(3, 271, Hkv, d)
    x = [t.cuda() for t in (q, k, v)]
    o = torch.full_like(x[0], 7.0)
    late, ready = torch.zeros(4, dtype=torch.int32, device="cuda"), cu.cuda()
    work = torch.randn(8192, 8192, device="cuda")
    out = torch.empty_like(work)
    s = torch.cuda.Stream()
    torch.mm(work, work, out=out)  # the library is loaded
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(30):
            torch.mm(work, work, out=out)
        late.copy_(ready)
    gdr.gdr_attn_prefill_varlen(*x, late, late, o, stream=s.cuda_stream if handle else s)
    s.synchronize()
    at = 0
    for n in lens:
        check("o", o[at:at + n], *attend(q[at:at + n], k[at:at + n], v[at:at + n], 0, 0, d ** -0.5, torch.bfloat16)["o"])
        at += n


def test_a_bad_offset_leaves_the_other_sequences_without_a_bound():
    """No bound is given and one sequence's offsets are far out of range: that one is skipped, the others are computed."""
    announce("attn bad offset without a bound")
    q, k = make(1, 60, 2, 64).cuda(), make(2, 60, 1, 64).cuda()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good, o = torch.empty_like(q), torch.full_like(q, 7.0)
    gdr.gdr_attn_prefill_varlen(q, k, k, dev([0, 20, 40, 60]), dev([0, 20, 40, 60]), good)
    gdr.gdr_attn_prefill_varlen(q, k, k, dev([0, 20, 40, 2 ** 31 - 1]), dev([0, 20, 40, 60]), o)
    assert torch.equal(o[:40], good[:40]) and (o[40:] == 7).all()


def test_offsets_written_on_the_default_stream_given_as_handle_0():
    """Handle 0 is the default stream, also while another stream is current."""
    announce("attn offsets, handle 0")
    q, k, v = make(1, 90, 4, 64), make(2, 90, 2, 64), make(3, 90, 2, 64)
    x = [t.cuda() for t in (q, k, v)]
    o = torch.full_like(x[0], 7.0)
    late, ready = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.tensor([0, 20, 90], dtype=torch.int32, device="cuda")
    work = torch.randn(8192, 8192, device="cuda")
    out = torch.empty_like(work)
    torch.mm(work, work, out=out)
    torch.cuda.synchronize()
    for _ in range(30):
        torch.mm(work, work, out=out)
    late.copy_(ready)
    assert torch.cuda.default_stream().cuda_stream == 0
    with torch.cuda.stream(torch.cuda.Stream()):
        gdr.gdr_attn_prefill_varlen(*x, late, late, o, stream=0)
    torch.cuda.synchronize()
    for a, b in ((0, 20), (20, 90)):
        check("o", o[a:b], *attend(q[a:b], k[a:b], v[a:b], 0, 0, 0.125, torch.bfloat16)["o"])
