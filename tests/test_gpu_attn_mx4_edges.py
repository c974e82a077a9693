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
