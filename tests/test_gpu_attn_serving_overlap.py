"""Tensors of one call that share memory, through the binding on the GPU: refused, and nothing written; or an output in its
own input's place, with the result it has elsewhere."""
import pytest
import torch

import gated_delta_rule_08_amd as gdr
from gpu_util import announce, ensure_built
from mx4_ref import Mx4Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(seed, dt, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dt)


def ints(xs):
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def refused(buffer, call):
    before = buffer.clone()
    with pytest.raises(gdr.GdrError, match="overlap"):
        call()
    torch.cuda.synchronize()
    assert torch.equal(buffer, before)


def test_rotation():
    announce("overlap rotation")
    T, H, d = 6, 2, 64
    pool = make(1, torch.float32, 8 * T * H * d).cuda()
    at = lambda i: pool[i:i + T * H * d].view(T, H, d)  # noqa: E731
    n = T * H * d
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    q, k = at(0), at(n)
    refused(pool, lambda: gdr.gdr_attn_norm_rope(q, k, pos, freq, at(2 * n), at(3 * n - 4)))
    refused(pool, lambda: gdr.gdr_attn_norm_rope(q, k, pos, freq, at(4), at(3 * n)))
    refused(pool, lambda: gdr.gdr_attn_norm_rope(q, k, pos, freq, at(2 * n), at(3 * n), w_q=pool[3 * n + 8:3 * n + 8 + d]))
    refused(pool, lambda: gdr.gdr_attn_norm_rope_backward(q, k, pos, freq, at(2 * n), at(3 * n), at(4 * n), at(5 * n - 64)))
    refused(pool, lambda: gdr.gdr_attn_norm_rope_backward(q, k, pos, freq, at(2 * n), at(3 * n), at(4 * n), at(5 * n), w_q=pool[6 * n:6 * n + d],
                                                          grad_w_q=pool[6 * n + 4:6 * n + 4 + d]))
    # views that interleave: queries, keys and their gradients in one buffer
    wide = make(2, torch.float32, T, 4 * H, d).cuda()
    g = make(3, torch.float32, 2, T, H, d).cuda()
    dq, dk = torch.empty_like(q), torch.empty_like(q)
    gdr.gdr_attn_norm_rope_backward(wide[:, :H].contiguous(), wide[:, H:2 * H].contiguous(), pos, freq, g[0], g[1], dq, dk)
    gdr.gdr_attn_norm_rope_backward(wide[:, :H], wide[:, H:2 * H], pos, freq, g[0], g[1], wide[:, 2 * H:3 * H], wide[:, 3 * H:])
    torch.cuda.synchronize()
    assert torch.equal(wide[:, 2 * H:3 * H], dq) and torch.equal(wide[:, 3 * H:], dk)


def test_page_plan():
    announce("overlap page plan")
    pool = ints(list(range(1, 200)))
    at = lambda i, n: pool[i:i + n]  # noqa: E731
    names = dict(lengths=at(0, 3), add=at(3, 3), free_pages=at(6, 20), n_free=at(26, 1), page_table=at(27, 12).view(3, 4),
                 cu_seqlens=at(39, 4), added=at(43, 3), lengths_out=at(46, 3), n_free_out=at(49, 1), slots=at(50, 30))
    call = lambda **kw: gdr.gdr_attn_plan_pages(**{**names, "page_size": 16, **kw})  # noqa: E731
    for kw in (dict(added=at(4, 3)), dict(lengths_out=at(1, 3)), dict(cu_seqlens=at(36, 4)), dict(slots=at(48, 30)),
               dict(page_table=at(25, 12).view(3, 4)), dict(added=at(0, 3)), dict(n_free_out=at(10, 1))):
        refused(pool, lambda: call(**kw))
    call()


def test_cache_and_decode():
    announce("overlap cache and decode")
    for Hq, Hkv, d, page, lengths, Tq in ((8, 2, 128, 32, [70, 1, 33, 600], 1), (4, 2, 64, 64, [4999, 1, 300, 0], 3),
                                          (4, 4, 64, 32, [1 + b % 60 for b in range(300)], 1)):
        c = Mx4Cache(lengths, [0] * len(lengths), Hkv, d, page)
        for b, n in enumerate(lengths):
            c.put(b, 0, make(b, torch.float32, n, Hkv, d), make(b + 1000, torch.float32, n, Hkv, d))
        dev, lens = c.device(), ints(lengths)
        for dt in (torch.float32, torch.bfloat16):
            q = make(7, dt, len(lengths), Tq, Hq, d).cuda()
            o = torch.empty_like(q)
            gdr.gdr_attn_decode_mx4(q, *dev, lens, o)
            gdr.gdr_attn_decode_mx4(q, *dev, lens, q)
            torch.cuda.synchronize()
            assert torch.equal(q, o)
    pool = torch.zeros(3 * q.numel(), dtype=q.dtype, device="cuda")
    at = lambda i: pool[i:i + q.numel()].view(q.shape)  # noqa: E731
    refused(pool, lambda: gdr.gdr_attn_decode_mx4(at(0), *dev, lens, at(8)))
    x = make(1, torch.float32, 5, Hkv, d).cuda()
    kc, ks, vc, vs, table = dev
    refused(kc, lambda: gdr.gdr_attn_append_mx4(x, x, ints([0, 5] + [5] * 299), lens, kc, ks, kc.view(vc.shape), vs, table))
    out = torch.zeros(11, Hkv, d, device="cuda")
    refused(out, lambda: gdr.gdr_attn_read_mx4(*dev, ints([0, 5] + [6] * 299), out[:6], out[5:]))
