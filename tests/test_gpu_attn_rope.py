"""Norm and rotation of queries and keys, and its backward, against the formulas in float64.

Bounds (u32 = 2^-24, u the type's unit).  1 / sqrt(mean + eps): the sum of d squares is off by d u32, its root by half of
that; with the root's own rounding, the products by x, the root and w: (d / 2 + 8) u32 relative for each y.  A turned
channel is y_a cos - y_b sin: cos and sin are off by 4 u32 (their own 2 and a quarter-turn angle rounded to fp32), the
products and the difference by 3 more, and a position's angle t by 8 2^-53 |t|: so it is off by at most
((d / 2 + 16) u32 + 8 2^-53 |t|) (|y_a| + |y_b|), and u of its value.  The gradients go back through the same steps.
"""
import math

import pytest
import torch

import gated_delta_rule_08_amd as gdr
from attn_ref import U32, check, unit
from gpu_util import announce, ensure_built

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(seed, dt, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dt)


def pairs(x, half, il):
    a = x[..., 0:2 * half:2] if il else x[..., :half]
    b = x[..., 1:2 * half:2] if il else x[..., half:2 * half]
    return a, b


def joined(a, b, rest, il):
    t = torch.stack([a, b], -1).flatten(-2) if il else torch.cat([a, b], -1)
    return torch.cat([t, rest], -1)


def turn(x, t, il):
    """x [..., H, d] turned by angles t [..., rot / 2]; and |a| + |b| of each channel's pair (|x| of the others)."""
    half = t.shape[-1]
    a, b = pairs(x, half, il)
    c, s = t.cos()[..., None, :], t.sin()[..., None, :]
    rest = x[..., 2 * half:]
    return joined(a * c - b * s, b * c + a * s, rest, il), joined(a.abs() + b.abs(), a.abs() + b.abs(), rest.abs(), il)


def angle_error(t, shape, il):
    e = (8 * 2.0 ** -53) * t.abs()[..., None, :].expand(*shape[:-1], t.shape[-1])
    return joined(e, e, torch.zeros(*shape[:-1], shape[-1] - 2 * t.shape[-1], dtype=torch.float64), il)


def reference(x, w, t, il, norm, eps, g=None):
    """{name: (value, bound)} in float64 for x [..., H, d] of the given type."""
    d, u = x.shape[-1], unit(x.dtype)
    x = x.double()
    w = torch.ones(d, dtype=torch.float64) if w is None else w.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt() if norm else torch.ones(())
    hat = x * r
    e = (d / 2 + 16) * U32 + angle_error(t, x.shape, il)
    out, both = turn(hat * w, t, il)
    got = {"out": (out, e * both + u * out.abs() * (1 + 1e-3))}
    if g is None:
        return got
    back, both = turn(g.double(), -t, il)
    eb = e * both
    if not norm:
        got["grad"] = (back, eb + u * back.abs() * (1 + 1e-3))
        return got
    uw, mean = back * w, (back * w * hat).mean(-1, keepdim=True)
    grad = (uw - hat * mean) * r
    c = (2 * d + 32) * U32
    size = uw.abs() + hat.abs() * (uw * hat).abs().mean(-1, keepdim=True)
    err = eb * w.abs() + hat.abs() * (eb * w.abs() * hat.abs()).mean(-1, keepdim=True)
    got["grad"] = (grad, (c * size + err) * r + u * grad.abs() * (1 + 1e-3))
    axes = tuple(range(x.dim() - 1))
    terms = back * hat
    n = terms[..., 0].numel()
    got["grad_w"] = (terms.sum(axes), (eb * hat.abs() + (n + d / 2 + 10) * U32 * terms.abs()).sum(axes))
    return got


def frequencies(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2).double() / max(rot, 1))).float()


def run(dt, lead, Hq, Hkv, d, rot, il, norm=True, weights=True, fused=False, far=0, eps=1e-6, scale=1.0, seed=0):
    T = DT[dt]
    tokens = math.prod(lead)
    if fused:
        qkv = make(seed, T, *lead, Hq + 2 * Hkv, d) * scale
        dev = qkv.cuda()
        q, k = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :]
        qd, kd = dev[..., :Hq, :], dev[..., Hq:Hq + Hkv, :]
    else:
        q, k = make(seed, T, *lead, Hq, d) * scale, make(seed + 1, T, *lead, Hkv, d) * scale
        qd, kd = q.cuda(), k.cuda()
    wq, wk = (1 + 0.3 * make(seed + 2, torch.float32, d), 0.5 * make(seed + 3, torch.float32, d)) if weights else (None, None)
    g = torch.Generator().manual_seed(seed + 4)
    pos = torch.randint(-far, far + 1, lead, generator=g, dtype=torch.int64) if far else torch.arange(tokens).reshape(lead)
    pos = pos.to(torch.int32)
    freq = frequencies(rot)
    t = pos[..., None].double() * freq.double()
    gq, gk = make(seed + 5, T, *lead, Hq, d), make(seed + 6, T, *lead, Hkv, d)
    up = lambda x: None if x is None else x.cuda()
    qo, ko = torch.full(q.shape, 7.0, dtype=T, device="cuda"), torch.full(k.shape, 7.0, dtype=T, device="cuda")
    how = dict(w_q=up(wq), w_k=up(wk), eps=eps, norm=norm, interleaved=il)
    gdr.gdr_attn_norm_rope(qd, kd, pos.cuda(), freq.cuda(), qo, ko, **how)
    if fused:
        wide = torch.full((*lead, Hq + 2 * Hkv, d), 7.0, dtype=T, device="cuda")
        dq, dk = wide[..., :Hq, :], wide[..., Hq:Hq + Hkv, :]
    else:
        dq, dk = torch.full_like(qo, 7.0), torch.full_like(ko, 7.0)
    dwq = torch.full((d,), 7.0, device="cuda") if norm and weights else None
    dwk = torch.full((d,), 7.0, device="cuda") if norm and weights else None
    gdr.gdr_attn_norm_rope_backward(qd, kd, pos.cuda(), freq.cuda(), gq.cuda(), gk.cuda(), dq, dk, grad_w_q=dwq, grad_w_k=dwk, **how)
    torch.cuda.synchronize()
    for name, x, w, g, out, dx, dw in (("q", q, wq, gq, qo, dq, dwq), ("k", k, wk, gk, ko, dk, dwk)):
        if not x.numel():
            if dw is not None:
                assert (dw == 0).all()
            continue
        ref = reference(x, w, t, il, norm, eps, g)
        check(name, out, *ref["out"])
        check("grad_" + name, dx, *ref["grad"])
        if dw is not None:
            check("grad_w_" + name, dw, *ref["grad_w"])
    if fused:
        assert (wide[..., Hq + Hkv:, :] == 7).all()  # the values' places
    return qo, ko, dq, dk, dwq, dwk


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("lead,Hq,Hkv,d,rot,fused", [
    ((1,), 1, 1, 64, 64, False), ((7,), 4, 2, 128, 128, True), ((3, 5), 6, 2, 64, 32, True), ((2, 33), 5, 5, 128, 16, False),
    ((130,), 32, 8, 128, 128, True), ((64,), 3, 1, 64, 48, False), ((9,), 2, 0, 64, 64, False), ((9,), 0, 3, 128, 48, False),
    ((700,), 1, 1, 128, 64, True), ((1500,), 1, 0, 64, 64, False), ((2, 2, 3), 16, 1, 128, 112, True), ((1, 4), 2, 2, 64, 0, False),
])
def test_sizes(dt, il, lead, Hq, Hkv, d, rot, fused):
    announce("rope %s il=%s %s" % (dt, il, (lead, Hq, Hkv, d, rot, fused)))
    run(dt, lead, Hq, Hkv, d, rot, il, fused=fused)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("norm,weights", [(True, False), (False, False)])
def test_without_weights_or_norm(dt, norm, weights):
    announce("rope %s norm=%s" % (dt, norm))
    run(dt, (70,), 6, 2, 128, 64, False, norm=norm, weights=weights, fused=True)
    run(dt, (70,), 6, 2, 64, 64, True, norm=norm, weights=weights)


@pytest.mark.parametrize("far", [1 << 20, 2 ** 31 - 1])
def test_far_positions(far):
    """Positions over the whole range of int32, both signs."""
    announce("rope far %d" % far)
    run("f32", (200,), 2, 1, 128, 128, False, far=far)
    run("f32", (200,), 2, 1, 64, 64, True, far=far)


@pytest.mark.parametrize("scale", [1e-18, 1e-5, 1e15])
def test_magnitudes(scale):
    """Rows far below sqrt(eps), near it and far above; eps 0."""
    announce("rope magnitudes %g" % scale)
    run("f32", (40,), 3, 1, 64, 64, False, scale=scale)
    if scale > 1e-10:
        run("f32", (40,), 3, 1, 128, 128, True, scale=scale, eps=0.0)


def test_many_rows_and_repeats():
    """More chunks than the backward has workgroups; repeated calls agree bit by bit."""
    announce("rope many rows")
    a = run("bf16", (4100,), 32, 8, 64, 64, False, seed=3)
    b = run("bf16", (4100,), 32, 8, 64, 64, False, seed=3)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_zero_rows():
    """A row of zeros stays zeros, and so does its gradient's direction: dx = u w / sqrt(eps)."""
    announce("rope zero rows")
    q = torch.zeros(3, 2, 64, device="cuda")
    pos, freq = torch.arange(3, dtype=torch.int32, device="cuda"), frequencies(64).cuda()
    g = make(1, torch.float32, 3, 2, 64).cuda()
    out, dq, dw = torch.ones_like(q), torch.ones_like(q), torch.ones(64, device="cuda")
    none = q[:, :0]
    gdr.gdr_attn_norm_rope(q, none, pos, freq, out, none.clone(), w_q=dw.clone())
    gdr.gdr_attn_norm_rope_backward(q, none, pos, freq, g, none.clone(), dq, none.clone(), w_q=dw.clone(), grad_w_q=dw)
    torch.cuda.synchronize()
    assert (out == 0).all() and (dw == 0).all()
    back, both = turn(g.double().cpu(), -(pos.cpu()[:, None].double() * freq.cpu().double()), False)
    check("grad_q", dq, back * 1e3, 1e3 * 64 * U32 * both)


def test_in_place():
    announce("rope in place")
    for dt in DT.values():
        q, k = make(1, dt, 50, 4, 128).cuda(), make(2, dt, 50, 2, 128).cuda()
        gq, gk = make(3, dt, 50, 4, 128).cuda(), make(4, dt, 50, 2, 128).cuda()
        pos, freq = torch.arange(50, dtype=torch.int32, device="cuda"), frequencies(128).cuda()
        qo, ko, dq, dk = (torch.empty_like(x) for x in (q, k, q, k))
        gdr.gdr_attn_norm_rope(q, k, pos, freq, qo, ko)
        gdr.gdr_attn_norm_rope_backward(q, k, pos, freq, gq, gk, dq, dk)
        gdr.gdr_attn_norm_rope_backward(q, k, pos, freq, gq, gk, gq, gk)
        gdr.gdr_attn_norm_rope(q, k, pos, freq, q, k)
        torch.cuda.synchronize()
        assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(gq, dq) and torch.equal(gk, dk)


def test_gradient_against_differences():
    """Central differences of the forward itself, in fp32 with steps that leave about 3 digits."""
    announce("rope differences")
    T, Hq, d = 2, 2, 64
    q, k = make(1, torch.float32, T, Hq, d), make(2, torch.float32, T, 1, d)
    wq, wk = 1 + 0.3 * make(3, torch.float32, d), 1 + 0.3 * make(4, torch.float32, d)
    gq, gk = make(5, torch.float32, T, Hq, d), make(6, torch.float32, T, 1, d)
    pos, freq = torch.tensor([3, 70], dtype=torch.int32).cuda(), frequencies(32).cuda()

    def loss(q, k, wq, wk):
        qo, ko = torch.empty_like(q).cuda(), torch.empty_like(k).cuda()
        gdr.gdr_attn_norm_rope(q.cuda(), k.cuda(), pos, freq, qo, ko, w_q=wq.cuda(), w_k=wk.cuda())
        return float((qo.double().cpu() * gq.double()).sum() + (ko.double().cpu() * gk.double()).sum())

    grads = [torch.empty_like(x).cuda() for x in (q, k, wq, wk)]
    gdr.gdr_attn_norm_rope_backward(q.cuda(), k.cuda(), pos, freq, gq.cuda(), gk.cuda(), grads[0], grads[1], w_q=wq.cuda(),
                                    w_k=wk.cuda(), grad_w_q=grads[2], grad_w_k=grads[3])
    args = [q, k, wq, wk]
    h = 2.0 ** -8
    for n, x in enumerate(args):
        for at in (0, 5, 31, 40, x.numel() - 1):
            lo, hi = x.clone(), x.clone()
            lo.view(-1)[at] -= h
            hi.view(-1)[at] += h
            num = (loss(*args[:n], hi, *args[n + 1:]) - loss(*args[:n], lo, *args[n + 1:])) / (2 * h)
            # third derivative of order 1 / |x|^2 times the gradients: h^2 of it; 384 terms of fp32 roundings over 2 h
            assert abs(num - float(grads[n].view(-1)[at])) < 40 * h * h + 2 * 384 * 4 * U32 / (2 * h), (n, at)


def test_empty():
    announce("rope empty")
    q, k = torch.empty(0, 4, 64, device="cuda"), torch.empty(0, 2, 64, device="cuda")
    pos, freq = torch.empty(0, dtype=torch.int32, device="cuda"), frequencies(64).cuda()
    w = torch.ones(64, device="cuda")
    dwq, dwk = w.clone(), w.clone()
    gdr.gdr_attn_norm_rope(q, k, pos, freq, q.clone(), k.clone(), w_q=w, w_k=w)
    gdr.gdr_attn_norm_rope_backward(q, k, pos, freq, q, k, q.clone(), k.clone(), w_q=w, w_k=w, grad_w_q=dwq, grad_w_k=dwk)
    torch.cuda.synchronize()
    assert (dwq == 0).all() and (dwk == 0).all()
