"""Float64 reference of the attention operators and elementwise error bounds.

``attend`` computes one sequence's attention (and, with grad_o, its gradients)
from the definition in float64 on the CPU, together with a bound of the error
each output element may have.  The bounds come from the kernels' roundings
alone, u = eps / 2 being the largest relative error of one:

 * a score is a sum of d products and one scaling in fp32: it is off by at
   most ds = (d + 4) u32 scale sum |q||k| + 4 u32 |s|; so a weight is off by
   ds + 8 u32 (the exponential), relative, and by twice that once normalised;
 * a weight (and a score gradient) enters the second product rounded to the
   element type: u more, relative;
 * sums of n terms in fp32 add n u32 of the sum of magnitudes;
 * an output is rounded to its type: u of its value.

So |o - exact| <= (u + 2 ds + (n + 16) u32) sum p |v| + u |o|.  For the
gradients, with P off by e_p = 2 ds + (n + 16) u32 relatively,
delta_i off by sum |do| |o error| + d u32 sum |do| |o| and dP by
d u32 sum |do| |v|:  dS is off by
    E = P (dP error + delta error) + (u + e_p + 4 u32) |dS|,
and grad_q by scale sum E |k| + (n u32 + 2 u32) scale sum |dS| |k| + u |dq|,
the other gradients in the same way.
"""
import math

import torch

U32 = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def visible(Tq, Tk, window, sinks):
    p = torch.arange(Tq).reshape(-1, 1) + Tk - Tq
    j = torch.arange(Tk).reshape(1, -1)
    return (j <= p) & ((window == 0) | (j > p - window) | (j < sinks))


def attend(q, k, v, window, sinks, scale, dtype, grad_o=None):
    """q [Tq,Hq,d], k, v [Tk,Hkv,d] on the CPU.  Returns {name: (value, bound)}."""
    Tq, Hq, d = q.shape
    Tk, Hkv, _ = k.shape
    u, G = (0.0 if dtype == torch.float32 else unit(dtype)), Hq // Hkv
    uo = unit(dtype)
    q, k, v = q.double(), k.double(), v.double()
    see = visible(Tq, Tk, window, sinks)
    out = {n: (torch.zeros(s, dtype=torch.float64), torch.zeros(s, dtype=torch.float64))
           for n, s in (("o", q.shape), ("lse", q.shape[:2]), ("grad_q", q.shape), ("grad_k", k.shape), ("grad_v", v.shape))}
    raw = {n: torch.zeros_like(out[n][0]) for n in ("grad_k", "grad_v")}
    for h in range(Hq):
        qh, kh, vh = q[:, h], k[:, h // G], v[:, h // G]
        s = (qh @ kh.t()) * scale
        ds = ((d + 4) * U32 * abs(scale) * (qh.abs() @ kh.abs().t()) + 4 * U32 * s.abs()).masked_fill(~see, 0)
        es = ds.amax(-1, keepdim=True) if Tk else torch.zeros(Tq, 1, dtype=torch.float64)
        s = s.masked_fill(~see, -math.inf)
        lse = torch.logsumexp(s, -1, keepdim=True) if Tk else torch.full((Tq, 1), -math.inf, dtype=torch.float64)
        p = torch.exp(s - lse.nan_to_num(neginf=0.0)).masked_fill(~see, 0)
        n = see.sum(-1, keepdim=True)
        ep = 2 * es + (n + 16) * U32
        o = p @ vh
        eo = (u + ep) * (p @ vh.abs()) + uo * o.abs()
        out["o"][0][:, h], out["o"][1][:, h] = o, eo
        out["lse"][0][:, h] = lse[:, 0]
        out["lse"][1][:, h] = (es + (n + 16) * U32 + 8 * U32 * lse.abs().nan_to_num(posinf=0.0))[:, 0]
        if grad_o is None:
            continue
        g = grad_o[:, h].double()
        dp, delta = g @ vh.t(), (g * o).sum(-1, keepdim=True)
        e_delta = (g.abs() * eo).sum(-1, keepdim=True) + (d + 4) * U32 * (g.abs() * o.abs()).sum(-1, keepdim=True)
        e_dp = (d + 4) * U32 * (g.abs() @ vh.abs().t())
        dS = p * (dp - delta)
        E = p * (e_dp + e_delta) + (u + ep + 4 * U32) * dS.abs()
        many = (Tk + 4) * U32
        dq = scale * dS @ kh
        out["grad_q"][0][:, h] = dq
        out["grad_q"][1][:, h] = abs(scale) * ((E + many * dS.abs()) @ kh.abs()) + uo * dq.abs()
        many = (Tq * G + 4) * U32
        out["grad_k"][0][:, h // G] += scale * dS.t() @ qh
        out["grad_k"][1][:, h // G] += abs(scale) * ((E + many * dS.abs()).t() @ qh.abs())
        out["grad_v"][0][:, h // G] += p.t() @ g
        out["grad_v"][1][:, h // G] += ((u + ep + many) * p).t() @ g.abs()
    for n in raw:
        out[n][1].add_(uo * (out[n][0].abs() + out[n][1]))
    return out


def check(name, got, ref, bound):
    """got against ref elementwise; infinities must agree.  Returns the largest share of the bound used."""
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), "%s: infinities differ" % name
    err = (got - ref).masked_fill(inf, 0).abs()
    bad = ~(err <= bound + 1e-30)
    if bad.any():
        at = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d elements off, first at %s: got %r, exact %r, bound %.3g" % (
            name, int(bad.sum()), bad.numel(), at, float(got[at]), float(ref[at]), float(bound[at])))
    return float((err / (bound + 1e-30)).max()) if err.numel() else 0.0
