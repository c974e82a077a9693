"""Reference of the 4-bit cache in 64 bits on the CPU: the format from its definition, a paged cache of it, and the
attention over it with a bound of each output's error.

Blocks of 32 channels: scale byte b, value = code * 2^(b - 127), codes 0, 1/2, 1, 3/2, 2, 3, 4, 6 and a sign bit.  b is
the least in 1 .. 252 with max |x| <= 7 2^(b - 127); a value takes the nearest code, ties the even one.  A block with an
infinity or NaN is b = 255 with codes 0.

Bounds: as attn_ref has them (u32 = 2^-24, u the element type's unit).  With fp32 the query and the weights go in as three
bf16 pieces of 8 bits each, which hold all 24: nothing is lost, but a sum of n products has 3 n terms.  So a score is off by
at most ds = (P d + 4) u32 scale sum |q||k| + 4 u32 |s| with P = 3 (bf16: 1), and o by (u + 2 ds + (P n + 16) u32)
sum p |v| + u |o|, the first u only where the weights are rounded to bf16.
"""
import math

import torch

from attn_ref import U32, unit

VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def quantise(x):
    """x [..., d] -> (codes uint8 [..., d], scale bytes uint8 [..., d / 32])."""
    x = x.double().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    odd = ~torch.isfinite(x).all(-1)
    x = torch.where(odd[..., None], torch.zeros_like(x), x)
    top = torch.where(odd, torch.ones_like(top), top)
    b = torch.full(top.shape, 1, dtype=torch.int64)
    m, e = torch.frexp(top)
    b = torch.where(top > 0, e.long() - 3 + (m > 0.875).long() + 127, b).clamp(1, 252)
    y = (x.abs() / torch.ldexp(torch.ones(()).double(), (b - 127).double())[..., None]).clamp(max=6.0)
    far = (y[..., None] - torch.tensor(VALUES, dtype=torch.float64)).abs()
    best = far.amin(-1, keepdim=True)
    tie = far == best
    rank = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7])  # the even codes first
    code = torch.where(tie, rank, 8).argmin(-1)
    code = (code + 8 * torch.signbit(x)).to(torch.uint8)
    code = torch.where(odd[..., None], torch.zeros_like(code), code)
    return code.flatten(-2), torch.where(odd, torch.full_like(b, 255), b).to(torch.uint8)


def value(codes, scales):
    t = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64)
    s = torch.ldexp(torch.ones(()).double(), scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return t[codes.long()] * s.repeat_interleave(32, -1)


class Mx4Cache:
    """A paged 4-bit cache on the CPU: where no token is, scales of 255 and codes of 15, pages in random order."""

    def __init__(self, lengths, room, Hkv, d, page, seed=0, spare=2):
        self.page, self.lengths, self.Hkv, self.d = page, list(lengths), Hkv, d
        need = [-(-(n + r) // page) for n, r in zip(lengths, room)]
        order = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table = torch.full((len(lengths), max(1, max(need, default=1))), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
            order = order[n:]
        pages = sum(need) + spare
        self.kc = torch.full((pages, Hkv, page, d), 15, dtype=torch.uint8)  # one code to a byte
        self.vc = self.kc.clone()
        self.ks = torch.full((pages, Hkv, page, d // 32), 255, dtype=torch.uint8)
        self.vs = self.ks.clone()

    def put(self, b, at, k, v):
        """k, v [n, Hkv, d] to the positions from `at` of sequence b."""
        n = k.shape[0]
        pos = torch.arange(at, at + n)
        page, slot = self.table[b, pos // self.page].long(), pos % self.page
        for x, c, s in ((k, self.kc, self.ks), (v, self.vc, self.vs)):
            codes, scales = quantise(x)
            c[page, :, slot], s[page, :, slot] = codes, scales

    def get(self, b, at, n):
        """float64 keys and values [n, Hkv, d]."""
        pos = torch.arange(at, at + n)
        page, slot = self.table[b, pos // self.page].long(), pos % self.page
        return tuple(value(c[page, :, slot], s[page, :, slot]) for c, s in ((self.kc, self.ks), (self.vc, self.vs)))

    def packed(self):
        """k_codes, k_scales, v_codes, v_scales as the library takes them."""
        k = self.kc[..., 0::2] | (self.kc[..., 1::2] << 4)
        v = self.vc.unflatten(2, (-1, 32)).transpose(-1, -2)
        v = v[..., 0::2] | (v[..., 1::2] << 4)
        return k.contiguous(), self.ks.clone(), v.contiguous(), self.vs.clone()

    def device(self):
        return (*(x.cuda() for x in self.packed()), self.table.cuda())


def attend(q, k, v, n, window, sinks, scale, dtype):
    """q [Tq,Hq,d], the last of n positions, on float64 k, v [n,Hkv,d].  Returns (o, bound)."""
    Tq, Hq, d = q.shape
    G = Hq // k.shape[1] if k.shape[1] else 1
    P = 3 if dtype == torch.float32 else 1
    u, uo = (0.0 if dtype == torch.float32 else unit(dtype)), unit(dtype)
    q = q.double()
    o, bound = torch.zeros(Tq, Hq, d, dtype=torch.float64), torch.zeros(Tq, Hq, d, dtype=torch.float64)
    p0 = torch.arange(Tq).reshape(-1, 1) + n - Tq
    j = torch.arange(n).reshape(1, -1)
    see = (j <= p0) & ((window == 0) | (j > p0 - window) | (j < sinks))
    for h in range(Hq):
        kh, vh, qh = k[:, h // G], v[:, h // G], q[:, h]
        for i in range(Tq):
            at = see[i].nonzero()[:, 0]
            if not len(at):
                continue
            s = (kh[at] @ qh[i]) * scale
            ds = (P * d + 4) * U32 * abs(scale) * (kh[at].abs() @ qh[i].abs()) + 4 * U32 * s.abs()
            p = torch.softmax(s, 0)
            o[i, h] = p @ vh[at]
            bound[i, h] = (u + 2 * ds.max() + (P * len(at) + 16) * U32) * (p @ vh[at].abs()) + uo * o[i, h].abs()
    return o, bound
