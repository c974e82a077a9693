"""Performance cases of the operators around the attention layers: the norm and position rotation of queries
and keys with its gradients, the page plan of a serving step, and the key-value cache held in 4 bits (append,
read back, decode step).

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``prepare`` makes a
case's inputs on the GPU, ``run`` is one pass: with ``own`` the library's kernels, else the same
operator in elementary torch operations in fp32.  ``exact`` is the definition in float64 and
``work`` the bytes and operations a pass cannot do without.

The 4-bit format: 32 values share a scale 2^e (one byte, e + 127) and each is a sign and one of 0, 1/2, 1, 3/2,
2, 3, 4, 6 (the 8 codes in order), times 2^e.  e is the least integer with max |x| <= 7 2^e, within -126 .. 125;
a value goes to the nearest, ties to the even code, and 6 from there on.  The 32 values are consecutive channels
of one position and head, for keys and values alike.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # --- rotate: queries and keys of a fused projection, normalised per head and rotated ---
        # the prompt of a full-attention layer (32 query heads on 8 key heads)
        dict(name="rotate_prompt_t8192", op="rotate", dtype="bf16", B=1, T=8192, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, fused=True, far=0),
        # the new tokens of a serving batch, far into their contexts: launch latency counts
        dict(name="rotate_decode_b64", op="rotate", dtype="bf16", B=64, T=1, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, fused=True, far=1 << 20),
        # fp32, adjacent pairs, half of the channels rotated, odd sizes
        dict(name="rotate_f32_t777", op="rotate", dtype="f32", B=2, T=777, Hq=6, Hkv=2, d=64, rot=32,
             interleaved=True, fused=False, far=4096),
        # --- rotate_train: forward and backward ------------------------------------------------
        # a training sequence; the weights' gradients sum over every token and head
        dict(name="rotate_train_t8192", op="rotate_train", dtype="bf16", B=1, T=8192, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, fused=True, far=0),
        # a small fp32 batch, every query head with its own key head
        dict(name="rotate_train_f32_t300", op="rotate_train", dtype="f32", B=3, T=100, Hq=4, Hkv=4, d=64, rot=64,
             interleaved=True, fused=False, far=0),
        # --- pages: page table, offsets and slots of a serving step from the requests' lengths --
        # prompts admitted beside running requests, more of them than there are pages for
        dict(name="pages_prompts", op="pages", N=64, held=2000, add=4096, page=64, short=True),
        # one token for each of a large batch
        dict(name="pages_decode_b256", op="pages", N=256, held=8000, add=1, page=16, short=False),
        # --- append: a prompt's part into the 4-bit cache, the whole context read back for its attention
        # a batch of prompts continuing 100 tokens each
        dict(name="mx4_append_prompts", op="append", dtype="bf16", B=8, T=4096, past=100, lo=1000, Hkv=8, d=128, page=64),
        # short odd prompts (one of them empty) in fp32
        dict(name="mx4_append_ragged_f32", op="append", dtype="f32", B=5, T=77, past=3, lo=0, Hkv=2, d=64, page=32),
        # --- decode: the last token(s) of every sequence over the 4-bit cache -------------------
        # a serving batch, full attention, contexts of 16 .. 8000 tokens: the largest
        dict(name="mx4_decode_b64_t8000", op="decode", dtype="bf16", B=64, T=8000, lo=16, Tq=1, Hq=32, Hkv=8, d=128,
             page=64, window=0, sinks=0),
        # a single long context: split over its length and joined
        dict(name="mx4_decode_b1_t32768", op="decode", dtype="bf16", B=1, T=32768, lo=32768, Tq=1, Hq=32, Hkv=8, d=128,
             page=32, window=0, sinks=0),
        # a short draft of 3 tokens verified, fp32, under a window, one context shorter than the draft
        dict(name="mx4_decode_verify_b3_t700", op="decode", dtype="f32", B=3, T=700, lo=2, Tq=3, Hq=4, Hkv=4, d=64,
             page=32, window=256, sinks=4),
    ]


def _log(rng, lo, hi):
    return min(hi, int(lo * math.exp(rng.random() * math.log(hi / lo + 1))))


def draw(rng):
    op = rng.choice(["rotate", "rotate_train", "pages", "append", "decode", "decode"])
    if op == "pages":
        add = rng.choice([1, 1, _log(rng, 2, 8192)])
        N = min(_log(rng, 1, 2048), (1 << 18) // add)
        return dict(op=op, N=N, held=_log(rng, 1, 8192), add=add, page=rng.choice([16, 32, 64, 128, 256]),
                    short=rng.random() < 0.3)
    dtype, d = rng.choice(["bf16", "bf16", "bf16", "f32"]), rng.choice([64, 128])
    Hq, Hkv = rng.choice([(4, 4), (8, 2), (6, 2), (16, 1), (32, 8), (32, 32), (12, 4), (5, 5)])
    if op in ("rotate", "rotate_train"):
        B, T = _log(rng, 1, 16), _log(rng, 1, 8192)
        T = max(1, min(T, (1 << 25) // (B * (Hq + Hkv) * d)))
        return dict(op=op, dtype=dtype, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2, 16, 48]),
                    interleaved=rng.random() < 0.5, fused=rng.random() < 0.5, far=rng.choice([0, _log(rng, 100, 1 << 20)]))
    if op == "append":
        T = _log(rng, 1, 8192)
        B = max(1, min(_log(rng, 1, 64), (1 << 25) // (T * Hkv * d)))
        return dict(op=op, dtype=dtype, B=B, T=T, past=rng.randint(0, 300), lo=rng.randint(0, T), Hkv=Hkv, d=d,
                    page=rng.choice([32, 64, 128, 256]))
    T = _log(rng, 1, 32768)
    B = max(1, min(_log(rng, 1, 128), (1 << 19) // T, (1 << 28) // (T * Hkv * d)))
    window = rng.choice([0, _log(rng, 16, 4096)])
    return dict(op=op, dtype=dtype, B=B, T=T, lo=rng.randint(1, T), Tq=rng.choice([1, 1, 1, rng.randint(2, 8)]), Hq=Hq,
                Hkv=Hkv, d=d, page=rng.choice([32, 64, 128, 256]), window=window,
                sinks=rng.choice([0, rng.randint(1, 8), rng.randint(1, 100)]) if window else 0)


def _lengths(case):
    """Lengths of a ragged batch, evenly from lo to T (the longest); prepare() permutes them."""
    B, lo, T = case["B"], case["lo"], case["T"]
    return [T - (T - lo) * i // max(1, B - 1) for i in range(B)]


def _requests(case):
    """(tokens held, tokens to add) of each request of a serving step: with add > 1 every second one is a new or
    continued prompt of up to `add` tokens, the others take one token."""
    N, held, add = case["N"], case["held"], case["add"]
    lens = [held * ((7 * i) % (N + 1)) // N for i in range(N)]
    if add == 1:
        return lens, [1] * N
    return ([0 if i % 4 == 0 else n for i, n in enumerate(lens)],
            [1 + (add - 1) * ((5 * i) % (N + 1)) // N if i % 2 == 0 else 1 for i in range(N)])


def _pages_of(case):
    """Pages of the requests before the step, pages they ask for, and what the free list holds."""
    lens, adds = _requests(case)
    page = case["page"]
    held = [-(-n // page) for n in lens]
    need = [-(-(n + a) // page) - h for n, a, h in zip(lens, adds, held)]
    return held, need, sum(need) * 4 // 5 if case["short"] else sum(need) + 5


def work(case):
    op = case["op"]
    if op == "pages":
        lens, adds = _requests(case)
        _, need, free = _pages_of(case)
        pages = tokens = 0
        for n, a in zip(need, adds):  # as far as the free pages go
            if pages + n > free:
                break
            pages, tokens = pages + n, tokens + a
        # lengths, additions; offsets, additions, lengths; pages taken and entered; slots
        return {"bytes": 4 * (5 * case["N"] + 3 + 2 * pages + tokens), "flops": 0}
    e, d, Hkv, B = (2 if case["dtype"] == "bf16" else 4), case["d"], case["Hkv"], case["B"]
    if op in ("rotate", "rotate_train"):
        rows, tokens = B * case["T"] * (case["Hq"] + Hkv), B * case["T"]
        byt = 2 * e * d * rows + 4 * tokens + 2 * case["rot"] + 8 * d
        flops = rows * (5 * d + 3 * case["rot"])
        if op == "rotate":
            return {"bytes": byt, "flops": flops}
        # the backward reads q, k and the gradients, and writes the inputs' and the weights'
        return {"bytes": byt + 3 * e * d * rows + 4 * tokens + 2 * case["rot"] + 16 * d,
                "flops": flops + rows * (14 * d + 3 * case["rot"])}
    coded = d // 2 + d // 32  # bytes of one position's and head's keys, or values, in the cache
    if op == "append":
        new, all_ = sum(_lengths(case)), sum(_lengths(case)) + case["past"] * B
        return {"bytes": 2 * Hkv * (new * (e * d + coded) + all_ * (coded + e * d)), "flops": 0}
    Hq, Tq, window, sinks = case["Hq"], case["Tq"], case["window"], case["sinks"]
    keys = pairs = 0
    for n in _lengths(case):
        lo = max(0, n - Tq - window + 1) if window else 0
        keys += n - lo + min(sinks, lo)
        for i in range(Tq):
            p = n - Tq + i
            if p >= 0:
                pairs += min(p + 1, window) + min(sinks, max(0, p + 1 - window)) if window else p + 1
    return {"bytes": 2 * Hkv * coded * keys + 2 * e * B * Tq * Hq * d, "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------- the 4-bit format


_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x):
    """fp32 [..., d] -> codes 0 .. 15 (uint8) [..., d], scale bytes [..., d / 32]."""
    x = x.unflatten(-1, (-1, 32))
    top = x.abs().amax(-1, keepdim=True)
    # exponent of the largest value, one more if its mantissa is above 7 / 4, less 2
    e = ((top.view(torch.int32) + 0x1FFFFF) >> 23).sub_(2).clamp_(1, 252)
    y = (x / (e << 23).view(torch.float32)).abs_()
    c = (y > 0.25).to(torch.uint8)
    c += y >= 0.75
    c += y > 1.25
    c += y >= 1.75
    c += y > 2.5
    c += y >= 3.5
    c += y > 5.0
    c += torch.signbit(x).to(torch.uint8) << 3
    return c.flatten(-2), e.squeeze(-1).to(torch.uint8)


def _value(codes, scales):
    """Codes [..., d] and scale bytes [..., d / 32] -> what they stand for in fp32."""
    table = torch.tensor(_MAGNITUDES + tuple(-x for x in _MAGNITUDES), device=codes.device)
    s = (scales.to(torch.int32) << 23).view(torch.float32)
    return (table[codes.int()].unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _pack_keys(c):
    """Codes [..., positions, d] -> bytes [..., positions, d / 2], the even channel in the low half."""
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _unpack_keys(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _pack_values(c):
    """Codes [..., positions, d] -> bytes [..., positions / 32, d, 16]: a channel's 32 positions, the even in the low half."""
    return _pack_keys(c.unflatten(-2, (-1, 32)).transpose(-1, -2))


def _unpack_values(b):
    return _unpack_keys(b).transpose(-1, -2).flatten(-3, -2)


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def ints(xs):
        return torch.tensor(xs, dtype=torch.int32, device=dev)

    st = dict(case=case)
    if op == "pages":
        lens, adds = _requests(case)
        held, need, free = _pages_of(case)
        order = torch.randperm(case["N"], generator=torch.Generator().manual_seed(seed)).tolist()
        lens, adds, held = ([x[i] for i in order] for x in (lens, adds, held))
        page, N = case["page"], case["N"]
        pages = torch.randperm(sum(held) + free, generator=torch.Generator().manual_seed(seed + 1)).tolist()
        width = max(-(-(n + a) // page) for n, a in zip(lens, adds)) + 1
        table = []
        for n in held:
            table.append(pages[:n] + [-1] * (width - n))
            pages = pages[n:]
        st.update(lengths=ints(lens), add=ints(adds), page_table=ints(table), free_pages=ints(pages or [0]),
                  n_free=ints([len(pages)]), cu=ints([0] * (N + 1)), added=ints([0] * N), lengths_out=ints([0] * N),
                  n_free_out=ints([0]), slots=ints([-1] * sum(adds)))
        return st
    dt, B, T, Hkv, d = _DTYPES[case["dtype"]], case["B"], case["T"], case["Hkv"], case["d"]
    if op in ("rotate", "rotate_train"):
        Hq, rot = case["Hq"], case["rot"]
        if case["fused"]:  # queries, keys and values side by side, as one projection writes them
            qkv = normal(B, T, Hq + 2 * Hkv, d).to(dt)
            q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        else:
            q, k = normal(B, T, Hq, d).to(dt), normal(B, T, Hkv, d).to(dt)
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device=dev, dtype=torch.int32)
        st.update(q=q, k=k, positions=first + torch.arange(T, device=dev, dtype=torch.int32),
                  inv_freq=(10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)).float(),
                  w_q=1 + 0.2 * normal(d), w_k=1 + 0.2 * normal(d))
        if op == "rotate_train":
            st.update(grad_q_out=normal(B, T, Hq, d).to(dt), grad_k_out=normal(B, T, Hkv, d).to(dt))
        return st
    page = case["page"]
    order = torch.randperm(B, generator=torch.Generator().manual_seed(seed)).tolist()
    rows = [_lengths(case)[i] for i in order]
    past = case["past"] if op == "append" else 0
    need = [-(-(n + past) // page) for n in rows]
    free = torch.randperm(sum(need) + 3, generator=torch.Generator().manual_seed(seed + 1)).tolist()
    width, table = max(1, max(need)), []
    for n in need:
        table.append(free[:n] + [-1] * (width - n))
        free = free[n:]
    spread = torch.exp(0.5 * normal(2, Hkv, 1, d))  # some channels are larger than others, the keys' more so
    kc, ks = _quantise(normal(sum(need) + 3, Hkv, page, d) * spread[0])
    vc, vs = _quantise(normal(sum(need) + 3, Hkv, page, d) * spread[1].sqrt())
    st.update(k_codes=_pack_keys(kc), k_scales=ks, v_codes=_pack_values(vc).contiguous(), v_scales=vs,
              page_table=ints(table), scale=d ** -0.5, rows=rows)
    if op == "decode":
        st.update(q=normal(B, case["Tq"], case["Hq"], d).to(dt), lengths=ints(rows))
    else:
        total = sum(rows)
        st.update(k=(normal(total, Hkv, d) * spread[0, :, 0]).to(dt), v=(normal(total, Hkv, d) * spread[1, :, 0].sqrt()).to(dt),
                  cu=ints([sum(rows[:i]) for i in range(B + 1)]), lengths=ints([past] * B),
                  cu_all=ints([sum(rows[:i]) + past * i for i in range(B + 1)]))
    return st


# ---------------------------------------------------------------- the library's operators


def _own(st):
    import gated_delta_rule_08_amd as gdr
    c = st["case"]
    if c["op"] == "pages":
        gdr.gdr_attn_plan_pages(st["lengths"], st["add"], st["free_pages"], st["n_free"], st["page_table"], c["page"],
                                st["cu"], st["added"], st["lengths_out"], st["n_free_out"], st["slots"])
        return {x: st[x] for x in ("page_table", "cu", "added", "lengths_out", "n_free_out", "slots")}
    if c["op"] in ("rotate", "rotate_train"):
        q, k, how = st["q"], st["k"], dict(w_q=st["w_q"], w_k=st["w_k"], interleaved=c["interleaved"])
        qo, ko = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k))
        gdr.gdr_attn_norm_rope(q, k, st["positions"], st["inv_freq"], qo, ko, **how)
        if c["op"] == "rotate":
            return {"q": qo, "k": ko}
        dq, dk, dwq, dwk = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k, st["w_q"], st["w_k"]))
        gdr.gdr_attn_norm_rope_backward(q, k, st["positions"], st["inv_freq"], st["grad_q_out"], st["grad_k_out"], dq, dk,
                                        grad_w_q=dwq, grad_w_k=dwk, **how)
        return {"q": qo, "k": ko, "grad_q": dq, "grad_k": dk, "grad_w_q": dwq, "grad_w_k": dwk}
    cache = st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], st["page_table"]
    if c["op"] == "append":
        gdr.gdr_attn_append_mx4(st["k"], st["v"], st["cu"], st["lengths"], *cache)
        k = torch.empty(sum(st["rows"]) + c["past"] * c["B"], *st["k"].shape[1:], dtype=st["k"].dtype, device=st["k"].device)
        v = torch.empty_like(k)
        gdr.gdr_attn_read_mx4(*cache, st["cu_all"], k, v)
        return {"k": k, "v": v}
    o = torch.empty_like(st["q"])
    gdr.gdr_attn_decode_mx4(st["q"], *cache, st["lengths"], o, window=c["window"], sinks=c["sinks"], scale=st["scale"])
    return {"o": o}


# ---------------------------------------------------------------- the plain forms


def _plain_pages(st):
    page, lens, add, table = st["case"]["page"], st["lengths"].long(), st["add"].long(), st["page_table"]
    width, most, free, n_free = table.shape[1], st["slots"].numel(), st["free_pages"], st["n_free"].long()
    held = (lens + page - 1) // page
    fine = (lens >= 0) & (add >= 0) & (lens + add <= width * page)
    need = torch.where(fine, (lens + add + page - 1) // page - held, 0)
    add = torch.where(fine, add, 0)
    fits = (need.cumsum(0) <= n_free) & (add.cumsum(0) <= most)  # true up to the first that does not fit
    need, add = need * fits, add * fits
    cu = torch.cat([torch.zeros_like(n_free), add.cumsum(0)])
    t = torch.arange(most, device=table.device)
    seq = torch.searchsorted(cu[1:], t, right=True).clamp_(max=lens.numel() - 1)
    pos = lens[seq] + t - cu[seq]
    at = pos // page
    taken = (need.cumsum(0) - need)[seq] + at - held[seq]  # how many pages are taken before this token's, if it is new
    at = at.clamp_(max=width - 1)
    here = torch.where(at >= held[seq], free[(n_free - 1 - taken).clamp_(0, free.numel() - 1)], table[seq, at])
    used = t < cu[-1]
    flat = torch.cat([table.reshape(-1), table.new_zeros(1)])
    flat[torch.where(used & (pos % page == 0), seq * width + at, table.numel())] = here
    st["page_table"].copy_(flat[:-1].view_as(table))
    st["slots"].copy_(torch.where(used, here * page + pos % page, st["slots"]))
    st["cu"].copy_(cu)
    st["added"].copy_(add)
    st["lengths_out"].copy_(lens + add)
    st["n_free_out"].copy_(n_free - need.sum())
    return {x: st[x] for x in ("page_table", "cu", "added", "lengths_out", "n_free_out", "slots")}


_EPS = 1e-6


def _turn(x, cos, sin, interleaved):
    """Each pair of the first 2 cos.shape[-1] channels of x [..., H, d] turned by its angle."""
    half = cos.shape[-1]
    pairs = x[..., :2 * half].unflatten(-1, (half, 2) if interleaved else (2, half)).movedim(-1 if interleaved else -2, 0)
    a, b = pairs[0] * cos - pairs[1] * sin, pairs[1] * cos + pairs[0] * sin
    return torch.cat([torch.stack([a, b], -1 if interleaved else -2).flatten(-2), x[..., 2 * half:]], -1)


def _plain_rotate(st):
    c = st["case"]
    angle = st["positions"][..., None].double() * st["inv_freq"].double()
    cos, sin = angle.cos().float()[..., None, :], angle.sin().float()[..., None, :]
    got = {}
    for name in ("q", "k"):
        x, w = st[name].float(), st["w_" + name]
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
        got[name] = _turn(x * r * w, cos, sin, c["interleaved"]).to(st[name].dtype)
        if c["op"] == "rotate_train":
            u = _turn(st["grad_%s_out" % name].float(), cos, -sin, c["interleaved"])
            x = x * r
            got["grad_w_" + name] = (u * x).double().sum((0, 1, 2)).float()
            u = u * w
            got["grad_" + name] = ((u - x * (u * x).mean(-1, keepdim=True)) * r).to(st[name].dtype)
    return got


def _cache_values(st, pages):
    """The fp32 keys and values [..., Hkv, page, d] of pages [...]."""
    return (_value(_unpack_keys(st["k_codes"][pages]), st["k_scales"][pages]),
            _value(_unpack_values(st["v_codes"][pages]), st["v_scales"][pages]))


def _plain_append(st):
    c = st["case"]
    page, table, cu = c["page"], st["page_table"].long(), st["cu"].long()
    row = torch.arange(st["k"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = st["lengths"].long()[seq] + row - cu[seq]
    at, slot = table[seq, pos // page], pos % page
    kc, ks = _quantise(st["k"].float())
    vc, vs = _quantise(st["v"].float())
    st["k_codes"][at, :, slot], st["k_scales"][at, :, slot], st["v_scales"][at, :, slot] = _pack_keys(kc), ks, vs
    wide = _unpack_values(st["v_codes"])  # one code to a byte, as two positions share one
    wide[at, :, slot] = vc
    st["v_codes"].copy_(_pack_values(wide))
    cu = st["cu_all"].long()
    row = torch.arange(row.numel() + c["past"] * c["B"], device=cu.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = row - cu[seq]
    at, slot = table[seq, pos // page], pos % page
    return {"k": _value(_unpack_keys(st["k_codes"][at, :, slot]), st["k_scales"][at, :, slot]).to(st["k"].dtype),
            "v": _value(wide[at, :, slot], st["v_scales"][at, :, slot]).to(st["v"].dtype)}


def _visible(pos, keys, window, sinks):
    """Truth values [..., queries, keys] of the mask for positions pos [..., queries]."""
    back = pos[..., :, None] - keys
    seen = back >= 0
    if window:
        seen &= (back < window) | (keys < sinks)
    return seen


def _plain_decode(st):
    c = st["case"]
    B, Tq, Hq, Hkv, d = c["B"], c["Tq"], c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    k, v = (x.permute(0, 2, 1, 3, 4).reshape(B * Hkv, -1, d) for x in _cache_values(st, st["page_table"].long().clamp(min=0)))
    keys = torch.arange(k.shape[1], device=k.device)
    pos = st["lengths"].long()[:, None] - Tq + torch.arange(Tq, device=k.device)
    # keys and values behind a sequence's last are of no one, whatever they hold
    seen = _visible(pos, keys, c["window"], c["sinks"]).reshape(B, 1, 1, Tq, -1).expand(B, Hkv, G, Tq, -1)
    q = st["q"].float().reshape(B, Tq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B * Hkv, G * Tq, d)
    p = torch.bmm(q, k.transpose(1, 2).contiguous()).mul_(st["scale"]).view(B, Hkv, G, Tq, -1).masked_fill(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total == 0, torch.ones_like(total), total))
    o = torch.bmm(p.view(B * Hkv, G * Tq, -1), v).view(B, Hkv, G, Tq, d).permute(0, 3, 1, 2, 4)
    return {"o": o.reshape(B, Tq, Hq, d).to(st["q"].dtype)}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return (_plain_pages if op == "pages" else _plain_append if op == "append" else _plain_decode if op == "decode"
            else _plain_rotate)(state)


# ---------------------------------------------------------------- the definition in float64


def _rotated(x, w, positions, inv_freq, interleaved):
    """x [B, T, H, d] in float64 through the norm and the rotation, the pairs as complex numbers."""
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + _EPS) * w
    half = inv_freq.numel()
    if interleaved:
        re, im = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
    else:
        re, im = y[..., :half], y[..., half:2 * half]
    angle = positions.double()[..., None] * inv_freq.double()
    z = torch.complex(re, im) * torch.polar(torch.ones_like(angle), angle)[:, :, None]
    turned = torch.stack([z.real, z.imag], -1).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1)


def _nearest(x):
    """x [n, Hkv, d] in float64 -> the nearest values of the 4-bit format."""
    x = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))  # m 2^e with m in [1/2, 1)
    e = torch.where(m > 0.875, e - 2, e - 3).clamp(-126, 125)
    y = torch.ldexp(x.abs(), -e).clamp(max=6.0)[..., None]
    even, odd = (y.new_tensor(_MAGNITUDES[i::2]) for i in (0, 1))
    de, ie = (y - even).abs().min(-1)
    do, io = (y - odd).abs().min(-1)
    y = torch.where(de <= do, even[ie], odd[io])
    return torch.ldexp(torch.where(x < 0, -y, y), e).flatten(-2)


def _page_rows(st, table, n, what, Hkv):
    """What the cache holds of a sequence's first n positions, in float64 [n, Hkv, d]."""
    pages = torch.tensor(table, device=st["page_table"].device)
    scale = torch.ldexp(torch.ones((), dtype=torch.float64, device=pages.device), st[what + "_scales"][pages].double() - 127)
    b = st[what + "_codes"][pages]
    if what == "k":
        low, high = b & 15, b >> 4
        c = torch.cat([low[..., None], high[..., None]], -1).reshape(*b.shape[:-1], -1)  # [pages, Hkv, page, d]
    else:
        low, high = b & 15, b >> 4  # [pages, Hkv, page / 32, d, 16]
        c = torch.cat([low[..., None], high[..., None]], -1).reshape(*b.shape[:-1], 32)
        c = c.permute(0, 1, 2, 4, 3).reshape(*b.shape[:2], -1, b.shape[3])
    mag = torch.tensor(_MAGNITUDES, dtype=torch.float64, device=pages.device)[(c & 7).long()]
    x = torch.where(c >= 8, -mag, mag) * scale.repeat_interleave(32, -1)
    return x.permute(0, 2, 1, 3).reshape(-1, Hkv, x.shape[-1])[:n]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "pages":
        lens, adds, page = st["lengths"].tolist(), st["add"].tolist(), case["page"]
        table, free = st["page_table"].tolist(), st["free_pages"].tolist()[:int(st["n_free"])]
        width, slots, cu, open_ = len(table[0]), [], [0], True
        for n in range(case["N"]):
            want = -(-(lens[n] + adds[n]) // page) - -(-lens[n] // page)
            open_ = open_ and want <= len(free) and len(slots) + adds[n] <= st["slots"].numel()
            if open_:
                for p in range(lens[n], lens[n] + adds[n]):
                    if p % page == 0:
                        table[n][p // page] = free.pop()
                    slots.append(table[n][p // page] * page + p % page)
            cu.append(len(slots))
        added = [b - a for a, b in zip(cu, cu[1:])]

        def ints(xs):
            return torch.tensor(xs, dtype=torch.int32)

        return {"page_table": ints(table).view(-1, width), "cu": ints(cu), "added": ints(added),
                "lengths_out": ints([a + b for a, b in zip(lens, added)]), "n_free_out": ints([len(free)]),
                "slots": ints(slots + [-1] * (st["slots"].numel() - len(slots)))}
    if op in ("rotate", "rotate_train"):
        got = {}
        for name in ("q", "k"):
            x, w = st[name].double(), st["w_" + name].double()
            if op == "rotate_train":
                x.requires_grad_(), w.requires_grad_()
            y = _rotated(x, w, st["positions"], st["inv_freq"], case["interleaved"])
            got[name] = y.detach()
            if op == "rotate_train":
                got["grad_" + name], got["grad_w_" + name] = torch.autograd.grad(y, (x, w), st["grad_%s_out" % name].double())
        return got
    Hkv, d, table = case["Hkv"], case["d"], st["page_table"].tolist()
    if op == "append":
        got = {}
        for what in ("k", "v"):
            new, parts = _nearest(st[what].double()), []
            for n in range(case["B"]):
                held = _page_rows(st, [p for p in table[n] if p >= 0], case["past"], what, Hkv) if case["past"] else new[:0]
                parts += [held, new[sum(st["rows"][:n]):sum(st["rows"][:n + 1])]]
            got[what] = torch.cat(parts)
        return got
    G, Tq = case["Hq"] // Hkv, case["Tq"]
    o = torch.zeros(case["B"], Tq, case["Hq"], d, dtype=torch.float64, device=st["q"].device)
    for b, n in enumerate(st["rows"]):
        k, v = (_page_rows(st, [p for p in table[b] if p >= 0], n, what, Hkv) for what in ("k", "v"))
        j = torch.arange(n, device=k.device)
        for i in range(Tq):
            p = n - Tq + i
            if p < 0:
                continue
            see = j <= p
            if case["window"]:
                see = see & ((j > p - case["window"]) | (j < case["sinks"]))
            for h in range(Hkv):
                s = torch.mv(k[:, h], st["q"][b, i, h * G].double()) if G == 1 else None
                s = s[None] if G == 1 else st["q"][b, i, h * G:(h + 1) * G].double() @ k[:, h].t().contiguous()
                w = torch.softmax((s * st["scale"]).masked_fill(~see, -math.inf), -1)
                o[b, i, h * G:(h + 1) * G] = w @ v[:, h].contiguous()
    return {"o": o}
