"""Argument checks of the operators around the attention layers, on the CPU: every call here is refused (or has
nothing to do) before any HIP call."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_08_amd as gdr

OK, NULL, SHAPE, UNSUP, MISAL, WS, ENUM, ALIAS = 0, -1, -2, -3, -4, -5, -6, -8
BIG = 2 ** 31 - 1
# fake, non-NULL, aligned "device" addresses
P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdr.library_path()):
        from gated_delta_rule_08_amd import build
        build.build()
    return gdr.load_library()


def swap(ptrs, i, value):
    ptrs = list(ptrs)
    ptrs[i] = value
    return ptrs


def off(p, n):
    return ctypes.c_void_p(p.value + n)


def test_norm_rope(lib):
    def call(dtype=1, flags=0, tokens=8, Hq=4, Hkv=2, d=64, rot=32, sq=256, sk=128, ptrs=P[:8]):
        return lib.gdr_attn_norm_rope(dtype, flags, tokens, Hq, Hkv, d, rot, 1e-6, sq, sk, *ptrs, None)

    assert call(dtype=2) == ENUM and call(flags=4) == ENUM and call(flags=-1) == ENUM
    for kw in (dict(tokens=-1), dict(Hq=-1), dict(Hkv=-1), dict(rot=-16), dict(sq=255), dict(sk=127), dict(sq=1 << 40),
               dict(sk=-128), dict(tokens=1 << 27), dict(Hq=1 << 16), dict(Hkv=1 << 16), dict(tokens=BIG, Hq=BIG)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(d=32), dict(d=96), dict(d=256), dict(rot=8), dict(rot=2), dict(rot=80), dict(flags=2)):
        assert call(**kw) == UNSUP, kw
    for i in (0, 1, 4, 5, 6, 7):  # the weights are optional
        assert call(ptrs=swap(P[:8], i, None)) == NULL, i
    for i in range(8):
        assert call(ptrs=swap(P[:8], i, off(P[i], 2))) == MISAL, i
    assert call(sq=260) == MISAL and call(dtype=0, sq=258) == MISAL and call(sk=132) == MISAL
    # in place where the input is dense
    assert call(sq=512, ptrs=swap(P[:8], 6, P[0])) == ALIAS and call(sk=512, ptrs=swap(P[:8], 7, P[1])) == ALIAS
    for kw in (dict(tokens=0), dict(Hq=0, Hkv=0)):
        assert call(ptrs=[None] * 8, sq=0, sk=0, **kw) == OK
    assert call(flags=2, ptrs=swap(swap(swap(P[:8], 2, None), 3, None), 0, None)) == NULL


def test_norm_rope_backward(lib):
    def call(dtype=1, flags=0, tokens=8, Hq=4, Hkv=2, d=64, rot=32, strides=(256, 128, 256, 128), ptrs=P[:12], ws=P[12], n=1 << 40):
        return lib.gdr_attn_norm_rope_backward(dtype, flags, tokens, Hq, Hkv, d, rot, 1e-6, *strides, *ptrs, ws, n, None)

    size = lib.gdr_attn_norm_rope_backward_workspace_bytes
    assert call(dtype=7) == ENUM and call(flags=8) == ENUM
    for kw in (dict(tokens=-1), dict(Hq=-2), dict(tokens=1 << 28), dict(strides=(255, 128, 256, 128)),
               dict(strides=(256, 128, 64, 128)), dict(strides=(256, 128, 256, 0))):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(d=80), dict(rot=24), dict(flags=2)):
        assert call(**kw) == UNSUP, kw
    for i in (0, 1, 4, 5, 6, 7, 8, 9):
        assert call(ptrs=swap(P[:12], i, None)) == NULL, i
    for i in range(12):
        assert call(ptrs=swap(P[:12], i, off(P[i], 2))) == MISAL, i
    assert call(ws=off(P[12], 8)) == MISAL
    need = size(1, 8, 4, 2, 64)
    assert need > 0 and call(ws=None) == WS and call(n=need - 1) == WS
    assert call(strides=(256, 128, 512, 128), ptrs=swap(P[:12], 8, P[6])) == ALIAS
    none = [None] * 12
    assert call(ptrs=none, tokens=0, ws=None, n=0) == OK and call(ptrs=none, Hq=0, Hkv=0, ws=None, n=0) == OK
    # without the norm neither q nor k is read, and there are no weights
    no_norm = [None] * 4 + P[4:10] + [None, None]
    assert call(flags=2, ptrs=swap(no_norm, 8, None), ws=None, n=0) == NULL
    for i in (2, 3, 10, 11):
        assert call(flags=2, ptrs=swap(no_norm, i, P[0])) == UNSUP
    for bad in ((5, 8, 4, 2, 64), (1, -8, 4, 2, 64), (1, 8, 4, 2, 65), (1, 0, 4, 2, 64), (1, 8, 0, 0, 64), (1, BIG, BIG, 2, 64)):
        assert size(*bad) == 0, bad
    # bounded by the workgroups, not by the rows
    assert size(1, 1 << 20, 32, 8, 128) <= 1 << 20


def test_outputs_that_are_other_tensors_are_refused(lib):
    def rope(ptrs, Hq=2, Hkv=2, flags=0):
        return lib.gdr_attn_norm_rope(1, flags, 8, Hq, Hkv, 64, 32, 1e-6, 128, 128, *ptrs, None)

    def back(ptrs, Hq=2, Hkv=2, flags=0):
        return lib.gdr_attn_norm_rope_backward(1, flags, 8, Hq, Hkv, 64, 32, 1e-6, 128, 128, 128, 128, *ptrs, P[12], 1 << 40, None)

    for out, other in ((6, 1), (6, 7), (7, 0)):  # q_out: k, k_out; k_out: q
        assert rope(swap(P[:8], out, P[other])) == ALIAS, (out, other)
    # grad_q: q, k, grad_k_out, grad_k; grad_k: q, k, grad_q_out; grad_w_k: grad_w_q
    for out, other in ((8, 0), (8, 1), (8, 7), (8, 9), (9, 0), (9, 1), (9, 6), (11, 10)):
        assert back(swap(P[:12], out, P[other])) == ALIAS, (out, other)
    for out, others in ((4, (0, 1, 2, 3, 5, 6, 7, 8, 9)), (5, (0, 1, 2, 3, 6, 7, 8, 9)), (6, (0, 2, 3, 7, 8, 9)),
                        (7, (1, 2, 3, 8, 9)), (8, (0, 1, 2, 3, 9)), (9, (0, 1, 2))):
        for other in others:
            assert lib.gdr_attn_plan_pages(4, 16, 8, 9, 100, *swap(P[:10], out, P[other]), None) == ALIAS, (out, other)
    append, read = cache_calls(lib)
    assert read(ptrs=swap(P[:9], 8, P[7])) == ALIAS
    for out, other in ((6, 4), (7, 5), (4, 0), (4, 1), (6, 0), (6, 1)):
        assert append(ptrs=swap(P[:9], out, P[other])) == ALIAS, (out, other)


def test_plan_pages(lib):
    def call(N=4, page=16, width=8, stack=9, tokens=100, ptrs=P[:10]):
        return lib.gdr_attn_plan_pages(N, page, width, stack, tokens, *ptrs, None)

    for kw in (dict(N=-1), dict(N=BIG), dict(width=-1), dict(width=1 << 28), dict(stack=-1), dict(tokens=-1)):
        assert call(**kw) == SHAPE, kw
    for page in (0, -16, 3, 48, 1 << 17):
        assert call(page=page) == UNSUP
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 9):  # the slots are optional
        assert call(ptrs=swap(P[:10], i, None)) == NULL, i
    for i in range(10):
        assert call(ptrs=swap(P[:10], i, off(P[i], 2))) == MISAL, i


def cache_calls(lib):
    def append(dtype=1, N=2, total=8, Hkv=2, d=64, page=32, pages=8, width=4, ptrs=P[:9]):
        return lib.gdr_attn_append_mx4(dtype, N, total, Hkv, d, page, pages, width, *ptrs, None)

    def read(dtype=1, N=2, total=8, Hkv=2, d=64, page=32, pages=8, width=4, ptrs=P[:9]):
        return lib.gdr_attn_read_mx4(dtype, N, total, Hkv, d, page, pages, width, *ptrs, None)

    return append, read


def test_append_and_read(lib):
    append, read = cache_calls(lib)
    for call, optional in ((append, ()), (read, (6,))):
        assert call(dtype=2) == ENUM
        for kw in (dict(N=-1), dict(total=-1), dict(total=BIG), dict(Hkv=-1), dict(Hkv=1 << 16), dict(pages=-1), dict(width=-1),
                   dict(width=1 << 27), dict(pages=1 << 26), dict(total=1 << 28)):
            assert call(**kw) == SHAPE, kw
        for kw in (dict(d=32), dict(d=192), dict(page=16), dict(page=1), dict(page=48), dict(page=0), dict(page=1 << 17)):
            assert call(**kw) == UNSUP, kw
        for i in range(9):
            if i not in optional:
                assert call(ptrs=swap(P[:9], i, None)) == NULL, i
            assert call(ptrs=swap(P[:9], i, off(P[i], 2))) == MISAL, i
        for kw in (dict(N=0), dict(total=0), dict(Hkv=0), dict(pages=0), dict(width=0)):
            assert call(ptrs=[None] * 9, **kw) == OK, kw


def test_decode(lib):
    def call(dtype=1, B=2, Tq=1, Hq=4, Hkv=2, d=64, page=32, pages=8, width=4, window=0, sinks=0, ptrs=P[:8], ws=P[9], n=1 << 40):
        return lib.gdr_attn_decode_mx4(dtype, B, Tq, Hq, Hkv, d, page, pages, width, window, sinks, 1.0, *ptrs, ws, n, None)

    size = lib.gdr_attn_decode_mx4_workspace_bytes
    assert call(dtype=3) == ENUM
    for kw in (dict(B=-1), dict(Tq=-1), dict(Hq=-4), dict(Hq=5), dict(pages=-1), dict(width=-1), dict(window=-1), dict(sinks=-1),
               dict(B=BIG), dict(width=1 << 28), dict(pages=1 << 27), dict(Hq=1 << 16, Hkv=1 << 16), dict(B=1 << 22, Hq=64),
               dict(B=256, width=(1 << 26) - 128, page=32)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(d=192), dict(page=16), dict(page=33), dict(page=1 << 17), dict(Tq=65)):
        assert call(**kw) == UNSUP, kw
    for i in range(8):
        assert call(ptrs=swap(P[:8], i, None)) == NULL, i
        assert call(ptrs=swap(P[:8], i, off(P[i], 2))) == MISAL, i
    for kw in (dict(B=0), dict(Tq=0), dict(Hq=0, Hkv=0), dict(pages=0), dict(width=0)):
        assert call(ptrs=[None] * 8, ws=None if "pages" not in kw else P[9], **kw) == OK, kw
    need = size(1, 2, 1, 4, 2, 64, 32, 100, 0, 0)
    assert need > 0 and call(width=100, ws=None) == WS and call(width=100, n=need - 1) == WS
    assert call(width=100, ws=off(P[9], 8)) == MISAL
    assert size(1, 2, 1, 4, 2, 64, 32, 16, 0, 0) == 0 and size(1, 2, 1, 4, 2, 64, 32, 17, 0, 0) > 0
    assert size(1, 2, 1, 4, 2, 64, 32, 1000, 300, 4) == 0
    for bad in ((7, 2, 1, 4, 2, 64, 32, 100, 0, 0), (1, 2, 65, 4, 2, 64, 32, 100, 0, 0), (1, 2, 1, 4, 3, 64, 32, 100, 0, 0),
                (1, 2, 1, 4, 2, 64, 16, 100, 0, 0), (1, 0, 1, 4, 2, 64, 32, 100, 0, 0), (1, 2, 1, 4, 2, 64, 32, 100, -1, 0)):
        assert size(*bad) == 0, bad


# ---------------------------------------------------------------- the binding


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_binding_refuses():
    q, k, pos, freq = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64), ints(5), torch.ones(16)
    good = dict(q=q, k=k, positions=pos, inv_freq=freq, q_out=q.clone(), k_out=k.clone())
    for bad in (dict(k=torch.zeros(4, 2, 64)), dict(k=torch.zeros(5, 2, 128)), dict(positions=ints(4)), dict(q_out=k), dict(k_out=q),
                dict(positions=pos.long()), dict(inv_freq=freq.double()), dict(inv_freq=torch.ones(4, 4)), dict(k=k.bfloat16()),
                dict(w_q=torch.ones(32)), dict(w_k=torch.ones(64).bfloat16()), dict(q=q.half(), k=k.half())):
        with pytest.raises(ValueError):
            gdr.gdr_attn_norm_rope(**{**good, **bad})
    with pytest.raises(ValueError, match="GPU"):
        gdr.gdr_attn_norm_rope(**good)
    with pytest.raises(ValueError, match="gradient shapes"):
        gdr.gdr_attn_norm_rope_backward(q, k, pos, freq, k, k, q, k)
    lens, table, cu = ints(3), ints(3, 4), ints(4)
    plan = dict(lengths=lens, add=lens, free_pages=ints(9), n_free=ints(1), page_table=table, page_size=16, cu_seqlens=cu,
                added=lens, lengths_out=lens, n_free_out=ints(1))
    for bad in (dict(add=ints(2)), dict(cu_seqlens=ints(3)), dict(n_free=ints(2)), dict(page_table=ints(12)), dict(added=lens.long()),
                dict(slots=ints(2, 2)), dict(n_free_out=ints(1).float()), dict(free_pages=ints(3, 3))):
        with pytest.raises(ValueError):
            gdr.gdr_attn_plan_pages(**{**plan, **bad})
    with pytest.raises(ValueError, match="GPU"):
        gdr.gdr_attn_plan_pages(**plan)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    cache = dict(k_codes=u8(6, 2, 64, 32), k_scales=u8(6, 2, 64, 2), v_codes=u8(6, 2, 2, 64, 16), v_scales=u8(6, 2, 64, 2),
                 page_table=table)
    x = torch.zeros(7, 2, 64)
    append = lambda **kw: gdr.gdr_attn_append_mx4(**{**cache, **dict(k=x, v=x, cu_seqlens=cu, lengths=lens), **kw})  # noqa: E731
    read = lambda **kw: gdr.gdr_attn_read_mx4(**{**cache, **dict(k=x, v=x, cu_seqlens=cu), **kw})  # noqa: E731
    decode = lambda **kw: gdr.gdr_attn_decode_mx4(**{**cache, **dict(q=torch.zeros(3, 4, 64), o=torch.zeros(3, 4, 64), lengths=lens), **kw})  # noqa: E731
    for call in (append, read, decode):
        for bad in (dict(k_codes=u8(6, 2, 64, 64)), dict(k_scales=u8(6, 2, 64, 4)), dict(v_codes=u8(6, 2, 64, 32)),
                    dict(v_scales=u8(5, 2, 64, 2)), dict(v_scales=ints(6, 2, 64, 2)), dict(page_table=ints(2, 4)),
                    dict(page_table=ints(12)), dict(k_codes=u8(6, 64, 32))):
            with pytest.raises(ValueError):
                call(**bad)
        with pytest.raises(ValueError, match="GPU"):
            call()
    for bad in (dict(lengths=ints(4)), dict(cu_seqlens=ints(3)), dict(v=x[:6]), dict(k=x[:, :1], v=x[:, :1])):
        with pytest.raises(ValueError):
            append(**bad)
    for bad in (dict(first=ints(2)), dict(first=lens.long()), dict(v=x.double()), dict(k=x[0])):
        with pytest.raises(ValueError):
            read(**bad)
    for bad in (dict(q=torch.zeros(3, 5, 64)), dict(o=torch.zeros(3, 4, 128)), dict(lengths=lens.long()), dict(q=torch.zeros(4, 64))):
        with pytest.raises(ValueError):
            decode(**bad)


def test_token_strides():
    """Views whose tokens are evenly apart pass their stride; others are refused."""
    s = gdr._token_stride
    qkv = torch.zeros(3, 5, 8, 64)
    assert s("q", qkv[:, :, :4], 4, 64) == 512
    assert s("q", qkv[:, :, 4:6], 2, 64) == 512
    assert s("q", qkv, 8, 64) == 512
    assert s("q", qkv[:, :1, :4], 4, 64) == 5 * 512  # one token of each sequence
    assert s("q", qkv[1:2, 2:3, :4], 4, 64) == 256
    assert s("q", torch.zeros(0, 4, 64), 4, 64) == 256
    for bad in (qkv[:, :4, :4], qkv[:, ::2, :4], qkv.transpose(1, 2)[:, :4], qkv[..., ::2], qkv[:, :, ::2], qkv.transpose(0, 1)):
        with pytest.raises(ValueError):
            s("q", bad, bad.shape[-2], bad.shape[-1])
