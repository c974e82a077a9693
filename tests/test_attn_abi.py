"""Argument checks of the attention entry points, on the CPU: every call here is refused (or has nothing to
do) before any HIP call."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_08_amd as gdr

OK, NULL, SHAPE, UNSUP, MISAL, WS, ENUM = 0, -1, -2, -3, -4, -5, -6
BIG = 2 ** 31 - 1
# fake, non-NULL, aligned "device" addresses
P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(12)]


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


def prefill(lib, dtype=1, B=1, Tq=8, Tk=8, Hq=4, Hkv=2, d=64, window=0, sinks=0, ptrs=P[:5]):
    return lib.gdr_attn_prefill(dtype, B, Tq, Tk, Hq, Hkv, d, window, sinks, 1.0, *ptrs, None)


def test_prefill(lib):
    assert prefill(lib, dtype=2) == ENUM
    for kw in (dict(B=-1), dict(Tq=-1), dict(Tk=-1), dict(Hq=-1), dict(Hkv=-1), dict(window=-1), dict(sinks=-1),
               dict(Hq=5), dict(Hkv=0), dict(Hq=0), dict(Tq=BIG), dict(Tk=BIG), dict(Tq=1 << 28, Hq=32), dict(B=BIG, Hq=64, Hkv=64),
               dict(B=1 << 20, Tq=1 << 20), dict(Hq=1 << 16, Hkv=1 << 16), dict(Tq=1 << 27), dict(Tk=1 << 28)):
        assert prefill(lib, **kw) == SHAPE, kw
    for d in (0, 16, 63, 96, 256, -64):
        assert prefill(lib, d=d) == UNSUP
    for i in range(4):  # lse is optional
        assert prefill(lib, ptrs=swap(P[:5], i, None)) == NULL
        assert prefill(lib, ptrs=swap(P[:5], i, off(P[i], 8))) == MISAL
    assert prefill(lib, ptrs=swap(P[:5], 4, off(P[4], 2))) == MISAL
    for kw in (dict(B=0), dict(Tq=0), dict(Hq=0, Hkv=0)):
        assert prefill(lib, ptrs=[None] * 5, **kw) == OK
    assert prefill(lib, Tk=0, ptrs=[P[0], None, None, None, None]) == NULL  # o
    # more workgroups than one launch can have
    assert prefill(lib, B=40_000_000, Tq=1, Tk=1, Hq=2, Hkv=1) == SHAPE


def test_prefill_varlen(lib):
    def call(dtype=1, N=2, tq=8, tk=8, mq=8, Hq=4, Hkv=2, d=64, window=0, sinks=0, ptrs=P[:7]):
        return lib.gdr_attn_prefill_varlen(dtype, N, tq, tk, mq, Hq, Hkv, d, window, sinks, 1.0, *ptrs, None)

    assert call(dtype=-1) == ENUM
    for kw in (dict(N=-1), dict(tq=-1), dict(tk=-1), dict(mq=-1), dict(Hq=3), dict(window=-2), dict(tq=BIG), dict(tk=BIG)):
        assert call(**kw) == SHAPE, kw
    assert call(d=32) == UNSUP
    for i in range(6):
        assert call(ptrs=swap(P[:7], i, None)) == NULL
        assert call(ptrs=swap(P[:7], i, off(P[i], 2))) == MISAL
    for kw in (dict(N=0), dict(tq=0), dict(mq=0), dict(Hq=0, Hkv=0)):
        assert call(ptrs=[None] * 7, **kw) == OK


def test_backward(lib):
    def call(dtype=1, B=1, Tq=8, Tk=8, Hq=4, Hkv=2, d=64, window=0, sinks=0, ptrs=P[:9], ws=P[9], n=1 << 40):
        return lib.gdr_attn_backward(dtype, B, Tq, Tk, Hq, Hkv, d, window, sinks, 1.0, *ptrs, ws, n, None)

    size = lib.gdr_attn_backward_workspace_bytes
    assert call(dtype=9) == ENUM
    for kw in (dict(B=-1), dict(Tq=-1), dict(Tk=-1), dict(Hq=3), dict(sinks=-1), dict(Tq=BIG), dict(Tk=BIG)):
        assert call(**kw) == SHAPE, kw
    assert call(d=100) == UNSUP
    for i in range(9):
        assert call(ptrs=swap(P[:9], i, None)) == NULL
        assert call(ptrs=swap(P[:9], i, off(P[i], 2))) == MISAL
    assert call(ws=off(P[9], 8)) == MISAL
    need = size(1, 1, 8, 8, 4, 2, 64, 0, 0)
    assert need > 0 and call(ws=None) == WS and call(n=need - 1) == WS
    for kw in (dict(B=0), dict(Hq=0, Hkv=0), dict(Tq=0, Tk=0)):
        assert call(ptrs=[None] * 9, ws=None, n=0, **kw) == OK
    # key heads without query heads would leave their gradients unwritten
    assert call(Hq=0) == SHAPE
    # few key blocks, long lists of rows for the sinks' keys: room for those, not for every key
    for T, heads in ((60000, 1), (16384, 2), (65536, 4), (4096, 1)):
        for sinks in (1, 4, 200):
            assert size(1, 1, T, T, heads, heads, 128, 64, sinks) < 400 << 20, (T, heads, sinks)
    # sinks under a window need room for their partial sums; without a window they hide nothing
    assert size(1, 1, 65536, 65536, 4, 2, 64, 128, 4) > size(1, 1, 65536, 65536, 4, 2, 64, 128, 0)
    assert size(1, 1, 65536, 65536, 4, 2, 64, 0, 4) == size(1, 1, 65536, 65536, 4, 2, 64, 0, 0)
    assert size(1, 1, 65536, 65536, 4, 2, 64, 65536, 4) == size(1, 1, 65536, 65536, 4, 2, 64, 0, 0)
    for bad in ((5, 1, 8, 8, 4, 2, 64, 0, 0), (1, -1, 8, 8, 4, 2, 64, 0, 0), (1, 1, 8, 8, 4, 3, 64, 0, 0),
                (1, 1, 8, 8, 4, 2, 80, 0, 0), (1, 1, BIG, 8, 4, 2, 64, 0, 0), (1, 1, 0, 8, 4, 2, 64, 0, 0)):
        assert size(*bad) == 0, bad


def test_decode(lib):
    def call(dtype=1, B=2, Hq=4, Hkv=2, d=64, page=16, pages=8, width=4, window=0, sinks=0, ptrs=P[:8], ws=P[9], n=1 << 40):
        return lib.gdr_attn_decode(dtype, B, Hq, Hkv, d, page, pages, width, window, sinks, 1.0, *ptrs, ws, n, None)

    size = lib.gdr_attn_decode_workspace_bytes
    assert call(dtype=3) == ENUM
    for kw in (dict(B=-1), dict(Hq=-4), dict(Hq=5), dict(pages=-1), dict(width=-1), dict(window=-1), dict(sinks=-1),
               dict(B=BIG), dict(width=1 << 28), dict(B=256, width=(1 << 27) - 1024), dict(pages=1 << 27), dict(pages=1 << 26, page=16, Hkv=4)):
        assert call(**kw) == SHAPE, kw
    assert call(d=192) == UNSUP
    for page in (0, -16, 3, 24, 1 << 17):
        assert call(page=page) == UNSUP
    for i in range(8):
        assert call(ptrs=swap(P[:8], i, None)) == NULL
        assert call(ptrs=swap(P[:8], i, off(P[i], 2))) == MISAL
    for kw in (dict(B=0), dict(Hq=0, Hkv=0), dict(pages=0), dict(width=0)):
        assert call(ptrs=[None] * 8, **kw) == OK
    need = size(1, 1, 8, 2, 128, 16, 1024, 0, 0)
    assert need > 0 and size(1, 1, 8, 2, 128, 16, 1024, 64, 0) < need  # a window bounds the parts
    long = dict(B=1, Hq=8, d=128, width=1024, pages=2000)
    assert call(ws=None, **long) == WS and call(n=need - 1, **long) == WS and call(ws=off(P[9], 4), **long) == MISAL
    assert size(1, 1, 8, 2, 128, 16, 2, 0, 0) == 0                     # short rows are one part
    for bad in ((7, 1, 8, 2, 128, 16, 1024, 0, 0), (1, 1, 8, 3, 128, 16, 1024, 0, 0), (1, 1, 8, 2, 128, 12, 1024, 0, 0),
                (1, 1, 8, 2, 128, 16, -1, 0, 0), (1, 1, 8, 2, 128, 16, 1 << 30, 0, 0)):
        assert size(*bad) == 0, bad


def test_append(lib):
    def call(dtype=1, N=2, total=10, Hkv=2, d=64, page=16, pages=8, width=4, ptrs=P[:7]):
        return lib.gdr_attn_append(dtype, N, total, Hkv, d, page, pages, width, *ptrs, None)

    assert call(dtype=2) == ENUM
    for kw in (dict(N=-1), dict(total=-1), dict(Hkv=-1), dict(pages=-1), dict(width=-3), dict(total=BIG), dict(pages=1 << 29)):
        assert call(**kw) == SHAPE, kw
    assert call(d=8) == UNSUP and call(page=48) == UNSUP
    for i in range(7):
        assert call(ptrs=swap(P[:7], i, None)) == NULL
        assert call(ptrs=swap(P[:7], i, off(P[i], 2))) == MISAL
    for kw in (dict(N=0), dict(total=0), dict(Hkv=0), dict(pages=0), dict(width=0)):
        assert call(ptrs=[None] * 7, **kw) == OK


def test_binding_refuses_what_does_not_fit():
    q, k, v, o = torch.zeros(1, 4, 4, 64), torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 4, 64)
    with pytest.raises(ValueError, match="GPU"):
        gdr.gdr_attn_prefill(q, k, v, o)
    with pytest.raises(ValueError, match="GPU"):
        gdr.gdr_attn_backward(q, k, v, o, torch.zeros(1, 4, 4), q, q, k, v)
    for bad in ((q[0], k[0], v[0], o[0]), (q, k, v[:, :3], o), (q, k, v, o[..., :32]), (q, k.expand(2, 4, 2, 64), v.expand(2, 4, 2, 64), o),
                (q, k.bfloat16(), v, o), (q.half(), k.half(), v.half(), o.half()), (q[:, :, :3], k, v, o[:, :, :3])):
        with pytest.raises(ValueError):
            gdr.gdr_attn_prefill(*bad)
    with pytest.raises(ValueError, match="lse"):
        gdr.gdr_attn_prefill(q, k, v, o, torch.zeros(1, 4, 2))
    with pytest.raises(ValueError, match="gradient"):
        gdr.gdr_attn_backward(q, k, v, o, torch.zeros(1, 4, 4), q, k, k, v)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="cu_k"):
        gdr.gdr_attn_prefill_varlen(q[0], k[0], v[0], cu, cu.long(), o[0])
    with pytest.raises(ValueError, match="cu_k"):
        gdr.gdr_attn_prefill_varlen(q[0], k[0], v[0], cu, torch.zeros(3, dtype=torch.int32), o[0])
    pages, table, lens = torch.zeros(3, 2, 16, 64), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    d = (q[:, 0], k[:, 0], v[:, 0])
    with pytest.raises(ValueError, match="GPU"):
        gdr.gdr_attn_decode(*d, pages, pages, table, lens, o[:, 0])
    with pytest.raises(ValueError, match="pages"):
        gdr.gdr_attn_decode(*d, pages[:, :1], pages[:, :1], table, lens, o[:, 0])
    with pytest.raises(ValueError, match="page_table"):
        gdr.gdr_attn_decode(*d, pages, pages, table.expand(2, 2), lens, o[:, 0])
    with pytest.raises(ValueError, match="lengths"):
        gdr.gdr_attn_decode(*d, pages, pages, table, lens.long(), o[:, 0])
    with pytest.raises(ValueError, match="cu_seqlens"):
        gdr.gdr_attn_append(k[0], v[0], lens, lens, pages, pages, table)
    with pytest.raises(ValueError, match="share dtype"):
        gdr.gdr_attn_append(k[0], v[0], cu, lens, pages.bfloat16(), pages.bfloat16(), table)
