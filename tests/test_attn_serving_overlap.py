"""Buffers that share memory, in the calls around the attention layers: refused before any HIP call where an output would
lie in another tensor, wholly or in part; accepted where it takes its own input's place or fits between the rows of a view."""
import ctypes
import os
import random

import pytest
import torch

import gated_delta_rule_08_amd as gdr

HIP, ALIAS, APART = -7, -8, 1 << 24
BASE = 1 << 40  # fake device addresses, never read: accepted calls end at the launch, which fails without a GPU


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdr.library_path()):
        from gated_delta_rule_08_amd import build
        build.build()
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; calls that are not refused would be launched")
    return gdr.load_library()


def spaced(sizes, gap=0):
    """Addresses of tensors of these bytes one right behind another (16-byte aligned)."""
    out, at = [], BASE
    for n in sizes:
        out.append(at)
        at += (n + 15) // 16 * 16 + gap
    return out


def probe(call, sizes, outs, own):
    """call(addresses) is accepted with tensors one behind another, and refused as soon as an output's first or last bytes,
    and no more, lie in another tensor, or another's lie in it."""
    good = spaced(sizes)
    assert call(good, APART) == HIP and call(good, 0) == HIP
    for o in outs:
        for x in range(len(sizes)):
            if x == o:
                continue
            moved = list(good)
            moved[o] = good[x]
            want = HIP if own.get(o) == x else ALIAS
            assert call(apart_but(moved, sizes, o, x), APART) == want, (o, x)
            assert call(apart_but(moved, sizes, o, x), 0) == want, (o, x)
            # one 16-byte unit in common, at either end
            for at in (good[x] + (sizes[x] - 1) // 16 * 16, good[x] - (sizes[o] - 1) // 16 * 16):
                if at == good[x]:
                    continue
                moved[o] = at
                assert call(apart_but(moved, sizes, o, x), APART) == ALIAS, (o, x, at - good[x])
                assert call(apart_but(moved, sizes, o, x), 0) == HIP, (o, x)


def apart_but(addresses, sizes, o, x):
    """The others out of the way of o and x."""
    far = (max(addresses[i] + sizes[i] for i in (o, x)) // 16 + 1) * 16 + (1 << 20)
    out = []
    for i, a in enumerate(addresses):
        if i not in (o, x):
            a, far = far, far + (sizes[i] + 15) // 16 * 16
        out.append(a)
    return out


@pytest.mark.parametrize("rot", [64, 32])
def test_norm_rope(lib, rot):
    T, Hq, Hkv, d = 5, 4, 2, 64
    sizes = [T * Hq * d * 2, T * Hkv * d * 2, 4 * d, 4 * d, 4 * T, 2 * rot, T * Hq * d * 2, T * Hkv * d * 2]

    def call(p, flag):
        return lib.gdr_attn_norm_rope(1 | flag, 0, T, Hq, Hkv, d, rot, 1e-6, Hq * d, Hkv * d, *map(ctypes.c_void_p, p), None)

    probe(call, sizes, (6, 7), {6: 0, 7: 1})
    # q and k one tensor: neither output may take its place
    p = spaced(sizes)
    same = lib.gdr_attn_norm_rope(1 | APART, 0, T, 2, 2, d, rot, 1e-6, 2 * d, 2 * d, *map(ctypes.c_void_p, [p[1]] * 2 + p[2:6] + [p[1], p[7]]), None)
    assert same == ALIAS


def test_norm_rope_backward(lib):
    T, Hq, Hkv, d, rot = 3, 2, 1, 64, 48
    q, k, w = T * Hq * d * 2, T * Hkv * d * 2, 4 * d
    need = lib.gdr_attn_norm_rope_backward_workspace_bytes(1, T, Hq, Hkv, d)
    sizes = [q, k, w, w, 4 * T, 2 * rot, q, k, q, k, w, w, need]

    def call(p, flag, flags=0, weights=True):
        p = [ctypes.c_void_p(x) for x in p]
        if flags:
            p[2] = p[3] = p[10] = p[11] = None
        return lib.gdr_attn_norm_rope_backward(1 | flag, flags, T, Hq, Hkv, d, rot, 1e-6, Hq * d, Hkv * d, Hq * d, Hkv * d, *p,
                                               need, None)

    probe(call, sizes, (8, 9, 10, 11, 12), {8: 6, 9: 7})
    p = spaced(sizes)
    for o in (8, 9):  # q and k are not read without the norm
        for x in (0, 1):
            at = list(p)
            at[o] = p[x]
            assert call(apart_but(at, sizes, o, x), APART, flags=2) == HIP


def test_plan_pages(lib):
    N, page, width, stack, tokens = 9, 16, 5, 40, 77
    sizes = [4 * N, 4 * N, 4 * stack, 4, 4 * N * width, 4 * N + 4, 4 * N, 4 * N, 4 * tokens, 4]

    def call(p, flag):
        return lib.gdr_attn_plan_pages(N, page | flag, width, stack, tokens, *map(ctypes.c_void_p, p), None)

    probe(call, sizes, (4, 5, 6, 7, 8, 9), {6: 1, 7: 0, 9: 3})
    p = spaced([4, 4, 4])
    for a, b in ((0, 0), (0, 1)):  # no requests: the offsets' first and the pages left are written all the same
        r = lib.gdr_attn_plan_pages(0, page | APART, 0, 0, 0, None, None, None, ctypes.c_void_p(p[2]), None, ctypes.c_void_p(p[a]),
                                    None, None, None, ctypes.c_void_p(p[b]), None)
        assert r == (ALIAS if a == b else HIP)


def test_cache_calls(lib):
    N, total, Hkv, d, page, pages, width = 3, 10, 2, 64, 32, 4, 6
    rows, dense = pages * Hkv * page, total * Hkv * d * 4
    cache = [rows * d // 2, rows * d // 32, rows * d // 2, rows * d // 32]

    def append(p, flag):
        return lib.gdr_attn_append_mx4(0 | flag, N, total, Hkv, d, page, pages, width, *map(ctypes.c_void_p, p), None)

    probe(append, [dense, dense, 4 * N + 4, 4 * N] + cache + [4 * N * width], (4, 5, 6, 7), {})

    def read(p, flag):
        return lib.gdr_attn_read_mx4(0 | flag, N, total, Hkv, d, page, pages, width, *map(ctypes.c_void_p, p), None)

    probe(read, cache + [4 * N * width, 4 * N + 4, 4 * N, dense, dense], (7, 8), {})
    B, Tq, Hq, wide = 3, 2, 4, 200
    need = lib.gdr_attn_decode_mx4_workspace_bytes(1, B, Tq, Hq, Hkv, d, page, wide, 0, 0)
    assert need > 0

    def decode(p, flag):
        return lib.gdr_attn_decode_mx4(1 | flag, B, Tq, Hq, Hkv, d, page, pages, wide, 0, 0, 0.1, *map(ctypes.c_void_p, p), need, None)

    probe(decode, [B * Tq * Hq * d * 2] + cache + [4 * B * wide, 4 * B, B * Tq * Hq * d * 2, need], (7, 8), {7: 0})


def rows_of(p, width, stride, T):
    return [(p + i * stride, p + i * stride + width) for i in range(T)]


def meet(a, b):
    return any(x < v and u < y for x, y in a for u, v in b)


def test_views(lib):
    """Rows of a fused projection, against every pair of rows: outputs that interleave are accepted, ones that touch are not."""
    r = random.Random(5)
    seen = {True: 0, False: 0}
    for case in range(4000):
        T, Hq, Hkv, d = r.choice([1, 2, 3, 7]), r.choice([1, 2]), r.choice([1, 2, 3]), 64
        wq, wk = Hq * d, Hkv * d
        wide = r.choice([wq + wk, wq + 2 * wk, 3 * (wq + wk), 1000 * d])
        # grad_q and grad_k somewhere in one buffer; the others far away
        sq = r.choice([wide, wide, wide, wq, wq + d])
        sk = r.choice([wide, wide, wide, wk, 2 * wide, wk + 2 * d])
        step = r.choice([8, d, wq, wide])
        gq, gk = (BASE + 2 * step * r.randrange(0, max(2, 3 * wide // step)) for _ in range(2))
        far = [BASE + (1 << 30) + (i << 22) for i in range(8)]
        p = far + [gq, gk, None, None, None]
        got = lib.gdr_attn_norm_rope_backward(1 | APART, 0, T, Hq, Hkv, d, 64, 1e-6, wq, wk, sq, sk,
                                              *[ctypes.c_void_p(x) for x in p], 0, None)
        want = meet(rows_of(gq, 2 * wq, 2 * sq, T), rows_of(gk, 2 * wk, 2 * sk, T))
        assert got == (ALIAS if want else HIP), (case, T, Hq, Hkv, wide, sq, sk, gq - BASE, gk - BASE)
        seen[want] += 1
        # a dense output beside the rows of a view that is read
        p = [gq, far[1], None, None, far[2], far[3], gk, far[5]]
        got = lib.gdr_attn_norm_rope(1 | APART, 0, T, Hkv, 0, d, 64, 1e-6, max(wk, sk), 0, *[ctypes.c_void_p(x) for x in p], None)
        rows = rows_of(gq, 2 * wk, 2 * max(wk, sk), T)
        want = meet(rows, [(gk, gk + 2 * wk * T)])
        own = gq == gk and (max(wk, sk) == wk)
        if gq == gk and T == 1 and not own:
            continue  # one token: its stride says nothing
        assert got == (ALIAS if want and not own else HIP), (case, T, Hkv, sk, gq - BASE, gk - BASE)
        seen[want] += 1
    assert min(seen.values()) > 1000


def test_the_largest_sizes_do_not_overflow(lib):
    """Tables and stacks whose bytes leave 64 bits or fill the address space."""
    big = 2 ** 31 - 4097
    p = [ctypes.c_void_p(BASE + (i << 36)) for i in range(10)]
    for flag in (0, APART):
        r = lib.gdr_attn_plan_pages(2 ** 31 - 2, 1 | flag, big, 2 ** 31 - 1, 2 ** 31 - 1, *p, None)
        assert r == (ALIAS if flag else HIP)
        r = lib.gdr_attn_append_mx4(flag, 2 ** 31 - 1, 5, 1, 64, 32, 4, big // 32, *p[:9], None)
        assert r in (HIP, -2)
    p = [ctypes.c_void_p(BASE + (i << 42)) for i in range(10)]
    p[4] = ctypes.c_void_p(BASE + (1 << 47))
    r = lib.gdr_attn_plan_pages(2 ** 31 - 2, 1 | APART, 16, 2 ** 31 - 1, 2 ** 31 - 1, *p, None)
    assert r == HIP
