"""Backward of the rotation alone: queries and keys are not read, and how they lie is no reason to refuse the call."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_08_amd as gdr

HIP, MISAL = -7, -4


def test_library():
    if not os.path.exists(gdr.library_path()):
        from gated_delta_rule_08_amd import build
        build.build()
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; calls that are not refused would be launched")
    lib = gdr.load_library()
    p = [0x100000 * (i + 1) for i in range(10)]

    def call(flags, q, k, stride=0):
        at = [ctypes.c_void_p(x) for x in [q, k] + p[2:]]
        at[2] = at[3] = None
        return lib.gdr_attn_norm_rope_backward(1, flags, 8, 4, 2, 64, 32, 1e-6, stride, stride, 256, 128, *at, None, None, None, 0, None)

    for q, k in ((p[0] + 2, p[1]), (p[0], p[1] + 4), (0, 0)):
        assert call(2, q or None, k or None) == HIP
    assert call(0, p[0] + 2, p[1], 256) == MISAL and call(0, p[0], p[1] + 4, 256) == MISAL


@pytest.mark.gpu
def test_binding():
    from gpu_util import announce, ensure_built
    ensure_built()
    announce("unread queries")
    B, T, Hq, Hkv, d = 3, 5, 4, 2, 64
    g = torch.Generator().manual_seed(1)
    q = torch.randn(B, Hq, T, d + 1, generator=g).cuda()[..., 1:].transpose(1, 2)
    k = torch.randn(B, T, Hkv, 2 * d, generator=g).cuda()[..., ::2]
    gq, gk = torch.randn(B, T, Hq, d, generator=g).cuda(), torch.randn(B, T, Hkv, d, generator=g).cuda()
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1), torch.ones(32, device="cuda")
    got, want = ([torch.empty_like(x) for x in (gq, gk)] for _ in range(2))
    gdr.gdr_attn_norm_rope_backward(q, k, pos, freq, gq, gk, *got, norm=False)
    gdr.gdr_attn_norm_rope_backward(q.contiguous(), k.contiguous(), pos, freq, gq, gk, *want, norm=False)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and not torch.equal(got[0], gq)
    with pytest.raises(ValueError):
        gdr.gdr_attn_norm_rope_backward(q, k, pos, freq, gq, gk, *got)
