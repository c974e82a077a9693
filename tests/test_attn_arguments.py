"""Arguments of the attention entry points at the ends of their ranges, on the CPU: every call here ends before any
HIP call."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_08_amd as gdr

OK, NULL, SHAPE = 0, -1, -2
BIG = 2 ** 31 - 1
P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(8)]  # fake, aligned addresses


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdr.library_path()):
        from gated_delta_rule_08_amd import build
        build.build()
    return gdr.load_library()


def test_a_loose_bound_of_the_queries_is_no_error(lib):
    """max_q is any upper bound: what it says beyond total_q sizes nothing."""
    def call(mq, tq=8, q=None, N=2):
        return lib.gdr_attn_prefill_varlen(1, N, tq, 8, mq, 32, 8, 64, 0, 0, 1.0, q, *P[1:7], None)

    for mq in (8, 9, 1 << 24, 1 << 29, BIG):
        assert call(mq) == NULL, mq  # past the sizes, at the missing q
        assert call(mq, tq=0) == OK, mq
    assert call(-1) == SHAPE and call(BIG, tq=BIG) == SHAPE


def test_integers_beyond_32_bits_keep_their_meaning(lib):
    """A window far beyond the keys is no window, one far below 0 is refused; neither becomes its low 32 bits."""
    size = gdr.gdr_attn_backward_workspace_bytes
    args = (torch.bfloat16, 1, 9000, 9000, 8, 2, 64)
    full, narrow = size(*args), size(*args, 1000)
    assert full > 0 and narrow > 0 and full != narrow
    for window in (9000, BIG, 2 ** 32 + 1000, 2 ** 40):
        assert size(*args, window) == full, window
    for window in (-1, -2 ** 31, -2 ** 32, -2 ** 32 + 1000, -2 ** 40):
        assert size(*args, window) == 0, window
    assert size(*args, 1000, -2 ** 32) == 0
    for i in range(1, 7):  # sizes
        assert size(*args[:i], 2 ** 32 + args[i], *args[i + 1:]) == 0, i
    pages = (torch.bfloat16, 2, 8, 2, 64, 16, 1024)
    assert gdr.gdr_attn_decode_workspace_bytes(*pages) > 0
    for i in range(1, 7):
        assert gdr.gdr_attn_decode_workspace_bytes(*pages[:i], 2 ** 32 + pages[i], *pages[i + 1:]) == 0, i
    assert gdr._attn_int(2 ** 32 + 5) == BIG and gdr._attn_int(-2 ** 32 + 5) == -1 and gdr._attn_int(5) == 5


def test_calls_pass_their_integers_whole(monkeypatch):
    """What the binding hands to the library for the window, the sinks and the bound of a packed call."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, args)) or 0

    monkeypatch.setattr(gdr, "load_library", Lib)
    monkeypatch.setattr(gdr, "_attn_device", lambda *ts: 0)
    monkeypatch.setattr(gdr, "_attn_launch", lambda dev, stream, fn, *args: fn(*args))
    q, k, o = torch.zeros(8, 4, 64), torch.zeros(8, 2, 64), torch.zeros(8, 4, 64)
    cu = torch.tensor([0, 8], dtype=torch.int32)
    gdr.gdr_attn_prefill_varlen(q, k, k, cu, cu, o, max_seqlen_q=2 ** 32 + 2, window=-2 ** 32, sinks=2 ** 33)
    name, args = seen.pop()
    assert name == "gdr_attn_prefill_varlen" and args[4] == BIG and args[8] == -1 and args[9] == BIG


def test_a_workspace_is_recorded_on_the_stream_of_its_own_device(monkeypatch):
    """A stream given as a handle belongs to the tensors' device, whichever device is current."""
    made = []

    class Stream:
        cuda_stream = 77

    class Tensor:
        def record_stream(self, s):
            made.append("recorded")

    def external(handle, device=None):
        made.append((handle, device))
        return Stream()

    current = type("Current", (), {"cuda_stream": 0})
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: Tensor())
    device = torch.device("cuda", 1)
    gdr._workspace(16, device, 77)
    assert made == [(77, device), "recorded"]


def test_handle_0_is_the_default_stream(monkeypatch):
    """The workspace of a call on handle 0 is recorded on the default stream where another one is current."""
    recorded = []

    class Tensor:
        def record_stream(self, s):
            recorded.append(s)

    default, current = (type("Stream", (), {"cuda_stream": n}) for n in (0, 9))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: default)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: type("Pool", (), {"cuda_stream": 5}))
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: Tensor())
    gdr._workspace(16, torch.device("cuda", 0), 0)
    assert recorded == [default]
