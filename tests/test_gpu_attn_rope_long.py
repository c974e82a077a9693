"""Norm and rotation of as many rows as take 16 bytes a lane in bf16, on both sides of where that begins (32768 rows), with the
reference and the bounds of test_gpu_attn_rope.py."""
import pytest

from gpu_util import announce, ensure_built
from test_gpu_attn_rope import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 32), (64, 48), (64, 64), (128, 0), (128, 16), (128, 48), (128, 64),
                                   (128, 112), (128, 128)])
def test_many_rows(d, rot, il):
    announce("rope many rows %d %d il=%s" % (d, rot, il))
    run("bf16", (4096,), 6, 2, d, rot, il, fused=True)  # 32768 rows
    run("bf16", (4095,), 6, 2, d, rot, il, weights=rot != 16)  # 8 bytes a lane


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("il", [False, True])
def test_few_heads(d, il):
    """One and two heads: chunks end with the 32 tokens whose angles they hold."""
    announce("rope few heads %d il=%s" % (d, il))
    run("bf16", (40001,), 1, 0, d, d, il)
    run("bf16", (32771,), 0, 1, d, 48, il, norm=False, weights=False)
    run("bf16", (2, 8200), 1, 1, d, d // 2, il, fused=True, far=1 << 20)


@pytest.mark.parametrize("il", [False, True])
def test_many_heads_and_odd_tokens(il):
    announce("rope many heads il=%s" % il)
    run("bf16", (803,), 40, 1, 128, 96, il, fused=True)
    run("bf16", (33,), 1000, 24, 64, 16, il, weights=False)
