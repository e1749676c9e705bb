"""The paged cache's operators where they can go wrong: refused calls, lists, scales, values at the
ends of the types' ranges. Tolerances: see test_gpu_paged.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from helpers import assert_device_ok, rope_gpu  # noqa: E402,F401
from test_gpu_paged import Case, f64  # noqa: E402,F401

D = 128


@pytest.fixture(scope="module")
def q3():
    import qwen3_decoder_block_b200 as m
    return m


def test_a_refused_attention_call_leaves_nothing_on_the_stream(q3):
    """A row stride that no tensor map can hold is refused; the call's own plan kernel, which would
    report the negative context, must not have been launched."""
    c = Case(q3, [1], [40], 16)
    c.t_ctx.fill_(-1)
    c.ldq = 1 << 39
    with pytest.raises(q3.Qwen3Error, match="ldq"):
        c.attend()
    assert q3.check_device_error() == q3.OK


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("qlens", [[1, 1], [200, 1], [1] * 17 + [40]])
def test_workspace_at_any_16_bytes(q3, qlens, fp8):
    """A workspace may begin at any multiple of 16 bytes."""
    c = Case(q3, qlens, [700 + 13 * b for b in range(len(qlens))], 32, fp8=fp8, seed=3)
    c.darken()
    n = q3.workspace_size(c.cfg, q3.OP_ATTENTION_PAGED, len(qlens), max(qlens), 1)
    whole = torch.full((n + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    assert whole.data_ptr() % 256 == 0
    for at in (16, 48, 112, 240):
        o = c.attend(ws=whole[at:at + n])
        assert_device_ok()
        c.check(o)
        assert (whole[:at] == 0xAB).all() and (whole[at + n:] == 0xAB).all()
        whole.fill_(0xAB)
