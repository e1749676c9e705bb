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
