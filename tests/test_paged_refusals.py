"""CPU checks of the paged-cache calls' limits and of what the binding refuses."""
import ctypes

import pytest

from test_paged_abi import ALL, calls, q3  # noqa: F401


@pytest.mark.parametrize("B", [1 << 26, (1 << 27) + 5, 2 ** 31 - 20, 2 ** 31 - 1])
def test_too_many_sequences_are_refused(q3, B):  # noqa: F811
    """Beyond 2^30 (sequence, query head) rows 32-bit coordinates end; near 2^31 sequences a scan over
    them would not."""
    for name, (st, msg) in calls(q3, B=B, ws_bytes=1 << 62).items():
        assert name in ALL and st == q3.ESHAPE and "2^30" in msg, (name, st, msg)


def test_many_sequences_pass_the_limit(q3):  # noqa: F811
    """(the next check is the workspace's, or the device's)"""
    for st, msg in calls(q3, B=(1 << 26) - 1, ws_bytes=16).values():
        assert "2^30" not in msg and st != q3.ESHAPE
