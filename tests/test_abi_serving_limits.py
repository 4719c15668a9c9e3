"""CPU-only: the sizes from which the serving calls refuse, at their borders, before any HIP call."""
import ctypes

import pytest

from quantized_delta_rule_gdn_amd import lib

BAD = lib.DAMP_ERR_INVALID_ARGUMENT
X = 0x100000   # never dereferenced: every case is settled on the host


def _linear_step(B, H, d):
    # (a slot list off its alignment, so that a size that is taken still goes no further than the checks)
    return lib.load().fp32_linear_step(X, 4, H, d, d, X, B, X, X, X, 1, X, 0, X + 4, None)


@pytest.mark.parametrize("d,limit", [(16, 2 ** 26), (32, 2 ** 26), (64, 2 ** 24), (128, 2 ** 24)])
def test_linear_step_stays_below_the_launch_limit(d, limit):
    """One workgroup a state, of 64 threads (d of 16 and 32) or 256: less than 2^32 threads."""
    L = lib.load()
    for B, H in ((limit, 1), (1, limit), (limit // 16, 16), (2 ** 31 - 1, 1), (limit // 2, 3)):
        st = L.fp32_linear_step(X, 4, H, d, d, X, B, X, X, X, 1, X, 0, X, None)
        assert st == BAD and "grid limit" in lib.last_error(), (B, H)
    for B, H in ((limit - 1, 1), (1, limit - 1), (3, limit // 3)):
        assert _linear_step(B, H, d) == BAD and "16-byte" in lib.last_error(), (B, H)
