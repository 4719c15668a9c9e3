"""CPU-only: the sizes from which the serving calls refuse, at their borders, before any HIP call."""
import pytest

from quantized_delta_rule_gdn_amd import lib

BAD = lib.DAMP_ERR_INVALID_ARGUMENT
X = 0x100000   # never dereferenced: every case is settled on the host


def _linear_step(B, H, d):
    # (the readout off its alignment, so that a size that is taken still goes no further than the checks)
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


def _need(delta, B, T, H, d=64, dt=1, decay=0):
    return lib.load().fp32_prefill_workspace_bytes(delta, B, T, H, d, dt, decay)


@pytest.mark.parametrize("delta", [0, 1])
@pytest.mark.parametrize("B,T,H", [(1, 2 ** 31 - 1, 1), (1, 2 ** 30, 2), (2 ** 28, 2 ** 31 - 1, 64), (2 ** 21, 2 ** 22, 1), (2 ** 31 - 1, 2 ** 31 - 1, 65536),
                                   (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (1, 64, 65537), (3, 2 ** 24 * 64, 1)])
def test_prefill_workspace_is_0_where_the_call_refuses(delta, B, T, H):
    assert _need(delta, B, T, H) == 0
    L, call = lib.load(), [X, 4, H, 64, 64, X, X, None, B, T, X, X, X, 1, X, 0]
    st = L.fp32_delta_prefill(*call, X, X, X, 1 << 60, None) if delta else L.fp32_linear_prefill(*call, X, X, 1 << 60, None)
    assert st in (BAD, lib.DAMP_ERR_UNSUPPORTED), "what the size function calls invalid is refused"


@pytest.mark.parametrize("change", [dict(dt=2), dict(dt=-1), dict(decay=3), dict(decay=-1), dict(B=-1), dict(T=-1), dict(H=-1), dict(d=96)])
def test_prefill_workspace_of_invalid_arguments(change):
    for delta in (0, 1):
        assert _need(**{**dict(delta=delta, B=3, T=5000, H=2, d=128), **change}) == 0
    assert _need(1, 3, 5000, 2, 128, decay=2) == 0 and _need(0, 3, 5000, 2, 128, decay=2) > 0


def test_prefill_workspace_up_to_the_limits():
    """Just below the limits the size is the formula's: 41.5 KB a chunk and head, d^2 + 1 floats a segment and head."""
    chunk = 5 * 64 * 64 * 2 + 2 * 64 * 4
    assert _need(1, 1, 64 * (2 ** 24 - 2), 1) == (2 ** 24 - 1) * chunk
    assert _need(1, 1, 64 * 255, 65535) == 256 * 65535 * chunk
    assert _need(0, 1, 64 * 255, 65535) == 0                         # prompts alone fill the chip: none is cut
    T = 64 * (2 ** 24 - 2)
    length = (-(-T // 512) + 63) // 64 * 64
    assert _need(0, 1, T, 1, 128) == (T // length + 1) * (128 * 128 + 1) * 4
