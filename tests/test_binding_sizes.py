"""CPU-only: sizes beyond 32 bits are refused by the binding of the paged cache, not cut to their lower 32
bits on their way into the library (tensors without memory stand in for the long ones)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from quantized_delta_rule_gdn_amd import lib  # noqa: E402


class Library:
    def __init__(self):
        self.calls = []

    def kv_decode_attention_workspace_bytes(self, *a):
        return 0

    def kv_build_tables(self, *a):
        self.calls.append(a)
        return lib.DAMP_OK

    kv_decode_attention = kv_build_tables


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(lib, "load", lambda: L)
    monkeypatch.setattr(lib, "_first", lambda t, *a: t.device)
    monkeypatch.setattr(lib, "_On", lambda *a: contextlib.nullcontext(None))
    return L


def _meta(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="meta")


def _tables(T=5, free=7, blocks=3, page=16):
    return lib.kv_build_tables(_meta(1), _meta(1), _meta(free), _meta(1, blocks), page, _meta(T, dtype=torch.int64), None, _meta(2), _meta(1))


def test_tables_of_more_than_32_bits_are_refused(library):
    _tables()
    assert len(library.calls) == 1
    for x in (dict(T=2 ** 32 + 3), dict(T=2 ** 31), dict(free=2 ** 32 + 1), dict(blocks=2 ** 32 + 2), dict(blocks=2 ** 31)):
        with pytest.raises(ValueError):
            _tables(**x)
    assert len(library.calls) == 1
    for page in (16 - 2 ** 32, 16 + 2 ** 32, -(2 ** 31) - 16, 2 ** 63 + 16, -5, 2 ** 31 - 1):
        _tables(page=page)
        got = library.calls[-1][5]
        assert -(2 ** 31) <= got < 2 ** 31 and got not in range(1, 32769), "the library refuses it"


def _attention(blocks=3, max_len=None):
    q = _meta(2, 4, 64, dtype=torch.bfloat16)
    p = _meta(9, 2, 16, 64, dtype=torch.bfloat16)
    lib.kv_decode_attention(q, p, p, _meta(2, blocks), _meta(2), torch.empty_like(q), max_len=max_len)


def test_attention_bounds_of_more_than_32_bits(library):
    _attention()
    assert library.calls[-1][11:13] == (3, 48)
    _attention(blocks=2 ** 30)
    assert library.calls[-1][11:13] == (2 ** 30, 2 ** 30)
    for n in (100 - 2 ** 32, -1, -(2 ** 63) + 7):
        _attention(max_len=n)
        assert library.calls[-1][12] < 0, "the library refuses a negative bound"
    _attention(max_len=2 ** 32 + 5)
    assert library.calls[-1][12] == 2 ** 30
    n = len(library.calls)
    with pytest.raises(ValueError):
        _attention(blocks=2 ** 32 + 1)
    assert len(library.calls) == n


def test_workspace_sizes_of_more_than_32_bits():
    """The size functions see what the calls would: sizes beyond 32 bits raise, a length bound stops at 2^30."""
    for x in (2 ** 32 + 1, 2 ** 31, -(2 ** 32) + 1):
        for n in ((x, 5000, 2, 64), (1, x, 2, 64), (1, 5000, x, 64), (1, 5000, 2, x)):
            with pytest.raises(ValueError):
                lib.prefill_workspace_bytes(True, *n, torch.bfloat16)
        for n in ((x, 4, 2, 64, 5000), (1, x, 2, 64, 5000), (1, 4, x, 64, 5000), (1, 4, 2, x, 5000)):
            with pytest.raises(ValueError):
                lib.kv_decode_attention_workspace_bytes(*n)
    size = lib.kv_decode_attention_workspace_bytes
    assert size(1, 4, 2, 64, 2 ** 32 + 5) == size(1, 4, 2, 64, 2 ** 40) == size(1, 4, 2, 64, 2 ** 30) > 0
    assert size(1, 4, 2, 64, 5000 - 2 ** 32) == 0
