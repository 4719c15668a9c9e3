"""CPU-only: a workspace that the binding allocates for a call lives until that call is back. The C call
runs without the interpreter's lock, so memory that were freed before it could be given to another
thread's call on the same stream, and be written between this call's launches."""
import contextlib
import weakref

import pytest

torch = pytest.importorskip("torch")

from quantized_delta_rule_gdn_amd import lib  # noqa: E402


class Library:
    """Stands in for the shared library: sizes a workspace, and looks at it during the call."""

    def __init__(self, nbytes):
        self.nbytes, self.made, self.seen = nbytes, [], []

    def fp32_prefill_workspace_bytes(self, *a):
        return self.nbytes

    kv_decode_attention_workspace_bytes = fp32_prefill_workspace_bytes

    def _call(self, *a):
        live = [t for t in (r() for r in self.made) if t is not None]
        self.seen.append([(t.data_ptr(), t.numel()) for t in live if t.data_ptr() in a])
        return lib.DAMP_OK

    fp32_linear_prefill = fp32_delta_prefill = kv_decode_attention = _call


@pytest.fixture
def library(monkeypatch):
    L, empty = Library(4096), torch.empty

    def recorded(*a, **k):
        t = empty(*a, **k)
        L.made.append(weakref.ref(t))
        return t

    cpu = torch.device("cpu")
    monkeypatch.setattr(lib, "load", lambda: L)
    monkeypatch.setattr(lib, "_first", lambda *a: cpu)
    monkeypatch.setattr(lib, "_On", lambda *a: contextlib.nullcontext(None))
    yield L, lambda: monkeypatch.setattr(torch, "empty", recorded)


def _prefill(delta, **more):
    H, d, T = 2, 16, 5
    x = [torch.zeros((T, H, d), dtype=torch.bfloat16) for _ in range(4)]
    one = torch.zeros(1, dtype=torch.int32)
    head = (torch.zeros((1, H, d, d)), one, torch.tensor([0, T], dtype=torch.int32), *x[:3], torch.ones((T, H)))
    return (lambda: lib.fp32_delta_prefill(*head, torch.ones((T, H)), x[3], **more)) if delta else (lambda: lib.fp32_linear_prefill(*head, x[3], **more))


def _attention(**more):
    q, p = torch.zeros((1, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    t, n, out = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.zeros_like(q)
    return lambda: lib.kv_decode_attention(q, p, p.clone(), t, n, out, **more)


CALLS = pytest.mark.parametrize("make", [lambda **k: _prefill(0, **k), lambda **k: _prefill(1, **k), _attention], ids=["linear", "delta", "attention"])


@CALLS
def test_a_workspace_made_for_a_call_lives_through_it(library, make):
    L, record = library
    call = make()
    record()
    call()
    assert len(L.seen) == 1 and [n for _, n in L.seen[0]] == [4096], "the workspace was gone when the call was made"
    assert L.made[-1]() is None, "the workspace outlived the call"


@CALLS
def test_a_given_workspace_is_used_and_checked(library, make):
    L, record = library
    ws = torch.zeros(5000, dtype=torch.uint8)
    call = make(workspace=ws)
    record()
    L.made.append(weakref.ref(ws))
    call()
    assert L.seen == [[(ws.data_ptr(), 5000)]] and len(L.made) == 1
    for bad in (ws[:4095], ws.to(torch.int8), ws[::2]):
        with pytest.raises((ValueError, TypeError)):
            make(workspace=bad)()
    with pytest.raises(TypeError):
        make(workspace=4096)()
    assert len(L.seen) == 1


@CALLS
def test_no_workspace_where_none_is_needed(library, make):
    L, record = library
    L.nbytes = 0
    call = make()
    record()
    call()
    assert L.seen == [[]] and not L.made
