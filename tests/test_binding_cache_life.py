"""CPU-only: the binding of the calls on a shared and drafted cache. Sizes beyond 32 bits are refused, not
cut to their lower 32 bits (tensors without memory stand in for the long ones), a workspace that the binding
allocates lives until the call is back, and a given one is used and checked."""
import contextlib
import weakref

import pytest

torch = pytest.importorskip("torch")

from quantized_delta_rule_gdn_amd import lib  # noqa: E402


class Library:
    """Stands in for the shared library: sizes a workspace, and looks at it during the call."""

    def __init__(self):
        self.nbytes, self.calls, self.made, self.seen = 0, [], [], []

    def kv_free_pages_workspace_bytes(self, *a):
        return self.nbytes

    kv_tree_attention_workspace_bytes = kv_latent_attention_workspace_bytes = kv_free_pages_workspace_bytes

    def _call(self, *a):
        self.calls.append(a)
        live = [t for t in (r() for r in self.made) if t is not None]
        self.seen.append([(t.data_ptr(), t.numel()) for t in live if t.data_ptr() in a])
        return lib.DAMP_OK

    kv_fork_tables = kv_copy_pages = kv_compact = kv_free_pages = kv_tree_attention = _call
    kv_latent_append = kv_latent_attention = kv_latent_prompt_attention = _call


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(lib, "load", lambda: L)
    monkeypatch.setattr(lib, "_first", lambda t, *a: t.device)
    monkeypatch.setattr(lib, "_On", lambda *a: contextlib.nullcontext(None))
    return L


META, CPU = "meta", "cpu"


def _t(*shape, dtype=torch.int32, dev=META):
    return torch.empty(shape, dtype=dtype, device=dev)


def _b(*shape, dev=META):
    return _t(*shape, dtype=torch.bfloat16, dev=dev)


def _fork(n=2, free=3, blocks=4, pages=9, page=16):
    lib.kv_fork_tables(_t(n), _t(n), _t(2), _t(free), _t(2, blocks), _t(pages), page, _t(n), _t(n), _t(n), _t(1))


def _copy(n=2, pages=9, H=2, page=16, d=64):
    lib.kv_copy_pages(_t(n), _t(n), _b(pages, H, page, d), _b(pages, H, page, d))


def _keep(num=3, B=2, blocks=4, pages=9):
    lib.kv_compact(_t(num), _t(B + 1), _t(B), _t(B), _t(B, blocks), _b(pages, 16, 576), None, _t(B))


def _free(B=2, blocks=4, pages=9, page=16, dev=META, **more):
    lib.kv_free_pages(None, _t(B, dev=dev), _t(B, blocks, dev=dev), _t(pages, dev=dev), page, _t(pages, dev=dev), _t(1, dev=dev), **more)


def _tree(T=3, B=2, blocks=4, words=None, max_new=None, max_len=None, dev=META, **more):
    mask = None if words is None else _t(T, words, dtype=torch.int64, dev=dev)
    lib.kv_tree_attention(_b(T, 4, 64, dev=dev), _b(9, 2, 16, 64, dev=dev), _b(9, 2, 16, 64, dev=dev), _t(B, blocks, dev=dev), _t(B, dev=dev), _t(B + 1, dev=dev),
                          _b(T, 4, 64, dev=dev), mask=mask, max_new=max_new, max_len=max_len, **more)


def _latent(T=3, B=2, blocks=4, max_new=None, max_len=None, dev=META, **more):
    lib.kv_latent_attention(_b(T, 4, 288, dev=dev), _b(9, 16, 288, dev=dev), _t(B, blocks, dev=dev), _t(B, dev=dev), _b(T, 4, 256, dev=dev), 0.1, cu_new=_t(B + 1, dev=dev),
                            max_new=max_new, max_len=max_len, **more)


def _append(T=3, pages=9):
    lib.kv_latent_append(_b(T, 256), _b(T, 32), _t(T, dtype=torch.int64), _b(pages, 16, 288))


def _prompt(Tq=3, Tk=3, H=2, B=1):
    lib.kv_latent_prompt_attention(_b(Tq, H, 96), _b(Tk, H, 64), _b(Tk, 32), _b(Tk, H, 64), _t(B + 1), _b(Tq, H, 64), cu_k=_t(B + 1))


LONG = [
    (_fork, [dict(n=2 ** 31), dict(n=2 ** 32 + 2), dict(free=2 ** 32 + 3), dict(blocks=2 ** 32 + 4), dict(pages=2 ** 32 + 9)]),
    (_copy, [dict(n=2 ** 32 + 2), dict(pages=2 ** 32 + 9), dict(H=2 ** 32 + 2), dict(page=2 ** 32 + 16), dict(d=2 ** 32 + 64)]),
    (_keep, [dict(num=2 ** 32 + 3), dict(B=2 ** 32 + 2), dict(blocks=2 ** 32 + 4), dict(pages=2 ** 32 + 9)]),
    (_free, [dict(B=2 ** 32 + 2), dict(blocks=2 ** 32 + 4), dict(pages=2 ** 32 + 9)]),
    (_tree, [dict(T=2 ** 32 + 3), dict(B=2 ** 32 + 2), dict(blocks=2 ** 32 + 4), dict(words=2 ** 32 + 1)]),
    (_latent, [dict(T=2 ** 32 + 3), dict(B=2 ** 32 + 2), dict(blocks=2 ** 32 + 4)]),
    (_append, [dict(T=2 ** 32 + 3), dict(pages=2 ** 32 + 9)]),
    (_prompt, [dict(Tq=2 ** 32 + 3), dict(Tk=2 ** 32 + 3), dict(H=2 ** 32 + 2), dict(B=2 ** 32 + 1)])]


@pytest.mark.parametrize("call,long", LONG, ids=[c.__name__ for c, _ in LONG])
def test_sizes_of_more_than_32_bits_are_refused(library, call, long):
    call()
    assert len(library.calls) == 1
    for x in long:
        with pytest.raises(ValueError):
            call(**x)
    assert len(library.calls) == 1


def test_bounds_and_page_sizes_keep_their_sign(library):
    for call, at in ((_fork, 11), (_free, 7)):
        for page in (16 - 2 ** 32, 16 + 2 ** 32, -(2 ** 31) - 16, 2 ** 63 + 16, -5):
            call(page=page)
            assert -(2 ** 31) <= library.calls[-1][at] < 2 ** 31 and library.calls[-1][at] not in range(1, 32769), "the library refuses it"
    for call, at in ((_tree, 17), (_latent, 16)):
        call()
        assert library.calls[-1][at] == 64 and library.calls[-1][10 if call is _tree else 9] == 3
        call(max_len=2 ** 32 + 5)
        assert library.calls[-1][at] == 2 ** 30
        call(max_len=100 - 2 ** 32)
        assert library.calls[-1][at] < 0, "the library refuses a negative bound"
        call(blocks=2 ** 30)
        assert library.calls[-1][at] == 2 ** 30
        call(max_new=2 ** 32 + 1)
        assert library.calls[-1][10 if call is _tree else 9] == 3, "no more new tokens than rows"


def test_a_mask_must_hold_the_new_tokens(library):
    _tree(T=64, words=1)
    _tree(T=65, words=1, max_new=64)
    for x in (dict(T=65, words=1), dict(T=200, words=2, max_new=129)):
        with pytest.raises(ValueError, match="words"):
            _tree(**x)
    assert len(library.calls) == 2


CALLS = pytest.mark.parametrize("call", [_free, _tree, _latent], ids=["free", "tree", "latent"])


@pytest.fixture
def recorded(library, monkeypatch):
    empty = torch.empty

    def record(*a, **k):
        t = empty(*a, **k)
        if t.dtype == torch.uint8:
            library.made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(torch, "empty", record)
    library.nbytes = 4096
    return library


@CALLS
def test_a_workspace_made_for_a_call_lives_through_it(recorded, call):
    call(dev=CPU)
    assert [n for _, n in recorded.seen[0]] == [4096], "the workspace was gone when the call was made"
    assert recorded.made[-1]() is None, "the workspace outlived the call"
    recorded.nbytes = 0
    made = len(recorded.made)
    call(dev=CPU)
    assert len(recorded.made) == made, "a workspace where none is needed"


@CALLS
def test_a_given_workspace_is_used_and_checked(recorded, call):
    ws = torch.zeros(5000, dtype=torch.uint8)
    recorded.made.append(weakref.ref(ws))
    call(dev=CPU, workspace=ws)
    assert recorded.seen == [[(ws.data_ptr(), 5000)]] and len(recorded.made) == 1
    for bad in (ws[:4095], ws.to(torch.int8), ws[::2], 4096):
        with pytest.raises((ValueError, TypeError)):
            call(dev=CPU, workspace=bad)
    assert len(recorded.seen) == 1
