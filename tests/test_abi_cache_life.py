"""CPU-only checks of the host side of the calls on a shared and drafted cache (forked tables, copies, kept
tokens, pages given back, attention of several tokens, latents): statuses and messages of every refusal, the
no-ops, and the workspace sizes, all before any HIP call."""
import ctypes

import pytest

from quantized_delta_rule_gdn_amd import lib

OK, BAD, UNSUP = lib.DAMP_OK, lib.DAMP_ERR_INVALID_ARGUMENT, lib.DAMP_ERR_UNSUPPORTED
X = 0x100000   # never dereferenced: every case is settled on the host
Y, Z = X + 2 ** 26, X + 2 ** 27


def _call(name, base, **change):
    assert not set(change) - set(base)
    return getattr(lib.load(), name)(*{**base, **change}.values())


def _refused(name, base, change, status, text):
    assert _call(name, base, **change) == status and text in lib.last_error(), lib.last_error()


FORK = dict(src=X, dst=X, n=0, lens=X, B=2, free=X, num_free=3, table=X, blocks=4, shares=X, pages=9, page=16, cs=X, cd=X, cr=X, used=X, stream=None)


@pytest.mark.parametrize("change,status,text", [
    (dict(n=-1), BAD, ">= 0"), (dict(B=-1), BAD, ">= 0"), (dict(num_free=-1), BAD, ">= 0"), (dict(blocks=-1), BAD, ">= 0"), (dict(pages=0), BAD, "num_pages"),
    (dict(page=24), UNSUP, "power of two"), (dict(page=65536), UNSUP, "power of two"), (dict(pages=2 ** 31 - 1, page=16), UNSUP, "2^32"), (dict(n=8001), UNSUP, "8000"),
    (dict(used=None), BAD, "NULL"), (dict(free=None), BAD, "NULL"), (dict(used=X + 2), BAD, "misaligned"),
    *[(dict(n=1, **{k: None}), BAD, "NULL") for k in ("src", "dst", "lens", "table", "shares", "cs", "cd", "cr")],
    *[(dict(n=1, **{k: X + 1}), BAD, "misaligned") for k in ("src", "dst", "lens", "free", "table", "shares", "cs", "cd", "cr")]])
def test_fork_refusals(change, status, text):
    _refused("kv_fork_tables", FORK, change, status, text)


COPY = dict(src=X, dst=X, rows=None, n=1, k=X, v=X, pages=9, H=2, page=16, d=64, stream=None)


@pytest.mark.parametrize("change,status,text", [
    (dict(n=-1), BAD, "n"), (dict(H=0), BAD, "positive"), (dict(d=0), UNSUP, "multiples of 8"), (dict(d=12), UNSUP, "multiples of 8"), (dict(d=2056), UNSUP, "multiples of 8"),
    (dict(page=3), UNSUP, "power of two"), (dict(pages=2 ** 28, H=16), UNSUP, "2^32"), (dict(src=None), BAD, "NULL"), (dict(dst=None), BAD, "NULL"), (dict(k=None), BAD, "NULL"),
    (dict(k=X + 8), BAD, "16-byte"), (dict(v=X + 8), BAD, "16-byte"), (dict(src=X + 2), BAD, "4-byte"), (dict(rows=X + 2), BAD, "4-byte"),
    (dict(n=2 ** 31 - 1, H=2), BAD, "launch limit"), (dict(n=2 ** 30, page=32768, d=2048, H=1), BAD, "launch limit")])
def test_copy_refusals(change, status, text):
    _refused("kv_copy_pages", COPY, change, status, text)
    assert _call("kv_copy_pages", COPY, n=0, src=None, k=None) == OK


KEEP = dict(kept=X, cu=X, num=5, lens=X, new=X, B=2, table=X, blocks=4, k=X, v=None, pages=9, H=2, page=16, d=64, out=Y, stream=None)


@pytest.mark.parametrize("change,status,text", [
    (dict(num=-1), BAD, "num_kept"), (dict(num=2 ** 30 + 1), BAD, "num_kept"), (dict(B=-1), BAD, "B"), (dict(blocks=-1), BAD, "max_blocks"), (dict(d=4), UNSUP, "multiples of 8"),
    (dict(H=-1), BAD, "positive"), (dict(page=0), UNSUP, "power of two"), *[(dict([(k, None)]), BAD, "NULL") for k in ("kept", "cu", "lens", "new", "table", "k", "out")],
    *[(dict([(k, X + 2)]), BAD, "4-byte") for k in ("kept", "cu", "lens", "new", "table", "out")], (dict(k=X + 8), BAD, "16-byte"), (dict(v=X + 4), BAD, "16-byte"),
    (dict(B=2 ** 24, H=2, out=X + 2 ** 30), BAD, "grid limit"), (dict(out=X), BAD, "overlaps"), (dict(out=X + 4), BAD, "overlaps"), (dict(out=X - 4), BAD, "overlaps"),
    (dict(lens=Z, new=Z, cu=Z, out=X + 16), BAD, "overlaps")])
def test_keep_refusals(change, status, text):
    _refused("kv_compact", KEEP, change, status, text)
    assert _call("kv_compact", KEEP, B=0, cu=None, lens=None) == OK


FREE = dict(keep=None, lens=X, B=2, table=X, blocks=4, shares=X, pages=70000, page=16, freed=Y, count=Z, ws=X, wsn=1 << 40, stream=None)


@pytest.mark.parametrize("change,status,text", [
    (dict(B=-1), BAD, "B"), (dict(blocks=-1), BAD, "max_blocks"), (dict(pages=0), BAD, "num_pages"), (dict(page=6), UNSUP, "power of two"),
    *[(dict([(k, None)]), BAD, "NULL") for k in ("lens", "table", "shares", "freed", "count")],
    *[(dict([(k, X + 2)]), BAD, "misaligned") for k in ("keep", "lens", "table", "shares", "freed", "count")],
    (dict(B=2 ** 24), BAD, "grid limit"), (dict(ws=None), BAD, "workspace"), (dict(ws=X + 8), BAD, "workspace"), (dict(wsn=16), BAD, "workspace"), (dict(freed=X + 4 * 69999), BAD, "overlap"),
    (dict(count=X + 400), BAD, "overlap"), (dict(count=Y), BAD, "overlap")])
def test_free_refusals(change, status, text):
    _refused("kv_free_pages", FREE, change, status, text)


def test_free_workspace_sizes():
    size = lib.load().kv_free_pages_workspace_bytes
    assert [size(n) for n in (-1, 0, 1, 8192)] == [0] * 4
    assert 0 < size(8193) <= size(65537) <= size(2 ** 24) <= size(2 ** 31 - 1) <= 2 ** 31
    need = size(70000)
    _refused("kv_free_pages", FREE, dict(wsn=need - 1), BAD, f"{need} bytes")


TREE = dict(q=X, k=X, v=X, table=X, lens=X, cu=X, mask=None, words=0, T=10, B=2, most=5, Hq=8, Hkv=2, d=64, pages=9, page=16, blocks=4, max_len=64, scale=1.0, out=X,
            ws=X, wsn=1 << 40, stream=None)
SIZES = [
    (dict(T=-1), BAD, ">= 0"), (dict(B=-1), BAD, ">= 0"), (dict(blocks=-1), BAD, ">= 0"), (dict(max_len=-1), BAD, "max_len"), (dict(max_len=2 ** 30 + 1), BAD, "max_len"),
    (dict(most=-1), BAD, "max_new"), (dict(most=2 ** 30 + 1), BAD, "max_new"), (dict(mask=X, words=0), BAD, "mask_words"), (dict(mask=X, words=-1), BAD, "mask_words"),
    (dict(mask=X, words=1, most=65), BAD, "mask_words"), (dict(pages=0), BAD, "num_pages"), (dict(page=48), UNSUP, "power of two"),
    *[(dict([(k, None)]), BAD, "NULL") for k in ("q", "k", "table", "lens", "out")], *[(dict([(k, X + 8)]), BAD, "16-byte") for k in ("q", "k", "out")],
    *[(dict([(k, X + 2)]), BAD, "4-byte") for k in ("table", "lens", "cu")], (dict(mask=X + 4, words=1), BAD, "8-byte"),
    (dict(B=2 ** 24, max_len=64), BAD, "grid limit"), (dict(B=2 ** 23, max_len=2 ** 30), BAD, "grid limit"), (dict(most=2 ** 28), BAD, "grid limit"),
    (dict(max_len=2 ** 20, ws=None), BAD, "workspace"), (dict(max_len=2 ** 20, ws=X + 8), BAD, "workspace"), (dict(max_len=2 ** 20, wsn=64), BAD, "workspace")]


@pytest.mark.parametrize("change,status,text", SIZES + [
    (dict(d=96), UNSUP, "d"), (dict(Hq=0), BAD, "num_q_heads"), (dict(Hq=7), BAD, "num_q_heads"), (dict(Hkv=0), BAD, "num_kv_heads"), (dict(v=None), BAD, "NULL"), (dict(cu=None), BAD, "NULL"),
    (dict(v=X + 8), BAD, "16-byte"), (dict(pages=2 ** 28, page=16), UNSUP, "2^32")])
def test_tree_refusals(change, status, text):
    _refused("kv_tree_attention", TREE, change, status, text)


def test_tree_without_rows():
    for change in (dict(T=0), dict(B=0), dict(most=0)):
        assert _call("kv_tree_attention", TREE, q=None, out=None, ws=None, **change) == OK


APPEND = dict(c=X, kr=X, slots=X, T=3, dc=512, dr=64, pages_=X, pages=9, page=64, stream=None)


@pytest.mark.parametrize("change,status,text", [
    (dict(T=-1), BAD, "T"), (dict(dc=128, dr=16), UNSUP, "512 + 64"), (dict(dr=32), UNSUP, "512 + 64"), (dict(dc=256), UNSUP, "512 + 64"), (dict(page=65), UNSUP, "power of two"),
    (dict(pages=-1), BAD, "num_pages"), *[(dict([(k, None)]), BAD, "NULL") for k in ("c", "kr", "slots", "pages_")],
    *[(dict([(k, X + 8)]), BAD, "16-byte") for k in ("c", "kr", "pages_")], (dict(slots=X + 4), BAD, "8-byte")])
def test_latent_append_refusals(change, status, text):
    _refused("kv_latent_append", APPEND, change, status, text)
    assert _call("kv_latent_append", APPEND, T=0, c=None) == OK


LATENT = dict(q=X, k=X, table=X, lens=X, cu=X, mask=None, words=0, T=10, B=2, most=5, H=8, dc=512, dr=64, pages=9, page=16, blocks=4, max_len=64, scale=1.0, out=X,
              ws=X, wsn=1 << 40, stream=None)


@pytest.mark.parametrize("change,status,text", SIZES + [
    (dict(dc=64, dr=8), UNSUP, "512 + 64"), (dict(H=0), BAD, "num_heads"), (dict(cu=None), BAD, "cu_new"), (dict(cu=None, T=2), BAD, "max_new"),
    (dict(cu=None, T=2, most=1, mask=X, words=1), BAD, "no mask"), (dict(pages=2 ** 29), UNSUP, "2^32")])
def test_latent_refusals(change, status, text):
    _refused("kv_latent_attention", LATENT, change, status, text)


def test_latent_without_rows():
    for change in (dict(T=0), dict(B=0), dict(most=0), dict(B=0, T=0, cu=None, most=1)):
        assert _call("kv_latent_attention", LATENT, q=None, out=None, ws=None, **change) == OK


PROMPT = dict(q=X, k=X, kt=128, kh=64, kr=X, v=X, vt=128, vh=64, cq=X, ck=X, B=1, Tq=10, Tk=10, H=2, d=64, scale=1.0, out=X, stream=None)


@pytest.mark.parametrize("change,status,text", [
    (dict(B=-1), BAD, "B"), (dict(Tq=-1), BAD, "Tq"), (dict(Tk=-1), BAD, "Tk"), (dict(Tq=2 ** 30 + 1), BAD, "2^30"), (dict(Tk=2 ** 30 + 1), BAD, "2^30"), (dict(H=0), BAD, "num_heads"),
    (dict(d=96), UNSUP, "d = 96"), (dict(kt=-8), BAD, "token stride"), (dict(vt=4), BAD, "token stride"), (dict(kt=2 ** 24 + 8), BAD, "token stride"), (dict(kh=12), BAD, "head stride"),
    (dict(vh=-8), BAD, "head stride"), (dict(vh=2 ** 40 + 8), BAD, "head stride"), *[(dict([(k, None)]), BAD, "NULL") for k in ("q", "k", "kr", "v", "cq", "ck", "out")],
    *[(dict([(k, X + 8)]), BAD, "16-byte") for k in ("q", "k", "kr", "v", "out")], (dict(cq=X + 2), BAD, "4-byte"), (dict(ck=X + 2), BAD, "4-byte"),
    (dict(Tq=2 ** 30, H=2), BAD, "grid limit"), (dict(B=2 ** 24, Tq=2 ** 24), BAD, "grid limit")])
def test_latent_prompt_refusals(change, status, text):
    _refused("kv_latent_prompt_attention", PROMPT, change, status, text)
    for none in (dict(B=0), dict(Tq=0)):
        assert _call("kv_latent_prompt_attention", PROMPT, q=None, cq=None, **none) == OK


@pytest.mark.parametrize("name,head,rows", [("kv_tree_attention_workspace_bytes", (32, 8, 128), 4), ("kv_latent_attention_workspace_bytes", (16, 512), 16)])
def test_attention_workspace_sizes(name, head, rows):
    """0 where the call refuses and where no request is cut; enough for any smaller call of the same requests
    (a captured one whose bounds were larger); the formula's parts: a partial readout, a maximum and a sum a row."""
    size = getattr(lib.load(), name)
    B, d = 5, head[-1]
    assert size(B, *head, 1, 100) == 0 and size(0, *head, 1, 9999) == 0 and size(-1, *head, 1, 9999) == 0
    for most, length in ((-1, 9999), (2 ** 30 + 1, 9999), (1, -1), (1, 2 ** 30 + 1), (2 ** 28, 9999)):
        assert size(B, *head, most, length) == 0
    assert size(2 ** 24, *head, 1, 100) == 0 and size(2 ** 23, *head, 1, 2 ** 30) == 0
    assert size(B, *[-1] * len(head), 1, 9999) == 0 and size(B, *head[:-1], 96, 1, 9999) == 0
    for most in (1, 3, 17, 40):
        n = size(B, *head, most, 9999)
        assert n > 0 and n == size(B, *head, most, 2 ** 30) and (n - 8 * B) % ((d + 2) * 4) == 0
        parts = (n - 8 * B) // ((d + 2) * 4)
        assert parts >= B * rows * most, "a place for every row"
    assert size(2000, *head, 4, 2 ** 20) == 0 or name.startswith("kv_latent"), "many requests are not cut"
    assert ctypes.sizeof(ctypes.c_size_t) == 8 and size(2 ** 12, *head, 1, 2 ** 30) < 2 ** 40
