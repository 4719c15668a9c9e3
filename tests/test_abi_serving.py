"""CPU-only checks of the serving entry points' host side: statuses and messages of every refusal, the
no-ops, and the workspace sizes, all before any HIP call."""
import ctypes

import pytest

from quantized_delta_rule_gdn_amd import lib

P = ctypes.c_void_p
OK, BAD, UNSUP = lib.DAMP_OK, lib.DAMP_ERR_INVALID_ARGUMENT, lib.DAMP_ERR_UNSUPPORTED
X = 0x100000   # never dereferenced: every case is settled on the host


def _call(name, order, base, **change):
    args = {**base, **change}
    return getattr(lib.load(), name)(*[args[k] for k in order])


STEP = ("pool", "slots", "H", "dk", "dv", "idx", "B", "q", "k", "v", "dt", "alpha", "decay", "out", "stream")
STEP_OK = dict(pool=X, slots=4, H=2, dk=64, dv=64, idx=X, B=0, q=X, k=X, v=X, dt=1, alpha=X, decay=0, out=X, stream=None)


@pytest.mark.parametrize("change,status,text", [
    (dict(B=-1), BAD, "B"), (dict(B=1, dt=5), BAD, "qkv_dtype"), (dict(B=1, decay=3), BAD, "decay"), (dict(B=1, pool=None), BAD, "pool is NULL"),
    (dict(B=1, pool=X + 4), BAD, "aligned"), (dict(B=1, slots=0), BAD, "num_slots"), (dict(B=1, H=0), BAD, "num_heads"),
    (dict(B=1, dk=48, dv=48), UNSUP, "supported"), (dict(B=1, dv=128), UNSUP, "supported"), (dict(B=1, k=None), BAD, "NULL"),
    (dict(B=1, alpha=None), BAD, "NULL"), (dict(B=1, out=X + 4), BAD, "16-byte"), (dict(B=1, q=X + 1), BAD, "misaligned"),
    (dict(B=2 ** 30, H=4), BAD, "grid")])
def test_linear_step_refusals(change, status, text):
    assert _call("fp32_linear_step", STEP, STEP_OK, **change) == status and text in lib.last_error()


def test_linear_step_empty_batch():
    for decay in (0, 1, 2):
        assert _call("fp32_linear_step", STEP, STEP_OK, decay=decay) == OK


PRE = ("pool", "slots", "H", "dk", "dv", "idx", "cu", "resume", "B", "T", "q", "k", "v", "dt", "alpha", "decay")
PRE_OK = dict(pool=X, slots=4, H=2, dk=64, dv=64, idx=X, cu=X, resume=None, B=1, T=10, q=X, k=X, v=X, dt=1, alpha=X, decay=0,
              beta=X, out=X, ws=X, wsn=1 << 40, stream=None)
REFUSED = [
    (dict(B=-1), BAD, "B"), (dict(T=-1), BAD, "T"), (dict(dt=2), BAD, "qkv_dtype"), (dict(decay=3), BAD, "decay"), (dict(pool=None), BAD, "pool"),
    (dict(slots=0), BAD, "num_slots"), (dict(dk=8, dv=8), UNSUP, "supported"), (dict(dk=64, dv=32), UNSUP, "supported"), (dict(cu=None), BAD, "NULL"),
    (dict(out=None), BAD, "NULL"), (dict(q=X + 8), BAD, "16-byte"), (dict(out=X + 2), BAD, "16-byte"), (dict(cu=X + 2), BAD, "misaligned"),
    (dict(resume=X + 1), BAD, "misaligned"), (dict(alpha=X + 1), BAD, "misaligned"), (dict(B=2 ** 28, H=64), BAD, "grid limit"),
    (dict(H=65537), UNSUP, "65,536"), (dict(B=2 ** 21, H=1), BAD, "grid limit"), (dict(T=2 ** 31 - 1, H=1), BAD, "grid limit"), (dict(T=2 ** 30, H=2), BAD, "grid limit")]


@pytest.mark.parametrize("change,status,text", REFUSED)
@pytest.mark.parametrize("name", ["fp32_linear_prefill", "fp32_delta_prefill"])
def test_prefill_refusals(name, change, status, text):
    order = PRE + (("beta",) if "delta" in name else ()) + ("out", "ws", "wsn", "stream")
    assert _call(name, order, PRE_OK, **change) == status and text in lib.last_error()


def test_delta_prefill_own_refusals_and_workspaces():
    order = PRE + ("beta", "out", "ws", "wsn", "stream")
    assert _call("fp32_delta_prefill", order, PRE_OK, beta=None) == BAD and "NULL" in lib.last_error()
    assert _call("fp32_delta_prefill", order, PRE_OK, decay=2) == BAD and "decay" in lib.last_error()
    for B, T in ((0, 10), (1, 0)):
        assert _call("fp32_delta_prefill", order, PRE_OK, B=B, T=T) == OK
    need = lib.load().fp32_prefill_workspace_bytes
    for delta in (0, 1):
        assert need(delta, 0, 10, 2, 64, 1, 0) == 0 and need(delta, 1, 10, 2, 48, 1, 0) == 0
        n = need(delta, 3, 5000, 2, 128, 1, 0)
        if n:
            name = "fp32_delta_prefill" if delta else "fp32_linear_prefill"
            o = order if delta else tuple(x for x in order if x != "beta")
            for change in (dict(ws=None), dict(wsn=n - 1), dict(ws=X + 16)):
                assert _call(name, o, PRE_OK, B=3, T=5000, dk=128, dv=128, **change) == BAD and "workspace" in lib.last_error()


TAB = ("seq", "new", "B", "free", "nf", "page", "table", "blocks", "slots", "pos", "T", "cu", "used", "stream")
TAB_OK = dict(seq=X, new=X, B=1, free=X, nf=1, page=16, table=X, blocks=1, slots=X, pos=None, T=1, cu=X, used=X, stream=None)


@pytest.mark.parametrize("change,status,text", [
    (dict(B=-1), BAD, ">= 0"), (dict(T=-1), BAD, ">= 0"), (dict(nf=-1), BAD, ">= 0"), (dict(blocks=-1), BAD, ">= 0"), (dict(page=0), UNSUP, "power of two"),
    (dict(page=48), UNSUP, "power of two"), (dict(page=65536), UNSUP, "power of two"), (dict(B=8001), UNSUP, "at most"), (dict(seq=None), BAD, "NULL"),
    (dict(table=None), BAD, "NULL"), (dict(free=None), BAD, "NULL"), (dict(slots=None), BAD, "NULL"), (dict(cu=None), BAD, "NULL"), (dict(used=None), BAD, "NULL"),
    (dict(slots=X + 4), BAD, "misaligned"), (dict(pos=X + 2), BAD, "misaligned")])
def test_tables_refusals(change, status, text):
    assert _call("kv_build_tables", TAB, TAB_OK, **change) == status and text in lib.last_error()


APP = ("k", "v", "slots", "T", "H", "d", "kp", "vp", "pages", "page", "stream")
APP_OK = dict(k=X, v=X, slots=X, T=1, H=2, d=64, kp=X, vp=X, pages=3, page=16, stream=None)


@pytest.mark.parametrize("change,status,text", [
    (dict(T=-1), BAD, "T"), (dict(H=0), BAD, "num_kv_heads"), (dict(pages=0), BAD, "num_pages"), (dict(d=96), UNSUP, "supports"), (dict(page=3), UNSUP, "power"),
    (dict(k=None), BAD, "NULL"), (dict(vp=None), BAD, "NULL"), (dict(kp=X + 8), BAD, "16-byte"), (dict(slots=X + 4), BAD, "8-byte"),
    (dict(pages=2 ** 17, page=32768, H=1), UNSUP, "2^32"), (dict(pages=2 ** 31 - 1, page=32768), UNSUP, "2^32")])
def test_append_refusals(change, status, text):
    assert _call("kv_append", APP, APP_OK, **change) == status and text in lib.last_error()
    assert _call("kv_append", APP, APP_OK, T=0) == OK


ATT = ("q", "kp", "vp", "table", "lens", "B", "Hq", "Hkv", "d", "pages", "page", "blocks", "max_len", "scale", "kn", "vn", "out", "ws", "wsn", "stream")
ATT_OK = dict(q=X, kp=X, vp=X, table=X, lens=X, B=1, Hq=4, Hkv=2, d=64, pages=3, page=16, blocks=2, max_len=32, scale=1.0, kn=None, vn=None, out=X,
              ws=X, wsn=1 << 40, stream=None)


@pytest.mark.parametrize("change,status,text", [
    (dict(B=-1), BAD, "B"), (dict(blocks=-1), BAD, "max_blocks"), (dict(max_len=-1), BAD, "max_len"), (dict(max_len=2 ** 30 + 1), BAD, "max_len"),
    (dict(Hq=3), BAD, "multiple"), (dict(Hq=0), BAD, "multiple"), (dict(Hkv=0), BAD, "num_kv_heads"), (dict(d=32), UNSUP, "supports"),
    (dict(page=12), UNSUP, "power"), (dict(q=None), BAD, "NULL"), (dict(table=None), BAD, "NULL"), (dict(kn=X), BAD, "together"), (dict(vn=X), BAD, "together"),
    (dict(out=X + 8), BAD, "16-byte"), (dict(kn=X, vn=X + 2), BAD, "16-byte"), (dict(lens=X + 2), BAD, "4-byte"),
    (dict(B=2 ** 30), BAD, "grid limit"), (dict(B=2 ** 20, Hq=16, Hkv=1), BAD, "grid limit"), (dict(pages=2 ** 20, page=4096), UNSUP, "2^32"),
    (dict(max_len=1 << 20, ws=None), BAD, "workspace"), (dict(max_len=1 << 20, wsn=16), BAD, "workspace"),
    (dict(max_len=1 << 20, ws=X + 4), BAD, "workspace")])
def test_attention_refusals(change, status, text):
    assert _call("kv_decode_attention", ATT, ATT_OK, **change) == status and text in lib.last_error()


def test_attention_empty_batch_and_workspace_sizes():
    assert _call("kv_decode_attention", ATT, ATT_OK, B=0) == OK
    need = lib.load().kv_decode_attention_workspace_bytes
    assert need(0, 4, 2, 64, 100) == 0 and need(1, 3, 2, 64, 100) == 0 and need(1, 4, 2, 96, 100) == 0 and need(1, 4, 2, 64, -1) == 0
    assert need(1, 4, 2, 64, 1) == 0 and need(2, 4, 2, 64, 1 << 16) > 0
