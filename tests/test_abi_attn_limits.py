"""CPU-only: how much workspace the attentions of several tokens ask for, and up to which sizes they take a call."""
import pytest

from quantized_delta_rule_gdn_amd import lib


@pytest.mark.parametrize("name,head,rows,width", [
    ("kv_tree_attention_workspace_bytes", (32, 8, 128), 128, 130), ("kv_tree_attention_workspace_bytes", (16, 2, 64), 128, 66),
    ("kv_latent_attention_workspace_bytes", (128, 512), 64, 514), ("kv_latent_attention_workspace_bytes", (64, 256), 64, 258)])
def test_the_workspace_is_what_one_round_of_workgroups_leaves(name, head, rows, width):
    """No more units of work, and no wider bound of a request's new tokens, ask for more: a partial readout, a maximum and a sum
    of the rows of at most 768 workgroups (3 a CU), and 8 bytes a request."""
    size = getattr(lib.load(), name)
    for B in (48, 64, 256, 512):
        for most in (32, 512):
            got = size(B, *head, most, 4096) - 8 * B
            assert 0 < got <= min(768 * rows * width * 4, 2 ** 26), (B, most, got)
            assert got == size(48, *head, 32, 4096) - 8 * 48


X = 0x100000   # never dereferenced: every case is settled on the host
MOST = {"kv_tree_attention": 2 ** 24 - 2 ** 10, "kv_latent_attention": 2 ** 23 - 2 ** 10}


def _takes(name, B, Hkv, group, most, max_len):
    """Whether the call with these sizes gets as far as its workspace, or to rows that are none."""
    if name == "kv_tree_attention":
        ws = lib.load().kv_tree_attention_workspace_bytes(B, Hkv * group, Hkv, 128, most, max_len)
        status = lib.load().kv_tree_attention(X, X, X, X, X, X, None, 0, 1, B, most, Hkv * group, Hkv, 128, 9, 16, 4, max_len, 1.0, X, None, 0, None)
    else:
        ws = lib.load().kv_latent_attention_workspace_bytes(B, group, 512, most, max_len)
        status = lib.load().kv_latent_attention(X, X, X, X, X, None, 0, 1, B, most, group, 512, 64, 9, 16, 4, max_len, 1.0, X, None, 0, None)
    assert status == lib.DAMP_ERR_INVALID_ARGUMENT
    assert ("workspace" in lib.last_error()) == (ws > 0) and ("grid limit" in lib.last_error()) == (ws == 0), lib.last_error()
    return ws > 0


@pytest.mark.parametrize("B", [1, 48, 256, 512])
@pytest.mark.parametrize("name,Hkv,group", [("kv_tree_attention", 1, 64), ("kv_tree_attention", 8, 128), ("kv_latent_attention", 1, 64), ("kv_latent_attention", 1, 128)])
def test_every_call_up_to_the_documented_size(name, Hkv, group, B):
    """Tiles of 64 query rows over all requests and key-value heads, requests that may be cut and so are joined."""
    most = MOST[name] // (B * Hkv * group // 64)
    if most * Hkv * group < 2 ** 30:
        assert _takes(name, B, Hkv, group, most, 4096)
    assert not _takes(name, B, Hkv, group, 4 * most, 4096)


def test_one_tile_a_request_up_to_the_documented_size():
    """Where tiles have 64 rows the limit is met on both sides."""
    assert _takes("kv_tree_attention", 512, 32766, 64, 1, 4096) and not _takes("kv_tree_attention", 512, 32768, 64, 1, 4096)
    assert _takes("kv_latent_attention", 512, 1, 64, 16382, 4096) and not _takes("kv_latent_attention", 512, 1, 64, 16384, 4096)


FORK = ("src", "dst", "lens", "free", "table", "shares", "cs", "cd", "cr", "used")


def _forked(**where):
    at = {name: X + 4096 * i for i, name in enumerate(FORK)}
    at.update(where)
    return lib.load().kv_fork_tables(at["src"], at["dst"], 3, at["lens"], 2, at["free"], 5, at["table"], 4, at["shares"], 9, 16, at["cs"], at["cd"], at["cr"], at["used"], None)


@pytest.mark.parametrize("written", ["lens", "table", "shares", "cs", "cd", "cr", "used"])
def test_a_fork_s_outputs_overlap_nothing(written):
    """Workgroups read the lists while others write: an array over another one is refused, also where it only reaches into it."""
    count = dict(src=3, dst=3, lens=2, free=5, table=8, shares=9, cs=3, cd=3, cr=3, used=1)
    for i, other in enumerate(FORK):
        if other == written:
            continue
        base = X + 4096 * i
        for at in (base, base + 4 * (count[other] - 1), base - 4 * (count[written] - 1)):
            assert _forked(**{written: at}) == lib.DAMP_ERR_INVALID_ARGUMENT and "overlaps" in lib.last_error(), (other, at - base)


@pytest.mark.parametrize("other,count", [("lens", 2), ("keep", 2), ("table", 8)])
def test_shares_overlap_nothing_that_is_read_beside_them(other, count):
    for offset in (0, 4 * (count - 1), -4 * 8):
        at = dict(keep=X, lens=X + 4096, table=X + 8192)
        status = lib.load().kv_free_pages(at["keep"], at["lens"], 2, at["table"], 4, at[other] + offset, 9, 16, X + 2 ** 20, X + 2 ** 21, None, 0, None)
        assert status == lib.DAMP_ERR_INVALID_ARGUMENT and "shares overlaps" in lib.last_error()
