"""The attentions of several new tokens, of latents and of prompts where a token that is lost, or read twice, must
show: all scores are equal and the values one-hot, so that every channel counts the tokens of its own. Lengths
around the borders of tiles, of a wave's share of them and of pages; requests that are cut and that are not, few and many.

Bounds. Equal scores give weights of exactly 1, so a channel is count / n with the division's and the sums'
roundings, (n / 32 + 300) 2^-24, and the readout's rounding to bf16, 2^-8. A token too few or too many shows where
the count is below 2^7, which it is up to 2^7 d tokens. References count in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from quantized_delta_rule_gdn_amd import lib  # noqa: E402
from test_gpu_tree import _i32  # noqa: E402

NAN = float("nan")


def _hot(t, by, d):
    return torch.nn.functional.one_hot((t // by) % d, d).to(torch.bfloat16)


def _paged(lens, page, width, value):
    """Pages [pages, page, width] in random order whose row of a request's token t is value(t), NaN elsewhere; the table."""
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(sum(lens)))
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    rows = torch.full((len(ids), page, width), NAN, dtype=torch.bfloat16, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        own = ids[at:at + need[b]]
        table[b, :need[b]] = own.to(torch.int32)
        at += need[b]
        t = torch.arange(need[b] * page, device="cuda")
        rows[own.cuda()] = torch.where((t < n)[:, None], value(t), NAN).reshape(need[b], page, width)
    return rows, table.cuda()


def _holds(out, lens, new, by, d, mask=None):
    """Every new token's readout [sum(new), heads, d] counts the tokens it sees: those up to its own, or of the new ones its mask's."""
    at = 0
    for b, (m, n) in enumerate(zip(lens, new)):
        if n == 0:
            continue
        hot = _hot(torch.arange(m, device="cuda"), by, d).double()
        seen = hot[:m - n].sum(0) + (hot[m - n:].cumsum(0) if mask is None else mask[b].double().cuda() @ hot[m - n:])
        want = seen / seen.sum(1, keepdim=True).clamp(min=1.0)
        err = (out[at:at + n].double() - want[:, None]).abs()
        bound = (2.0 ** -8 + (m / 32 + 300) * 2.0 ** -24) * want[:, None]
        over = (err > bound).nonzero()
        assert len(over) == 0, f"request {b}, {n} of {m} tokens: (token, head, channel) {over[:4].tolist()}"
        at += n
    assert bool((out[at:] == 7.0).all())


def _words(new, gen):
    """Random masks of the new tokens [n, n], and as words [sum(new), words]."""
    most, bits, rows = max(new), [], []
    for n in new:
        x = torch.rand((n, n), generator=gen) < 0.5
        w = torch.zeros((n, -(-most // 64)), dtype=torch.int64)
        for j in range(n):
            w[:, j // 64] |= torch.where(x[:, j], -(1 << 63) if j % 64 == 63 else 1 << (j % 64), 0)
        bits.append(x)
        rows.append(w)
    return bits, torch.cat(rows).cuda()


def _tree(lens, new, Hq, Hkv, d, page, by, masked=False):
    new = [min(a, n) for a, n in zip(new, lens)]
    v, table = _paged(lens, page, d, lambda t: _hot(t, by, d))
    v = v[:, None].expand(-1, Hkv, -1, -1).contiguous()
    k = v * 0.0
    T, gen = sum(new), torch.Generator().manual_seed(7)
    q = torch.randn((T + 2, Hq, d), generator=gen).bfloat16().cuda()
    out, bits, mask = torch.full_like(q, 7.0), None, None
    if masked:
        bits, mask = _words(new + [2], gen)
    cu = [sum(new[:b]) for b in range(len(new) + 1)]
    lib.kv_tree_attention(q, k, v, table, _i32(lens), _i32(cu), out, mask=mask, max_new=max(new))
    _holds(out, lens, new, by, d, bits)


BORDERS = [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1023, 1024, 1025, 2048, 3000]
# query rows of a key-value head: one wave's 16, tiles of 64, tiles of 128 (with enough of them)
ROWS = pytest.mark.parametrize("most,Hq,Hkv", [(1, 4, 2), (3, 5, 1), (9, 4, 2), (33, 8, 2), (70, 4, 1)])


@ROWS
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 16, 128])
def test_every_token_counts_once(most, Hq, Hkv, d, page):
    _tree(BORDERS, [most - b % 2 * (most // 2) for b in range(len(BORDERS))], Hq, Hkv, d, page, 1)
    _tree([5000, 1, 2049, 640], [most] * 4, Hq, Hkv, d, page, 32, masked=True)
    _tree([5000], [most], Hq, Hkv, d, page, 1)


@ROWS
@pytest.mark.parametrize("what", ["one of many", "two sizes", "ladder", "none is cut"])
def test_every_token_of_many_requests_counts_once(what, most, Hq, Hkv):
    lens = {"one of many": [40 + b % 90 for b in range(299)] + [7001], "two sizes": [50] * 200 + [2000 + b for b in range(60)], "ladder": [40 * (b + 1) + b % 7 for b in range(100)],
            "none is cut": [3000] + [20 + b % 50 for b in range(1099)]}[what]
    _tree(lens, [most - b % 3 * (most // 3) for b in range(len(lens))], Hq, Hkv, 64, 16, 1 if what == "one of many" else 64)


def _latent(lens, new, H, dc, page, by, masked=False):
    new = [min(a, n) for a, n in zip(new, lens)]
    W, d = dc + dc // 8, dc
    pages, table = _paged(lens, page, W, lambda t: torch.nn.functional.pad(_hot(t, by, d), (0, W - d)))
    T, gen = sum(new), torch.Generator().manual_seed(7)
    q = torch.randn((T + 2, H, W), generator=gen).bfloat16().cuda()
    q[..., :d] = 0.0
    out, bits, mask = torch.full((T + 2, H, d), 7.0, dtype=torch.bfloat16, device="cuda"), None, None
    if masked:
        bits, mask = _words(new + [2], gen)
    cu = [sum(new[:b]) for b in range(len(new) + 1)]
    lib.kv_latent_attention(q, pages, table, _i32(lens), out, 0.05, cu_new=_i32(cu), mask=mask, max_new=max(new))
    _holds(out, lens, new, by, d, bits)


LATENT_ROWS = pytest.mark.parametrize("most,H", [(1, 16), (3, 5), (2, 13), (1, 50), (5, 40)])


@LATENT_ROWS
@pytest.mark.parametrize("dc", [256, 512])
@pytest.mark.parametrize("page", [1, 16, 128])
def test_every_latent_counts_once(most, H, dc, page):
    _latent(BORDERS, [most - b % 2 * (most // 2) for b in range(len(BORDERS))], H, dc, page, 1)
    _latent([5000, 1, 2049, 640], [most] * 4, H, dc, page, 32, masked=True)


@LATENT_ROWS
@pytest.mark.parametrize("what", ["one of many", "ladder", "none is cut"])
def test_every_latent_of_many_requests_counts_once(what, most, H):
    lens = {"one of many": [40 + b % 90 for b in range(299)] + [7001], "ladder": [40 * (b + 1) + b % 7 for b in range(100)], "none is cut": [3000] + [20 + b % 50 for b in range(1099)]}[what]
    _latent(lens, [most - b % 3 * (most // 3) for b in range(len(lens))], H, 256, 16, 1 if what == "one of many" else 64)


def _prompts(nq, lens, H, d, by):
    v = torch.cat([_hot(torch.arange(n, device="cuda"), by, d) for n in lens])[:, None].expand(-1, H, -1).contiguous()
    q = torch.randn((sum(nq) + 2, H, d + d // 2), device="cuda").bfloat16()
    out = torch.full((sum(nq) + 2, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    cu_q, cu_k = ([sum(x[:b]) for b in range(len(x) + 1)] for x in (nq, lens))
    lib.kv_latent_prompt_attention(q, torch.zeros_like(v), torch.zeros((sum(lens), d // 2), dtype=torch.bfloat16, device="cuda"), v, _i32(cu_q), out, cu_k=_i32(cu_k))
    _holds(out, lens, nq, by, d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [1, 40])
@pytest.mark.parametrize("by", [1, 64])
def test_every_key_of_a_prompt_counts_once(d, H, by):
    """In row tiles of 64 queries, and of 128 where there are many; behind cached tokens and not."""
    nq = [1, 63, 64, 65, 127, 128, 129, 200, 700]
    for before in (0, 1, 100, 1000):
        _prompts(nq, [n + before * (b % 2) for b, n in enumerate(nq)], H, d, by)


@pytest.mark.parametrize("d,most", [(64, 768), (128, 512)])
def test_prompts_on_both_sides_of_the_wider_tiles(d, most):
    """As many full tiles of 64 rows as are taken so, and a few queries more."""
    for extra in (-2, -1, 0, 1):                      # (two rows are behind the last request)
        n = 64 * most // 16 + extra
        _prompts([n - 200, 200], [n - 200, 300], 16, d, 1)
