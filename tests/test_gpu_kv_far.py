"""kv_decode_attention where a token that is lost, or read twice, must show: all scores are equal and V is
one-hot, so that every channel counts the tokens of its own. Requests of more items than one round of the
join takes (256), items of more tokens than one run of page addresses holds (16,384), and lengths around
the items' borders.

Bounds. Equal scores give weights of exactly 1 within a request, so a channel is count / n with the division's
and the sums' roundings, (n / 32 + 300) 2^-24, and the readout's rounding to bf16, 2^-8. A tile too few or too
many is 32 tokens of about n / d: it shows where 32 d / n is above twice the bound."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from quantized_delta_rule_gdn_amd import lib  # noqa: E402


def _count(lens, Hq, Hkv, d, page, by, blocks=None, new=False, max_len=None):
    """Runs one call and checks every channel; token t counts in channel (t // by) % d, with 1 + head % 3."""
    B = len(lens)
    need = [-(-n // page) for n in lens]
    blocks = blocks or max(need)
    gen = torch.Generator().manual_seed(sum(lens))
    ids = torch.randperm(sum(need) + 2, generator=gen).to(torch.int32)
    nan = float("nan")
    kp = torch.full((len(ids), Hkv, page, d), nan, dtype=torch.bfloat16, device="cuda")
    vp = torch.full_like(kp, nan)
    head = (1 + torch.arange(Hkv, device="cuda") % 3).to(torch.bfloat16)
    table = torch.full((B, blocks), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        own = ids[at:at + need[b]]
        table[b, :need[b]] = own
        at += need[b]
        for i0 in range(0, need[b], 256):                       # (some pages at a time: V is large for many heads)
            i1 = min(i0 + 256, need[b])
            t = torch.arange(i0 * page, i1 * page, device="cuda")
            hot = torch.nn.functional.one_hot((t // by) % d, d).to(torch.bfloat16)
            live = (t < n)[:, None]
            v = torch.where(live, hot, torch.full_like(hot, nan)).reshape(i1 - i0, 1, page, d) * head[None, :, None, None]
            k = torch.where(live, torch.zeros_like(hot), torch.full_like(hot, nan)).reshape(i1 - i0, 1, page, d)
            vp[own[i0:i1].long().cuda()] = v
            kp[own[i0:i1].long().cuda()] = k.expand(-1, Hkv, -1, -1)
    q = torch.ones((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    extra = {}
    if new:   # the last token comes with the call: its page holds NaN there until then
        last = torch.tensor([n - 1 for n in lens], device="cuda")
        page_of = table.cuda().long().gather(1, (last // page)[:, None])[:, 0]
        extra = dict(k_new=kp[page_of, :, last % page].clone(), v_new=vp[page_of, :, last % page].clone())
        kp[page_of, :, last % page] = nan
        vp[page_of, :, last % page] = nan
    lib.kv_decode_attention(q, kp, vp, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), out, max_len=max_len, **extra)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        t = torch.arange(n)
        want = torch.bincount((t // by) % d, minlength=d).double() / n
        want = want[None] * (1 + torch.arange(Hkv) % 3).double()[:, None]                  # [Hkv, d]
        want = want.repeat_interleave(Hq // Hkv, 0)
        err = (out[b].double().cpu() - want).abs()
        bound = (2.0 ** -8 + (n / 32 + 300) * 2.0 ** -24) * want
        assert bool((err <= bound).all()), f"request {b} of {n}: channels {sorted(set((err > bound).nonzero()[:, 1].tolist()))[:8]}"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 16, 128])
@pytest.mark.parametrize("by", [1, 32])
def test_every_token_counts_once(d, page, by):
    _count([5000, 1, 2049, 1025, 640], 4, 2, d, page, by)
    _count([700, 65, 1024], 3, 1, d, page, by)                     # none is cut


@pytest.mark.parametrize("lens", [[255 + 256 * 5], [256 * 6], [256 * 6 + 1], [4096, 4097, 4127, 4128, 4129, 33]], ids=str)
def test_around_the_items_borders(lens):
    _count(lens, 2, 1, 64, 16, 32, new=True)
    _count(lens, 2, 1, 128, 8, 32)


@pytest.mark.parametrize("d,Hq", [(64, 1), (128, 5)])
def test_a_request_of_more_items_than_a_round_of_the_join(d, Hq):
    """More than 65,536 tokens of one key-value head: 274 and 391 items of 256."""
    _count([70001], Hq, 1, d, 16, 64, new=True)
    _count([100000], Hq, 1, d, 64, 128)


@pytest.mark.parametrize("page", [16, 32])
def test_items_of_more_tokens_than_a_run_of_page_addresses(page):
    """1,024 key-value heads: one item for the whole request, in two runs of page addresses."""
    _count([20003], 1024, 1024, 64, page, 64, new=True)


def test_requests_of_very_different_lengths():
    _count([40000] + [3] * 70 + [17000, 1, 300], 2, 1, 64, 16, 64)
