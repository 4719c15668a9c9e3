"""Attention of several new tokens and of latents where its parts meet (the waves of a workgroup, the runs of a request that
was cut), its workspace, its weights and its largest values. References: cache_ref in 64 bits, bounds cache_ref.tolerance."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import cache_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib  # noqa: E402
from test_gpu_tree import _i32, build, weight  # noqa: E402

LOW = -17.5     # a key's channel that puts a token's score 140 below the others' (a weight of 2^-202)


def _one_value(lens, most, Hq, Hkv, d, value, low=range(0), missing=0, page=16):
    """Request 0's last token holds `value` in channel 7, its tokens `low` score far below the others, and its first
    `missing` pages do not exist. Every new token of every request against the formula."""
    new = [min(most, n) for n in lens]
    gen, kp, vp, table, keys = build(lens, new, Hkv, d, page)
    for b, (k, v) in enumerate(keys):
        k[:] = (k.float() / 64).bfloat16()
        k[..., 5] = 0.0
        if b == 0:
            k[list(low), :, 5] = LOW
            v[-1, :, 7] = value
        pos = torch.arange(lens[b])
        p = table[b, pos // page].long()
        kp[p, :, pos % page], vp[p, :, pos % page] = k, v
    table[0, :missing] = -1
    T, cu = sum(new), [sum(new[:b]) for b in range(len(new) + 1)]
    q = torch.randn((T, Hq, d), generator=gen).bfloat16()
    q[..., 5] = 8.0
    out = torch.full_like(q, 7.0, device="cuda")
    lib.kv_tree_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32(lens), _i32(cu), out, max_new=most, scale=1.0)
    for b, n in enumerate(new):
        there = torch.arange(lens[b]) >= (missing * page if b == 0 else 0)
        k, v = (x[there].double() for x in keys[b])
        o, mag, e = ref.attend(q[cu[b]:cu[b + 1]].double(), k, v, ref.seen(n, lens[b])[:, there], 1.0)
        ref.is_close(out[cu[b]:cu[b + 1]], o, ref.tolerance(o, mag, e, lens[b], weight(most * Hq // Hkv)), f"request {b}")


VALUES = pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])


@VALUES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("most,Hq,Hkv", [(1, 1, 1), (1, 8, 2), (5, 6, 2), (12, 4, 2)])
def test_a_value_that_one_wave_took_out(value, d, most, Hq, Hkv):
    """An infinite value of a new token comes back as it is where the first tiles' tokens do not exist, or weigh nothing beside it."""
    _one_value([60], most, Hq, Hkv, d, value, missing=2)
    _one_value([60], most, Hq, Hkv, d, value, low=range(32))
    _one_value([150, 40], most, Hq, Hkv, d, value, low=[t for t in range(150) if t // 32 % 4 == 0])


@VALUES
@pytest.mark.parametrize("lens,most,Hq,Hkv,d", [([4000], 1, 8, 2, 64), ([4000], 12, 4, 4, 128), ([4000], 30, 4, 2, 64), ([4000, 7], 20, 8, 2, 128), ([4000] + [9] * 39, 8, 32, 4, 64)])
def test_a_value_in_a_run_that_weighs_nothing(value, lens, most, Hq, Hkv, d):
    """A run of the last tokens scores far below the others, so that its readouts count next to nothing; an infinity among them still does."""
    _one_value(lens, most, Hq, Hkv, d, value, low=range(2100, 4000))
    _one_value(lens, most, Hq, Hkv, d, value, low=range(0, 2000))


def _guarded(need, call, out):
    """A call with a workspace of exactly its bytes, which hold NaN before, and a region behind it that stays as it is."""
    assert need > 0
    guard = 2 ** 24
    ws = torch.full((need + guard,), 0xff, dtype=torch.uint8, device="cuda")
    out.fill_(7.0)
    call(ws[:need])
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xff).all()), "written behind the workspace"
    got = out.clone()
    call(torch.zeros(need + guard, dtype=torch.uint8, device="cuda"))
    assert torch.equal(got, out)
    return got


def _ones(lens, new, page):
    """A table over pages in order, which of their rows hold a token, and the running sums of the new tokens."""
    need = [-(-n // page) for n in lens]
    first = [sum(need[:b]) for b in range(len(need))]
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    live = torch.zeros((sum(need), page), dtype=torch.bool)
    for b, n in enumerate(lens):
        table[b, :need[b]] = torch.arange(first[b], first[b] + need[b])
        live[first[b]:first[b] + need[b]] = (torch.arange(need[b] * page) < n).reshape(-1, page)
    return table.cuda(), live.cuda(), _i32([sum(new[:b]) for b in range(len(new) + 1)])


# few units and many, of which none, one, some and nearly all are cut
LENGTHS = {"one long": [4000], "few": [3000, 17, 900, 2048], "ladder": [60 * (i + 1) for i in range(100)], "one of many": [100] * 299 + [9000],
           "two sizes": [40] * 200 + [2500] * 200, "even": [1500] * 128}


@pytest.mark.parametrize("what", LENGTHS)
@pytest.mark.parametrize("most,Hq,Hkv,d", [(2, 8, 4, 64), (12, 8, 4, 64), (40, 8, 2, 128)])
def test_the_workspace_of_cut_requests(what, most, Hq, Hkv, d):
    lens = LENGTHS[what]
    new = [min(n, most - b % 2) for b, n in enumerate(lens)]
    table, live, cu = _ones(lens, new, 16)
    kp = torch.randn((live.shape[0], Hkv, 16, d), device="cuda").bfloat16()
    vp = torch.where(live[:, None, :, None], 1.0, float("nan")).bfloat16().expand(-1, Hkv, -1, d).contiguous()
    q = torch.randn((sum(new), Hq, d), device="cuda").bfloat16()
    out, ln = torch.empty_like(q), _i32(lens)
    got = _guarded(lib.kv_tree_attention_workspace_bytes(len(lens), Hq, Hkv, d, most, max(lens)),
                   lambda ws: lib.kv_tree_attention(q, kp, vp, table, ln, cu, out, max_new=most, max_len=max(lens), workspace=ws), out)
    assert bool((got == 1.0).all())


@pytest.mark.parametrize("what", LENGTHS)
@pytest.mark.parametrize("most,H,dc", [(1, 16, 512), (2, 16, 256), (3, 40, 512)])
def test_the_workspace_of_cut_latents(what, most, H, dc):
    lens = LENGTHS[what]
    new = [min(n, most) for n in lens]
    table, live, cu = _ones(lens, new, 16)
    pages = torch.randn((live.shape[0], 16, dc + dc // 8), device="cuda").bfloat16()
    pages[..., :dc] = torch.where(live[..., None], 1.0, float("nan")).bfloat16()
    q = torch.randn((sum(new), H, dc + dc // 8), device="cuda").bfloat16()
    out, ln = torch.empty((sum(new), H, dc), dtype=torch.bfloat16, device="cuda"), _i32(lens)
    got = _guarded(lib.kv_latent_attention_workspace_bytes(len(lens), H, dc, most, max(lens)),
                   lambda ws: lib.kv_latent_attention(q, pages, table, ln, out, 0.05, cu_new=cu, max_new=most, max_len=max(lens), workspace=ws), out)
    assert bool((got == 1.0).all())


@pytest.mark.parametrize("most,there,Hq,Hkv,d", [(96, 96, 8, 2, 128), (400, 2, 32, 8, 64)])
def test_more_pieces_to_join_than_workgroups(most, there, Hq, Hkv, d):
    """The launch that joins takes several pieces a workgroup."""
    lens = [40 if b % 5 else 1700 for b in range(512)]
    new = [min(n, there) for n in lens]
    table, live, cu = _ones(lens, new, 16)
    kp = torch.randn((live.shape[0], Hkv, 16, d), device="cuda").bfloat16()
    vp = torch.where(live[:, None, :, None], 1.0, float("nan")).bfloat16().expand(-1, Hkv, -1, d).contiguous()
    q = torch.randn((sum(new), Hq, d), device="cuda").bfloat16()
    out, ln = torch.empty_like(q), _i32(lens)
    got = _guarded(lib.kv_tree_attention_workspace_bytes(512, Hq, Hkv, d, most, 1700),
                   lambda ws: lib.kv_tree_attention(q, kp, vp, table, ln, cu, out, max_new=most, max_len=1700, workspace=ws), out)
    assert bool((got == 1.0).all())


def test_as_many_latent_tiles_as_a_call_takes():
    """512 requests that may have 131,072 rows each: an eighth of the limit, and 2^24 pieces to join."""
    lens, H = [30 if b % 7 else 2000 for b in range(512)], 128
    new = [1 + b % 2 for b in range(512)]
    table, live, cu = _ones(lens, new, 16)
    pages = torch.randn((live.shape[0], 16, 576), device="cuda").bfloat16()
    pages[..., :512] = torch.where(live[..., None], 1.0, float("nan")).bfloat16()
    q = torch.randn((1024, H, 576), device="cuda").bfloat16()
    out, ln = torch.zeros((1024, H, 512), dtype=torch.bfloat16, device="cuda"), _i32(lens)
    lib.kv_latent_attention(q, pages, table, ln, out, 0.05, cu_new=cu, max_new=1024, max_len=4096)
    assert bool((out[:sum(new)] == 1.0).all()) and not bool(out[sum(new):].any())


@pytest.mark.parametrize("dc", [256, 512])
@pytest.mark.parametrize("H,most", [(1, 1), (5, 3), (16, 1), (4, 4)])
@pytest.mark.parametrize("n", [4, 17, 70, 900])
def test_latent_weights_of_few_rows(dc, H, most, n):
    """Up to 16 rows: values of either sign that cancel, so that a weight rounded once to bf16 would show."""
    W = dc + dc // 8
    gen, pages, _, table, keys = build([n], [most], 1, dc, 16, latent=W)
    k = keys[0]
    k[:, :dc] = 64.0 * (1 - 2 * torch.randint(0, 2, (n, dc), generator=gen))
    pos = torch.arange(n)
    pages[table[0, pos // 16].long(), pos % 16] = k
    q = torch.randn((most, H, W), generator=gen).bfloat16()
    q[..., :dc] = 0.0
    out = torch.zeros((most, H, dc), dtype=torch.bfloat16, device="cuda")
    lib.kv_latent_attention(q.cuda(), pages.cuda(), table.cuda(), _i32([n]), out, 0.02, cu_new=_i32([0, most]))
    kd = k.double()[:, None]
    o, mag, e = ref.attend(q.double(), kd, kd[..., :dc], ref.seen(most, n), 0.02)
    ref.is_close(out, o, ref.tolerance(o, mag, e, n, weight(H * most)), f"{n} tokens")


# Large values over long contexts: scores that pass the first tiles' by a little less than 2^8 (references stay where they
# are), values of half the bound 2^120 / n. All equal, so the mean is the value itself, and it comes back exactly.
LONG, RISE = 65536, 7.9


def _steps(n, low):
    """A score of RISE binary orders for all tokens but the first `low`, as a key's channel beside a query's of 8."""
    k = torch.full((n,), RISE * 0.6931 / 8).bfloat16()
    k[:low] = 0.0
    assert float(k.max()) * 8 / 0.6931 < 8.0
    return k


def _layout(B, n):
    """Request 0 of n tokens, the others of one; pages of 16 in order."""
    lens = [n] + [1] * (B - 1)
    table, live, cu = _ones(lens, [1] * B, 16)
    pos = torch.arange(n, device="cuda")
    return lens, table, live, cu, pos


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 2, 1), (1, 20, 1), (1, 280, 2), (520, 4, 4), (520, 160, 8), (520, 640, 8)])
def test_large_values(B, Hq, Hkv, d):
    """Of one request that is cut, and of one among so many that none is."""
    value = 2.0 ** 119 / LONG
    lens, table, live, cu, pos = _layout(B, LONG)
    kp = torch.zeros((live.shape[0], Hkv, 16, d), dtype=torch.bfloat16, device="cuda")
    kp[pos // 16, :, pos % 16, 5] = _steps(LONG, 256).cuda()[:, None]
    vp = torch.where(live[:, None, :, None], value, float("nan")).bfloat16().expand(-1, Hkv, -1, d).contiguous()
    q = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    q[..., 5] = 8.0
    out = torch.zeros_like(q)
    lib.kv_tree_attention(q, kp, vp, table, _i32(lens), cu, out, max_new=1, scale=1.0)
    assert bool((out == value).all())


@pytest.mark.parametrize("dc", [256, 512])
@pytest.mark.parametrize("B,H", [(1, 3), (1, 20), (1, 100), (1100, 1), (1100, 20), (1100, 40)])
def test_large_latents(B, H, dc):
    value = 2.0 ** 119 / LONG
    lens, table, live, cu, pos = _layout(B, LONG)
    pages = torch.zeros((live.shape[0], 16, dc + dc // 8), dtype=torch.bfloat16, device="cuda")
    pages[..., :dc] = torch.where(live[..., None], value, float("nan")).bfloat16()
    pages[pos // 16, pos % 16, dc + 5] = _steps(LONG, 256).cuda()
    q = torch.zeros((B, H, dc + dc // 8), dtype=torch.bfloat16, device="cuda")
    q[..., dc + 5] = 8.0
    out = torch.zeros((B, H, dc), dtype=torch.bfloat16, device="cuda")
    lib.kv_latent_attention(q, pages, table, _i32(lens), out, 1.0, cu_new=cu, max_new=1)
    assert bool((out == value).all())


@pytest.mark.parametrize("d,H,nq", [(64, 2, 3), (128, 2, 70), (64, 256, 70)])
def test_large_prompt_values(d, H, nq):
    n = 4096
    value = 2.0 ** 119 / n
    q, k, kr = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((nq, H, d + d // 2), (n, H, d), (n, d // 2)))
    q[..., 5], k[..., 5] = 8.0, _steps(n, 64).cuda()[:, None]
    v = torch.full((n, H, d), value, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((nq, H, d), dtype=torch.bfloat16, device="cuda")
    lib.kv_latent_prompt_attention(q, k, kr, v, _i32([0, nq]), out, cu_k=_i32([0, n]), scale=1.0)
    assert bool((out == value).all())


@pytest.mark.parametrize("d,most,Hq,Hkv", [(64, 1, 4, 1), (128, 3, 4, 1), (64, 20, 2, 1), (128, 70, 4, 2)])
def test_large_values_that_weigh_nothing(d, most, Hq, Hkv):
    """Values of 2^100 that score 2^-300 below the others: not even a small part of them is seen beside values of 2^-30."""
    n = 4000
    table, live, cu = _ones([n], [most], 16)
    pos = torch.arange(n, device="cuda")
    for low in (range(64), range(2000, n - 100), [t for t in range(n - 100) if t // 32 % 4 == 0]):
        kp = torch.zeros((live.shape[0], Hkv, 16, d), dtype=torch.bfloat16, device="cuda")
        vp = torch.full_like(kp, 2.0 ** -30)
        t = pos[list(low)]
        kp[t // 16, :, t % 16, 5], vp[t // 16, :, t % 16] = -26.0, 2.0 ** 100
        q = torch.zeros((most, Hq, d), dtype=torch.bfloat16, device="cuda")
        q[..., 5] = 8.0
        out = torch.zeros_like(q)
        lib.kv_tree_attention(q, kp, vp, table, _i32([n]), cu, out, scale=1.0)
        assert bool((out == 2.0 ** -30).all())


def test_the_default_bound_of_new_tokens():
    """Without max_new a call takes any batch that it takes with one: 512 requests, 16 drafted each, of which any may have all."""
    lens, new = [60] * 511 + [5000], [16] * 512
    table, live, cu = _ones(lens, new, 16)
    T, ln = sum(new), _i32(lens)
    kp = torch.randn((live.shape[0], 2, 16, 64), device="cuda").bfloat16()
    vp = torch.where(live[:, None, :, None], 1.0, float("nan")).bfloat16().expand(-1, 2, -1, 64).contiguous()
    q = torch.randn((T, 8, 64), device="cuda").bfloat16()
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    lib.kv_tree_attention(q, kp, vp, table, ln, cu, out)
    assert bool((out == 1.0).all())
    pages = torch.randn((live.shape[0], 16, 288), device="cuda").bfloat16()
    pages[..., :256] = torch.where(live[..., None], 1.0, float("nan")).bfloat16()
    q, out = torch.randn((T, 8, 288), device="cuda").bfloat16(), torch.zeros((T, 8, 256), dtype=torch.bfloat16, device="cuda")
    lib.kv_latent_attention(q, pages, table, ln, out, 0.05, cu_new=cu)
    assert bool((out == 1.0).all())
    assert torch.cuda.max_memory_allocated() - before < 2 ** 30


def test_a_scale_of_nan_is_seen():
    nan = float("nan")
    for most, Hq in ((1, 4), (20, 4), (70, 8)):
        table, live, cu = _ones([100], [most], 16)
        kp, vp = (torch.randn((live.shape[0], 1, 16, 64), device="cuda").bfloat16() for _ in range(2))
        q = torch.randn((most, Hq, 64), device="cuda").bfloat16()
        out = torch.zeros_like(q)
        lib.kv_tree_attention(q, kp, vp, table, _i32([100]), cu, out, scale=nan)
        assert bool(torch.isnan(out).all()), f"{most} tokens"
        pages, q, out = (torch.randn(s, device="cuda").bfloat16() for s in ((live.shape[0], 16, 288), (most, Hq, 288), (most, Hq, 256)))
        lib.kv_latent_attention(q, pages, table, _i32([100]), out, nan, cu_new=cu)
        assert bool(torch.isnan(out).all()), f"latents, {most} tokens"
    q, k, kr, out = (torch.randn(s, device="cuda").bfloat16() for s in ((90, 2, 96), (90, 2, 64), (90, 32), (90, 2, 64)))
    lib.kv_latent_prompt_attention(q, k, kr, k, _i32([0, 90]), out, scale=nan)
    assert bool(torch.isnan(out).all())


def test_forks_beside_empty_arrays():
    """A free list of no pages and a table of no blocks share no memory with anything, wherever they point."""
    lens, shares = _i32([5, 0]), _i32([0] * 9)
    copies = [_i32([7]) for _ in range(3)]
    used = _i32([7])
    lib.kv_fork_tables(_i32([0]), _i32([1]), lens, shares[4:4], torch.zeros((2, 0), dtype=torch.int32, device="cuda"), shares, 16, *copies, used)
    assert lens.tolist() == [5, 5] and shares.tolist() == [0] * 9 and [c.item() for c in copies] == [-1, -1, 0] and used.item() == 0
    with pytest.raises(lib.DampError, match="overlaps"):
        lib.kv_fork_tables(_i32([0]), _i32([1]), lens, shares[4:5], torch.zeros((2, 1), dtype=torch.int32, device="cuda"), shares, 16, *copies, used)
