"""Latent attention (kv_latent_append, kv_latent_attention, kv_latent_prompt_attention) against binary64.
Bounds: cache_ref.tolerance, the weights rounded once to bf16."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import cache_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib  # noqa: E402
from test_gpu_tree import _i32, build, random_bits  # noqa: E402


# ---- the store --------------------------------------------------------------------------------------
@pytest.mark.parametrize("dc,page", [(512, 64), (256, 16), (512, 1)])
def test_append(dc, page):
    gen = torch.Generator().manual_seed(dc + page)
    pages, T, dr = 7, 37, dc // 8
    n = pages * page
    p = torch.randn((pages, page, dc + dr), generator=gen).bfloat16()
    c, r = torch.randn((T, dc), generator=gen).bfloat16(), torch.randn((T, dr), generator=gen).bfloat16()
    slots = torch.full((T,), -1, dtype=torch.int64)
    perm = torch.randperm(T, generator=gen)[: min(T - 3, n)]
    slots[perm] = torch.randperm(n, generator=gen)[: perm.numel()]
    rest = [t for t in range(T) if t not in perm.tolist()]
    slots[rest[0]], slots[rest[1]] = n, 2 ** 40
    want = p.clone()
    for t in range(T):
        s = int(slots[t])
        if 0 <= s < n:
            want[s // page, s % page] = torch.cat([c[t], r[t]])
    got = p.cuda()
    lib.kv_latent_append(c.cuda(), r.cuda(), slots.cuda(), got)
    assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    lib.kv_latent_append(c[:0].cuda(), r[:0].cuda(), slots[:0].cuda(), got)


# ---- absorbed form ------------------------------------------------------------------------------------
def _absorbed(lens, new, H, dc, page, kind="tree", scale=None, max_len=None, seed=0, blocks=None, single=False):
    W = dc + dc // 8
    gen, pages, _, table, keys = build(lens, new, 1, dc, page, seed, latent=W, blocks=blocks)
    T = sum(new)
    q = torch.randn((T if single else T + 3, H, W), generator=gen).bfloat16()
    bits = [None if kind is None else random_bits(n, gen, kind) for n in new]
    most = max(new + [1])
    mask = None
    if kind is not None and not single:
        mask = torch.full((T + 3, -(-most // 64)), -1, dtype=torch.int64)
        for b, n in enumerate(new):
            mask[sum(new[:b]):sum(new[:b + 1])] = ref.words(bits[b], mask.shape[1])
        mask = mask.cuda()
    s = W ** -0.5 if scale is None else scale
    out = torch.full((q.shape[0], H, dc), 7.0, dtype=torch.bfloat16, device="cuda")
    pd, cu = pages.cuda(), np.cumsum([0] + new).tolist()
    if single:
        lib.kv_latent_attention(q.cuda(), pd, table.cuda(), _i32(lens), out, s, max_len=max_len)
    else:
        lib.kv_latent_attention(q.cuda(), pd, table.cuda(), _i32(lens), out, s, cu_new=_i32(cu), mask=mask, max_new=most, max_len=max_len)
    torch.cuda.synchronize()
    assert torch.equal(pd.cpu().view(torch.int16), pages.view(torch.int16)) and bool((out[T:] == 7.0).all())
    used = 0.0
    for b, n in enumerate(new):
        m = lens[b] if max_len is None else min(lens[b], max_len)
        k = keys[b][:m].double()[:, None]
        o, mag, e = ref.attend(q[cu[b]:cu[b + 1]].double(), k, k[..., :dc], ref.seen(n, lens[b], bits[b])[:, :m], s)
        used = max(used, ref.is_close(out[cu[b]:cu[b + 1]], o, ref.tolerance(o, mag, e, m, ref.BF16), f"request {b}: {n} of {lens[b]} tokens"))
    return used


@pytest.mark.parametrize("dc", [512, 256])
@pytest.mark.parametrize("page", [1, 8, 16, 64, 128])
def test_absorbed_lengths(dc, page):
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 300]
    _absorbed(lens, [1] * len(lens), 4, dc, page, None, single=True)
    _absorbed(lens, [0, 1, 2, 3, 16, 5, 1, 7, 9, 2, 1, 12, 3, 4], 4, dc, page, "any")


@pytest.mark.parametrize("dc", [512, 256])
@pytest.mark.parametrize("H", [1, 3, 8, 16, 17, 32, 33, 64, 128])
def test_absorbed_heads(dc, H):
    _absorbed([70, 5, 200], [1, 1, 1], H, dc, 16, None, single=True)
    _absorbed([70, 5, 130], [3, 5, 2], H, dc, 16, "tree")


@pytest.mark.parametrize("n", [1, 2, 5, 16, 33, 64, 65, 70, 130])
def test_absorbed_drafts(n):
    for kind in ("tree", "any", None):
        _absorbed([n + 37, n], [n, n], 2, 256, 16, kind)
    _absorbed([n + 100], [n], 5, 512, 64, "any")


@pytest.mark.parametrize("dc", [512, 256])
def test_absorbed_long_and_cut(dc):
    _absorbed([5000, 1, 0, 2049, 1025], [2, 1, 0, 3, 1], 4, dc, 16)
    _absorbed([3001], [1], 16, dc, 64, None, max_len=3001, single=True)
    _absorbed([900, 600], [20, 7], 8, dc, 1)
    _absorbed([100, 3], [20, 3], 2, dc, 16, blocks=4000)
    _absorbed([3000], [1], 3, dc, 64, None, max_len=777, single=True)


def test_absorbed_many_requests():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 200, 150)]
    _absorbed(lens, [int(min(x, y)) for x, y in zip(lens, rng.integers(0, 4, 150))], 3, 256, 16)
    lens[3], lens[90] = 2500, 3100
    _absorbed(lens, [1] * 150, 3, 256, 16, None, blocks=200, single=True)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_absorbed_not_finite_in_masked_places(value):
    """A drafted token's latent holds NaN or infinity: tokens that do not see it are as before."""
    for lens, new, H, dc in (([70, 64], [20, 3], 4, 512), ([1500], [12], 5, 256), ([200], [40], 2, 256)):
        W = dc + dc // 8
        gen, pages, _, table, keys = build(lens, new, 1, dc, 16, latent=W)
        T = sum(new)
        q = torch.randn((T, H, W), generator=gen).bfloat16()
        bits = [random_bits(n, gen, "any") for n in new]
        for b, n in enumerate(new):
            t = lens[b] - n + n // 2
            bits[b][:, n // 2] = False
            bits[b][n - 1, n // 2] = True
            keys[b][t, 3:9] = value
            pages[int(table[b, t // 16]), t % 16, 3:9] = value
        mask = torch.cat([ref.words(x, -(-max(new) // 64)) for x in bits]).cuda()
        out = torch.full((T, H, dc), 7.0, dtype=torch.bfloat16, device="cuda")
        cu = np.cumsum([0] + new).tolist()
        lib.kv_latent_attention(q.cuda(), pages.cuda(), table.cuda(), _i32(lens), out, W ** -0.5, cu_new=_i32(cu), mask=mask, max_new=max(new))
        for b, n in enumerate(new):
            k = keys[b].double()[:, None]
            o, mag, e = ref.attend(q[cu[b]:cu[b + 1] - 1].double(), torch.nan_to_num(k, nan=0.0, posinf=0.0, neginf=0.0), k[..., :dc], ref.seen(n, lens[b], bits[b])[:-1], W ** -0.5)
            ref.is_close(out[cu[b]:cu[b + 1] - 1], o, ref.tolerance(o, mag, e, lens[b], ref.BF16), f"request {b}")
            assert not bool(torch.isfinite(out[cu[b + 1] - 1, :, 3:9].float()).any())


def test_absorbed_pages_that_do_not_exist_and_equal_values():
    gen, pages, _, table, keys = build([100, 100], [10, 3], 1, 256, 16, latent=288)
    table[0, 2], table[1, 6], table[1, 0] = -3, 999, 10 ** 9
    q = torch.randn((13, 4, 288), generator=gen).bfloat16()
    out = torch.zeros((13, 4, 256), dtype=torch.bfloat16, device="cuda")
    lib.kv_latent_attention(q.cuda(), pages.cuda(), table.cuda(), _i32([100, 100]), out, 0.05, cu_new=_i32([0, 10, 13]), max_new=10)
    for b, (lo, hi, bad) in enumerate(((0, 10, (2,)), (10, 13, (0, 6)))):
        live = torch.tensor([p // 16 not in bad for p in range(100)])
        k = keys[b][live].double()[:, None]
        o, mag, e = ref.attend(q[lo:hi].double(), k, k[..., :256], ref.seen(hi - lo, 100)[:, live], 0.05)
        ref.is_close(out[lo:hi], o, ref.tolerance(o, mag, e, 100, ref.BF16), f"request {b}")
    for H in (3, 20, 70):
        pages = torch.ones((20, 64, 576), dtype=torch.bfloat16, device="cuda")
        pages[..., 512:] = torch.randn((20, 64, 64), device="cuda").bfloat16()
        q, out = torch.randn((1, H, 576), device="cuda").bfloat16(), torch.zeros((1, H, 512), dtype=torch.bfloat16, device="cuda")
        lib.kv_latent_attention(q, pages, torch.arange(20, dtype=torch.int32, device="cuda")[None], _i32([1270]), out, 0.07)
        assert bool((out == 1.0).all())


def test_absorbed_graph_and_stream():
    lens, new = [2600, 900, 3000], [2, 1, 4]
    gen, pages, _, table, _ = build(lens, new, 1, 512, 64, latent=576)
    q = torch.randn((7, 16, 576), generator=gen).bfloat16().cuda()
    pd, tab, ln, cu = pages.cuda(), table.cuda(), _i32(lens), _i32([0, 2, 3, 7])
    ws = torch.full((lib.kv_latent_attention_workspace_bytes(3, 16, 512, 4, 3000),), 255, dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    out = torch.zeros((7, 16, 512), dtype=torch.bfloat16, device="cuda")

    def run(w, **more):
        lib.kv_latent_attention(q, pd, tab, ln, out, 0.05, cu_new=cu, max_new=4, max_len=3000, workspace=w, **more)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(ws)
    for step in range(3):
        ln.copy_(_i32([2600 - 700 * step, 900 - 300 * step, 3000 - 1100 * step]))
        run(None)
        want = out.clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    s = torch.cuda.Stream()
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    run(None, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_absorbed_refusals():
    pages = torch.zeros((4, 16, 288), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 3, 288), dtype=torch.bfloat16, device="cuda")
    out, t, n, cu = q[..., :256].contiguous(), _i32([[0, 1], [2, 3]]), _i32([5, 6]), _i32([0, 1, 2])
    lib.kv_latent_attention(q, pages, t, n, out, 0.1)
    lib.kv_latent_attention(q, pages, t, n, out, 0.1, cu_new=cu)
    for bad in ((q.float(), pages, t, n, out), (q[..., :256].contiguous(), pages, t, n, out), (q, pages[0], t, n, out), (q, pages, t[0], n, out), (q, pages, t, n[:1], out),
                (q, pages, t, n, q), (q[:1], pages, t, n, out)):
        with pytest.raises((ValueError, TypeError)):
            lib.kv_latent_attention(*bad, 0.1)
    with pytest.raises(lib.DampError):
        lib.kv_latent_attention(q[:1], pages, t, n, out[:1], 0.1)
    with pytest.raises(ValueError):
        lib.kv_latent_attention(q, pages, t, n, out, 0.1, mask=torch.zeros((2, 1), dtype=torch.int64, device="cuda"))
    w = torch.zeros((4, 16, 90), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lib.DampError) as e:
        lib.kv_latent_append(torch.zeros((1, 80), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 10), dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"), w)
    assert e.value.status == lib.DAMP_ERR_UNSUPPORTED


# ---- expanded form ------------------------------------------------------------------------------------
def _prompt(nq, nk, H, d, scale=None, seed=0, form="apart", spoil=None, tail=3):
    gen = torch.Generator().manual_seed(seed + 13 * sum(nq) + d)
    Tq, Tk, dr = sum(nq), sum(nk), d // 2
    q = torch.randn((Tq + tail, H, d + dr), generator=gen).bfloat16()
    k, v = (torch.randn((Tk + tail, H, d), generator=gen).bfloat16() for _ in range(2))
    kr = torch.randn((Tk + tail, dr), generator=gen).bfloat16()
    k[Tk:], v[Tk:], kr[Tk:] = (float("nan"),) * 3
    if spoil:
        spoil(k, v, kr)
    out = torch.full((Tq + tail, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    cq, ck = np.cumsum([0] + nq).tolist(), np.cumsum([0] + nk).tolist()
    kd, vd = k.cuda(), v.cuda()
    if form == "side":                               # keys and values side by side
        kv = torch.cat([kd, vd], -1).contiguous()
        kd, vd = kv[..., :d], kv[..., d:]
    elif form == "heads":                            # heads first
        kd, vd = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (kd, vd))
    lib.kv_latent_prompt_attention(q.cuda(), kd, kr.cuda(), vd, _i32(cq), out, cu_k=None if nq is nk else _i32(ck), scale=scale)
    torch.cuda.synchronize()
    assert bool((out[Tq:] == 7.0).all())
    s = (d + dr) ** -0.5 if scale is None else scale
    used = 0.0
    for b, (n, m) in enumerate(zip(nq, nk)):
        kb = torch.cat([k[ck[b]:ck[b + 1]], kr[ck[b]:ck[b + 1], None].expand(-1, H, -1)], -1).double()
        live = torch.ones((n, m), dtype=torch.bool).tril(m - n)
        o, mag, e = ref.attend(q[cq[b]:cq[b + 1]].double(), kb, v[ck[b]:ck[b + 1]].double(), live, s)
        used = max(used, ref.is_close(out[cq[b]:cq[b + 1]], o, ref.tolerance(o, mag, e, m, ref.BF16), f"request {b}: {n} queries, {m} keys"))
    return used


LENGTHS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 257]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", ["apart", "side", "heads"])
def test_prompt_lengths(d, form):
    _prompt(LENGTHS, LENGTHS, 2, d, form=form)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_after_cached_tokens(d):
    nq = LENGTHS
    _prompt(nq, [n + x for n, x in zip(nq, [0, 5, 1, 63, 64, 65, 200, 0, 129, 1, 7, 300, 64, 31])], 2, d)
    _prompt([5, 100, 64, 3], [3, 40, 0, 2], 2, d)            # fewer keys than queries: the first see nothing


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [1, 3, 8, 16])
def test_prompt_heads_and_wide_tiles(d, H):
    _prompt([300, 129, 70], [300, 129, 70], H, d)
    n = [40] * (2 + 256 // H)                                # enough workgroups for the wider row tiles
    _prompt(n, n, H, d)


def test_prompt_long():
    _prompt([1500], [1500], 2, 128)
    _prompt([700, 900], [1200, 900], 18, 64)


@pytest.mark.parametrize("B", [1, 63, 64, 65, 200])
def test_prompt_many_requests(B):
    rng = np.random.default_rng(B)
    n = [int(x) for x in rng.integers(0, 9, B)]
    n[B // 2] = 150
    _prompt(n, n, 2, 64)


@pytest.mark.parametrize("scale", [0.02, -0.1, 0.0, 3.0])
def test_prompt_scales(scale):
    _prompt([100, 30], [100, 30], 2, 64, scale=scale)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d,H", [(64, 2), (128, 2), (128, 90)])
def test_prompt_not_finite_values(d, H, value):
    """A value that is not finite reaches the queries from its own token on, and no other."""
    def spoil(k, v, kr):
        v[50, :, 3:9], v[130, :, 20] = value, value
    n = [120, 77, 200]
    _prompt(n, n, H, d, spoil=spoil)


def test_prompt_not_finite_keys():
    n, d = [100, 60], 64
    gen = torch.Generator().manual_seed(2)
    q, k, v, kr = (torch.randn(s, generator=gen).bfloat16().cuda() for s in ((160, 2, 96), (160, 2, 64), (160, 2, 64), (160, 32)))
    cu, out, fine = _i32([0, 100, 160]), *(torch.zeros((160, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.kv_latent_prompt_attention(q, k, kr, v, cu, fine)
    k[40, 0, 3], kr[120, 5] = float("nan"), float("nan")
    lib.kv_latent_prompt_attention(q, k, kr, v, cu, out)
    assert torch.equal(out[:40], fine[:40]) and torch.equal(out[40:120, 1], fine[40:120, 1]) and torch.equal(out[100:120], fine[100:120])
    assert bool(torch.isnan(out[40:100, 0]).all()) and bool(torch.isnan(out[120:]).all())


def test_prompt_lists_that_do_not_fit_and_equal_values():
    gen = torch.Generator().manual_seed(2)
    q, k, v, kr = (torch.randn(s, generator=gen).bfloat16().cuda() for s in ((40, 2, 96), (40, 2, 64), (40, 2, 64), (40, 32)))
    out = torch.full((40, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for cu in ([0, 40, 90], [-5, 10, 40], [30, 10, 40], [0, 0, 0], [2 ** 31 - 1, 5, -2 ** 31]):
        lib.kv_latent_prompt_attention(q, k, kr, v, _i32(cu), out)
        lib.kv_latent_prompt_attention(q, k, kr, v, _i32([0, 20, 40]), out, cu_k=_i32(cu))
    lib.kv_latent_prompt_attention(q, k[:0], kr[:0], v[:0], _i32([0, 40]), out, cu_k=_i32([0, 0]))
    assert float(out.abs().max()) == 0.0
    v.fill_(1.0)
    lib.kv_latent_prompt_attention(q, k, kr, v, _i32([0, 40]), out)
    assert bool((out == 1.0).all())


def test_prompt_graph():
    gen = torch.Generator().manual_seed(2)
    q, k, v, kr = (torch.randn(s, generator=gen).bfloat16().cuda() for s in ((400, 4, 192), (400, 4, 128), (400, 4, 128), (400, 64)))
    cu, out = _i32([0, 100, 400]), torch.zeros((400, 4, 128), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.kv_latent_prompt_attention(q, k, kr, v, cu, out)
    for n in (100, 399, 17):
        cu.copy_(_i32([0, n, 400]))
        lib.kv_latent_prompt_attention(q, k, kr, v, cu, out)
        want = out.clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_prompt_refusals():
    q, k, kr = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((9, 2, 96), (9, 2, 64), (9, 32)))
    out, cu = torch.zeros_like(k), _i32([0, 9])
    lib.kv_latent_prompt_attention(q, k, kr, k, cu, out)
    for bad in ((q.float(), k, kr, k, cu, out), (q[..., :95].contiguous(), k, kr, k, cu, out), (q, k.float(), kr, k, cu, out), (q, k, kr[:8], k, cu, out),
                (q, k, kr, k[:8], cu, out), (q, k, kr, k, cu.long(), out), (q, k, kr, k, cu, out[:8]), (q, k.transpose(1, 2), kr, k, cu, out), (q, k.cpu(), kr, k, cu, out)):
        with pytest.raises((ValueError, TypeError)):
            lib.kv_latent_prompt_attention(*bad)
    odd = torch.zeros((9, 2, 67), dtype=torch.bfloat16, device="cuda")[..., :64]
    with pytest.raises(lib.DampError):
        lib.kv_latent_prompt_attention(q, odd, kr, k, cu, out)
