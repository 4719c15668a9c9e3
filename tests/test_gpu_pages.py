"""The life of the cache's pages (kv_fork_tables, kv_copy_pages, kv_compact, kv_free_pages) against lists:
whole numbers and moved rows, equal to the bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import cache_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib  # noqa: E402


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _bits(t):
    return t.cpu().view(torch.int16)


# ---- forks ----------------------------------------------------------------------------------------
def _fork(src, dst, lens, free, table, page, pages, shares=None):
    n, B = len(src), len(lens)
    tab, ln, sh = _i32(table).reshape(B, -1), _i32(lens), _i32(shares or [0] * pages)
    (cs, cd, cr), used = (_i32([77] * n) for _ in range(3)), _i32([77])
    lib.kv_fork_tables(_i32(src), _i32(dst), ln, _i32(free), tab, sh, page, cs, cd, cr, used)
    torch.cuda.synchronize()
    want = ref.fork(src, dst, lens, free, table, shares or [0] * pages, page, pages)
    assert tab.tolist() == want[0] and ln.tolist() == want[1] and sh.tolist() == want[2] and used.tolist() == [want[4]]
    assert list(zip(cs.tolist(), cd.tolist(), cr.tolist())) == want[3]


@pytest.mark.parametrize("page", [1, 16, 128])
@pytest.mark.parametrize("n", [1, 2, 63, 65, 257, 700])
def test_forks_random(n, page):
    rng = np.random.default_rng([n, page])
    B, blocks = 2 * n + 5, 9
    rows = rng.permutation(B)
    parents, dst = rows[n:], rows[:n]
    src = rng.choice(parents, n)
    lens = rng.integers(0, blocks * page + 1, B)
    pages = B * blocks + n + 3
    ids = rng.permutation(pages)
    table = ids[: B * blocks].reshape(B, blocks)
    free = ids[B * blocks:]
    _fork(src.tolist(), dst.tolist(), lens.tolist(), free.tolist(), table.tolist(), page, pages, rng.integers(0, 3, pages).tolist())


def test_forks_edges():
    t = [[3, 4, 5], [0, 1, 2], [-1, -1, -1], [-1, -1, -1]]
    _fork([0, 1], [2, 3], [20, 32, 0, 0], [7, 8], t, 16, 9)               # one partly filled, one whole
    _fork([0, 0], [2, 3], [20, 32, 0, 0], [7], t, 16, 9)                  # one page too few
    _fork([0, 0], [2, 3], [20, 32, 0, 0], [], t, 16, 9)                   # none
    _fork([0, 9, -1, 1], [2, 3, 3, 44], [20, 32, 0, 0], [7], t, 16, 9)    # rows outside the table
    _fork([0], [3], [0, 3, 4, 9], [7], t, 16, 9)                          # an empty request
    _fork([0], [3], [-4, 3, 4, 9], [7], t, 16, 9)
    _fork([0], [3], [100, 3, 4, 9], [7], t, 16, 9)                        # longer than its table
    _fork([0, 1], [2, 3], [40, 33, 0, 0], [70, 8], [[3, 99, -5], [0, 1, -2], [-1] * 3, [-1] * 3], 16, 9)   # pages that do not exist
    _fork([], [], [20, 32, 0, 0], [7], t, 16, 9)
    _fork(list(range(4000)), list(range(4000, 8000)), [3] * 8000, list(range(8000, 12000)), [[i] for i in range(8000)], 4, 12000)


def test_fork_refusals():
    z, t = _i32([0]), _i32([[0]])
    args = [z, _i32([0]), _i32([5]), z, t, z, 16, z.clone(), z.clone(), z.clone(), z.clone()]
    for i, bad in ((0, z.long()), (1, _i32([0, 0])), (2, _i32([0, 0])), (3, z.float()), (4, z), (5, t), (7, _i32([0, 0])), (10, _i32([0, 0])), (3, z.cpu())):
        with pytest.raises((ValueError, TypeError)):
            lib.kv_fork_tables(*args[:i], bad, *args[i + 1:])
    for page in (0, 24, 65536):
        with pytest.raises(lib.DampError):
            lib.kv_fork_tables(*args[:6], page, *args[7:])


# ---- copies ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("H,page,d", [(1, 1, 64), (3, 16, 128), (8, 32, 64), (2, 128, 128), (1, 64, 576), (1, 16, 8), (1, 512, 2048), (5, 4, 24)])
def test_copies(H, page, d):
    gen = torch.Generator().manual_seed(H * page + d)
    pages, n = 23, 9
    kp, vp = (torch.randn((pages, H, page, d), generator=gen).bfloat16() for _ in range(2))
    ids = torch.randperm(pages, generator=gen).tolist()
    src, dst = ids[:n], ids[n:2 * n]
    src[2], dst[3], src[4], dst[5] = -1, pages, pages + 7, -3
    rows = torch.randint(-2, page + 4, (n,), generator=gen).tolist()
    for use in (rows, None):
        wk, wv = kp.clone(), vp.clone()
        for i in range(n):
            if 0 <= src[i] < pages and 0 <= dst[i] < pages:
                m = page if use is None else min(max(use[i], 0), page)
                wk[dst[i], :, :m], wv[dst[i], :, :m] = kp[src[i], :, :m], vp[src[i], :, :m]
        gk, gv = kp.cuda(), vp.cuda()
        lib.kv_copy_pages(_i32(src), _i32(dst), gk, gv, rows=None if use is None else _i32(use))
        assert torch.equal(_bits(gk), _bits(wk)) and torch.equal(_bits(gv), _bits(wv))
        if H == 1:
            one = kp[:, 0].contiguous().cuda()
            lib.kv_copy_pages(_i32(src), _i32(dst), one, rows=None if use is None else _i32(use))
            assert torch.equal(_bits(one), _bits(wk[:, 0].contiguous()))
    lib.kv_copy_pages(_i32([]), _i32([]), gk, gv)


def test_copy_to_its_own_page_and_many():
    kp = torch.arange(5000 * 4 * 8, dtype=torch.float32).reshape(5000, 4, 8).bfloat16().cuda()
    want = kp.clone()
    want[2500:] = kp[:2500]
    lib.kv_copy_pages(torch.arange(2500, dtype=torch.int32, device="cuda"), torch.arange(2500, 5000, dtype=torch.int32, device="cuda"), kp)
    assert torch.equal(kp, want)
    lib.kv_copy_pages(_i32([3, 4]), _i32([3, 4]), kp)
    assert torch.equal(kp, want)


def test_copy_past_32_bits():
    """Pages whose byte offsets pass 2^32."""
    pages, page = 70000, 64
    k = torch.zeros((pages, page, 576), dtype=torch.bfloat16, device="cuda")
    assert k.numel() * 2 > 2 ** 32
    k[pages - 1] = 3.0
    k[5] = 2.0
    lib.kv_copy_pages(_i32([pages - 1, 5]), _i32([1, pages - 2]), k)
    assert bool((k[1] == 3.0).all()) and bool((k[pages - 2] == 2.0).all()) and float(k[6:pages - 2].abs().max()) == 0.0


# ---- kept tokens ------------------------------------------------------------------------------------
def _compact(lens, new, kept, H, page, d, seed=0, bad=()):
    gen = torch.Generator().manual_seed(seed + d + page)
    B = len(lens)
    blocks = max([-(-n // page) for n in lens] + [1]) + 1
    pages = B * blocks + 2
    table = torch.randperm(pages, generator=gen)[: B * blocks].reshape(B, blocks).to(torch.int32)
    for b, j in bad:
        table[b, j] = pages + 3 if j % 2 else -1
    kp, vp = (torch.randn((pages, H, page, d), generator=gen).bfloat16() for _ in range(2))
    wk, wv = kp.clone(), vp.clone()
    out = []
    for b, n in enumerate(lens):
        m = min(max(new[b], 0), max(n, 0))
        base = max(n, 0) - m
        out.append(base + min(len(kept[b]), m))
        for j, x in enumerate(kept[b][:m]):
            old, to = base + x, base + j
            if x >= m:
                continue
            po, pt = int(table[b, old // page]), int(table[b, to // page])
            if 0 <= po < pages and 0 <= pt < pages:
                wk[pt, :, to % page], wv[pt, :, to % page] = kp[po, :, old % page], vp[po, :, old % page]
    cu = np.cumsum([0] + [len(x) for x in kept]).tolist()
    flat = [x for r in kept for x in r]
    gk, gv, ol = kp.cuda(), vp.cuda(), _i32([77] * B)
    lib.kv_compact(_i32(flat), _i32(cu), _i32(lens), _i32(new), table.cuda(), gk, gv, ol)
    assert ol.tolist() == out
    assert torch.equal(_bits(gk), _bits(wk)) and torch.equal(_bits(gv), _bits(wv))
    if H == 1:
        one = kp[:, 0].contiguous().cuda()
        lib.kv_compact(_i32(flat), _i32(cu), _i32(lens), _i32(new), table.cuda(), one, None, ol)
        assert torch.equal(_bits(one), _bits(wk[:, 0].contiguous()))


@pytest.mark.parametrize("H,page,d", [(1, 1, 64), (3, 16, 128), (8, 32, 64), (1, 64, 576), (2, 8, 8), (1, 4, 2048), (1, 16, 24)])
def test_kept_random(H, page, d):
    rng = np.random.default_rng([H, page, d])
    lens = [0, 1, 2, 7, 33, 64, 65, 129, 300, 513]
    new = [0, 1, 1, 7, 12, 64, 40, 129, 300, 200]
    kept = [[j for j in range(m) if rng.random() < p] for m, p in zip(new, [0, 1, 0, 0.4, 0.5, 0.9, 0.2, 0.5, 0.5, 0.7])]
    _compact(lens, new, kept, H, page, d)
    _compact(lens, new, [list(range(m)) for m in new], H, page, d)                # all
    _compact(lens, new, [[] for m in new], H, page, d)                            # none
    _compact(lens, new, [list(range(m // 2, m)) for m in new], H, page, d)        # a run moved down
    _compact(lens, new, [list(range(1, m)) for m in new], H, page, d)             # all by one


def test_kept_long_and_odd_lists():
    rng = np.random.default_rng(4)
    kept = np.nonzero(rng.random(5000) < 0.5)[0].tolist()
    _compact([5000, 900], [5000, 900], [kept, list(range(0, 900, 3))], 2, 16, 128)
    _compact([40, 30], [8, 50], [[0, 3, 8, 9], [1, 5, 29]], 1, 16, 64)            # entries past the new tokens; more new than tokens
    _compact([40, 30], [40, 30], [[1, 20, 39], [2, 3, 17]], 1, 16, 64, bad=[(0, 1), (1, 0)])


def test_kept_lists_outside_the_array():
    kp = torch.randn((8, 1, 16, 64)).bfloat16().cuda()
    want, ol = kp.clone(), _i32([7, 7])
    lib.kv_compact(_i32([0, 1]), _i32([-5, 1, 900]), _i32([20, 20]), _i32([2, 2]), _i32([[0, 1], [2, 3]]), kp, kp.clone(), ol)
    assert ol.tolist() == [19, 19]
    want[3, :, 2] = want[3, :, 3]                                # request 1 keeps its second new token: 18 <- 19
    assert torch.equal(_bits(kp), _bits(want))


# ---- pages given back ----------------------------------------------------------------------------------
def _free(keep, lens, table, shares, page):
    pages = len(shares)
    sh, freed, count = _i32(shares), torch.full((pages,), -9, dtype=torch.int32, device="cuda"), _i32([-9])
    tab = _i32(table).reshape(len(lens), len(table[0]) if table else 3)
    was = tab.clone()
    lib.kv_free_pages(_i32(keep) if keep is not None else None, _i32(lens), tab, sh, page, freed, count)
    left, gone = ref.release(keep, lens, table, shares, page)
    assert count.tolist() == [len(gone)] and freed.tolist() == gone + [-9] * (pages - len(gone)) and sh.tolist() == left
    assert torch.equal(tab, was)


@pytest.mark.parametrize("pages", [1, 63, 4096, 4097, 8192, 8193, 20000, 65536, 65537, 300000])
def test_free_random(pages):
    rng = np.random.default_rng(pages)
    B, page = min(pages, 40), 16
    blocks = max(1, min(pages // B, 50))
    ids = rng.permutation(pages)[: B * blocks]
    table = ids.reshape(B, blocks)
    lens = rng.integers(0, blocks * page + 1, B)
    keep = (lens * rng.random(B)).astype(int)
    shares = (rng.random(pages) < 0.3) * rng.integers(1, 4, pages)
    _free(keep.tolist(), lens.tolist(), table.tolist(), shares.tolist(), page)
    _free(None, lens.tolist(), table.tolist(), shares.tolist(), page)


def test_free_shared_by_many_in_one_call():
    """Every request gives back the same pages; those with as many shares as holders but one are released once."""
    B = 300
    table = [[0, 1, 2, 3, 5 + b] for b in range(B)]
    shares = [B - 1, B, B - 2, 0, 7] + [0] * B
    _free(None, [80] * B, table, shares, 16)
    _free([16] * B, [80] * B, table, shares, 16)
    _free([80] * B, [80] * B, table, shares, 16)


def test_free_edges():
    t = [[3, 4, 5], [0, -1, 99]]
    _free([0, 0], [48, 48], t, [0] * 7, 16)
    _free([17, 100], [33, 48], t, [0] * 7, 16)
    _free([-3, 1], [200, -2], t, [0] * 7, 16)
    _free([0, 0], [5, 5], t, [0] * 7, 1)
    _free(None, [], [], [0] * 7, 16)
    _free([48, 48], [48, 48], t, [0] * 7, 16)


def test_free_workspace_and_refusals():
    assert lib.kv_free_pages_workspace_bytes(8192) == 0 and lib.kv_free_pages_workspace_bytes(8193) > 0
    z, t = _i32([0]), _i32([[0]])
    args = [z, _i32([5]), t, z, 16, z.clone(), z.clone()]
    for i, bad in ((0, _i32([0, 0])), (1, z.float()), (2, z), (3, t), (5, _i32([0, 0])), (6, _i32([0, 0])), (5, z.cpu())):
        with pytest.raises((ValueError, TypeError)):
            lib.kv_free_pages(*args[:i], bad, *args[i + 1:])
    with pytest.raises(ValueError):
        lib.kv_free_pages(None, _i32([5]), t, torch.zeros(70000, dtype=torch.int32, device="cuda"), 16, torch.zeros(70000, dtype=torch.int32, device="cuda"), z.clone(),
                          workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))


def test_fork_copy_keep_and_free_in_a_graph():
    """Captured once, replayed with other contents."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    pages, page, H, d, B = 70000, 16, 2, 64, 6
    kp, vp = (torch.randn((pages, H, page, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(pages, device="cuda", generator=gen)[: B * 8].reshape(B, 8).to(torch.int32)
    free = torch.arange(60000, 60010, dtype=torch.int32, device="cuda")
    lens, shares = _i32([100, 47, 0, 0, 64, 30]), torch.zeros(pages, dtype=torch.int32, device="cuda")
    src, dst = _i32([0, 1]), _i32([2, 3])
    cs, cd, cr = (torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(3))
    used, count, ol = _i32([0]), _i32([0]), torch.zeros(B, dtype=torch.int32, device="cuda")
    freed = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    kept, cu, new = _i32([1, 3, 0, 2]), _i32([0, 2, 2, 2, 2, 4, 4]), _i32([6, 2, 0, 0, 5, 1])
    state = [kp, vp, table, lens, shares, cs, cd, cr, used, count, ol, freed]

    def run():
        lib.kv_fork_tables(src, dst, lens, free, table, shares, page, cs, cd, cr, used)
        lib.kv_copy_pages(cs, cd, kp, vp, rows=cr)
        lib.kv_compact(kept, cu, lens, new, table, kp, vp, ol)
        lib.kv_free_pages(ol, lens, table, shares, page, freed, count)

    start = [t.clone() for t in state]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for n in (100, 31, 80):
        start[3][0] = n
        for t, s in zip(state, start):
            t.copy_(s)
        run()
        torch.cuda.synchronize()
        want = [t.clone() for t in state]
        for t, s in zip(state, start):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(state, want):
            assert torch.equal(t, w)
