"""Attention of several new tokens over a paged cache (kv_tree_attention) against binary64: masks and runs in
order, rows that see nothing, lengths and drafts around every tile border, pages, heads, cut requests.
Bounds: cache_ref.tolerance; the weights are two bf16 pieces, good to 2^-15 + 2^-20, or one rounding."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import cache_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib  # noqa: E402

PIECES = 2.0 ** -15 + 2.0 ** -20


def weight(rows):
    """What a weight is off by: two bf16 pieces for up to 16 query rows a key-value head, one rounding for more."""
    return PIECES if rows <= 16 else ref.BF16



def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def build(lens, new, Hkv, d, page, seed=0, latent=0, poison=True, blocks=None):
    """Pages, table and each request's keys and values (NaN wherever no token lies)."""
    gen = torch.Generator().manual_seed(seed + 7 * sum(lens) + d)
    need = [-(-n // page) for n in lens]
    blocks = blocks or max(need + [1]) + 1
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=gen).tolist()
    fill = float("nan") if poison else 0.0
    shape = (pages, page, latent) if latent else (pages, Hkv, page, d)
    kp, vp = (torch.full(shape, fill, dtype=torch.bfloat16) for _ in range(2))
    table = torch.full((len(lens), blocks), -1, dtype=torch.int32)
    keys, at = [], 0
    for b, n in enumerate(lens):
        table[b, : need[b]] = torch.tensor(ids[at:at + need[b]], dtype=torch.int32)
        at += need[b]
        pos = torch.arange(n)
        p = table[b, pos // page].long()
        if latent:
            k = torch.randn((n, latent), generator=gen).bfloat16()
            kp[p, pos % page] = k
            keys.append(k)
        else:
            k, v = (torch.randn((n, Hkv, d), generator=gen).bfloat16() for _ in range(2))
            kp[p, :, pos % page], vp[p, :, pos % page] = k, v
            keys.append((k, v))
    return gen, kp, vp, table, keys


def random_bits(n, gen, kind):
    """[n, n] truth values: a random tree's ancestors, or any pattern with empty rows."""
    if kind == "tree":
        bits = torch.eye(n, dtype=torch.bool)
        for i in range(1, n):
            p = int(torch.randint(-1, i, (1,), generator=gen))
            if p >= 0:
                bits[i] |= bits[p]
        return bits
    bits = torch.rand((n, n), generator=gen) < 0.4
    bits[torch.rand(n, generator=gen) < 0.3] = False
    return bits


def _attend(lens, new, Hq, Hkv, d, page, kind="tree", scale=None, max_len=None, max_new=None, seed=0, blocks=None, spoil=None, odd_words=0, big=1.0):
    gen, kp, vp, table, keys = build(lens, new, Hkv, d, page, seed, blocks=blocks)
    T = sum(new)
    q = (big * torch.randn((T + 3, Hq, d), generator=gen)).bfloat16()
    most = max(new + [1])
    words = -(-most // 64) + odd_words
    bits = [None if kind is None else random_bits(n, gen, kind) for n in new]
    if spoil:
        spoil(kp, vp, table, keys, bits)
    mask = None
    if kind is not None:
        mask = torch.full((T + 3, words), -1, dtype=torch.int64)
        for b, n in enumerate(new):
            at = sum(new[:b])
            mask[at:at + n] = ref.words(bits[b], words)
    out = torch.full((T + 3, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = np.cumsum([0] + new).tolist()
    kd, vd = kp.cuda(), vp.cuda()
    lib.kv_tree_attention(q.cuda(), kd, vd, table.cuda(), _i32(lens), _i32(cu), out, mask=None if mask is None else mask.cuda(),
                          max_new=most if max_new is None else max_new, scale=scale, max_len=max_len)
    torch.cuda.synchronize()
    assert torch.equal(kd.cpu().view(torch.int16), kp.view(torch.int16)) and torch.equal(vd.cpu().view(torch.int16), vp.view(torch.int16))
    assert bool((out[T:] == 7.0).all()), "rows behind the last request were written"
    s = d ** -0.5 if scale is None else scale
    used = 0.0
    for b, n in enumerate(new):
        live = ref.seen(n, lens[b], bits[b])
        m = lens[b] if max_len is None else min(lens[b], max_len)
        k, v = (x[:m].double() for x in keys[b])
        o, mag, e = ref.attend(q[cu[b]:cu[b + 1]].double(), k, v, live[:, :m], s)
        used = max(used, ref.is_close(out[cu[b]:cu[b + 1]], o, ref.tolerance(o, mag, e, m, weight(most * Hq // Hkv)), f"request {b}: {n} of {lens[b]} tokens"))
    return used


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 8, 16, 64])
@pytest.mark.parametrize("kind", ["tree", "any", None])
def test_lengths(d, page, kind):
    lens = [0, 1, 1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 300]
    new = [0, 0, 1, 2, 5, 16, 3, 7, 32, 33, 1, 40, 17, 2, 64, 9]
    _attend(lens, new, 4, 2, d, page, kind)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (3, 1), (7, 1), (16, 1), (17, 1), (40, 1), (32, 8), (10, 5)])
def test_heads(d, Hq, Hkv):
    _attend([129, 5, 260], [6, 5, 13], Hq, Hkv, d, 16)


@pytest.mark.parametrize("n", [1, 2, 4, 5, 8, 9, 16, 31, 63, 64, 65, 100, 128, 130, 200])
def test_drafts(n):
    """Around every number of rows from which a workgroup takes more, masks of one to four words."""
    for kind in ("tree", "any", None):
        _attend([n + 37, n, n + 200], [n, n, 1], 4, 1, 64, 16, kind)
    _attend([n + 37], [n], 8, 2, 128, 16, "any", odd_words=1)


@pytest.mark.parametrize("d", [64, 128])
def test_long_and_cut(d):
    _attend([5000, 1, 0, 2049, 1025], [12, 1, 0, 3, 16], 4, 1, d, 16)
    _attend([3001], [5], 8, 2, d, 32, max_len=3001)
    _attend([3001, 2900], [30, 7], 8, 2, d, 1)
    _attend([100, 3], [20, 3], 2, 1, d, 16, blocks=4000)            # a table far wider than the requests


def test_many_requests():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 300, 200)]
    _attend(lens, [int(min(x, y)) for x, y in zip(lens, rng.integers(0, 6, 200))], 2, 1, 64, 16)
    lens[3], lens[90] = 2500, 3100
    _attend(lens, [int(min(x, y)) for x, y in zip(lens, rng.integers(0, 6, 200))], 4, 2, 64, 16, blocks=200)


def test_a_row_sees_nothing():
    """A mask of zeros and no context: 0, whatever the keys hold."""
    for n in (1, 5, 40):
        gen, kp, vp, table, _ = build([n], [n], 1, 64, 16)
        q = torch.randn((n, 2, 64), generator=gen).bfloat16().cuda()
        out = torch.full_like(q, 7.0)
        lib.kv_tree_attention(q, kp.cuda(), vp.cuda(), table.cuda(), _i32([n]), _i32([0, n]), out, mask=torch.zeros((n, 1), dtype=torch.int64, device="cuda"))
        assert float(out.abs().max()) == 0.0


@pytest.mark.parametrize("what", ["v", "k", "both"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_in_masked_places(what, value):
    """A drafted token that some do not see holds a NaN or an infinity: those are as if it held anything else."""
    def spoil(kp, vp, table, keys, bits):
        for b, (k, v) in enumerate(keys):
            n = len(bits[b])
            if n < 3:
                continue
            t = k.shape[0] - n + n // 2
            bits_col = bits[b][:, n // 2]
            bits_col[: n - 1] = False                 # only the last token sees it
            bits_col[n - 1] = True
            p, row = int(table[b, t // 16]), t % 16
            if what != "k":
                v[t, :, 3:9] = value
                vp[p, :, row, 3:9] = value
            if what != "v":
                k[t, :, 5] = float("nan")
                kp[p, :, row, 5] = float("nan")
    if what == "v":
        _attend([70, 33, 1500, 64], [20, 33, 12, 3], 4, 2, 64, 16, "any", spoil=spoil)
        _attend([70, 200], [20, 9], 8, 1, 128, 16, "any", spoil=spoil)
    else:
        # the token that sees the key has no finite readout; the others must
        gen, kp, vp, table, keys = build([70], [20], 1, 64, 16)
        bits = [torch.ones((20, 20), dtype=torch.bool)]
        spoil(kp, vp, table, keys, bits)
        q = torch.randn((20, 2, 64), generator=gen).bfloat16()
        out = torch.full((20, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lib.kv_tree_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32([70]), _i32([0, 20]), out, mask=ref.words(bits[0]).cuda())
        o, mag, e = ref.attend(q[:19].double(), *(x.double() for x in keys[0]), ref.seen(20, 70, bits[0])[:19], 64 ** -0.5)
        ref.is_close(out[:19], o, ref.tolerance(o, mag, e, 70, weight(40)), what)
        assert bool(torch.isnan(out[19].float()).all())


def test_not_finite_in_the_context():
    """A value before the drafted tokens, in the tile that the first of them lies in."""
    def spoil(kp, vp, table, keys, bits):
        k, v = keys[0]
        for t in (30, 33, 44):
            v[t, :, t % 7] = float("inf")
            vp[int(table[0, t // 16]), :, t % 16, t % 7] = float("inf")
    _attend([70], [25], 4, 2, 64, 16, "tree", spoil=spoil)
    _attend([46], [1], 4, 2, 128, 16, "tree", spoil=spoil)


def test_pages_that_do_not_exist():
    gen, kp, vp, table, keys = build([100, 100], [10, 3], 2, 64, 16)
    table[0, 2], table[1, 6], table[1, 0] = -3, 999, 10 ** 9
    q = torch.randn((13, 4, 64), generator=gen).bfloat16()
    out = torch.zeros((13, 4, 64), dtype=torch.bfloat16, device="cuda")
    lib.kv_tree_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32([100, 100]), _i32([0, 10, 13]), out, max_new=10)
    for b, (lo, hi, bad) in enumerate(((0, 10, (2,)), (10, 13, (0, 6)))):
        live = torch.tensor([p // 16 not in bad for p in range(100)])
        k, v = (x[live].double() for x in keys[b])
        o, mag, e = ref.attend(q[lo:hi].double(), k, v, ref.seen(hi - lo, 100)[:, live], 64 ** -0.5)
        ref.is_close(out[lo:hi], o, ref.tolerance(o, mag, e, 100, weight(20)), f"request {b}")


def test_lengths_that_do_not_fit():
    """More new tokens than tokens, or than max_new; lists outside the rows; nothing is read or written outside."""
    gen, kp, vp, table, keys = build([5, 40], [5, 4], 2, 64, 16)
    q = torch.randn((12, 4, 64), generator=gen).bfloat16()

    def run(lens, cu, **more):
        out = torch.full((12, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lib.kv_tree_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32(lens), _i32(cu), out, **more)
        torch.cuda.synchronize()
        return out
    out = run([5, 40], [0, 8, 12])                        # 8 new tokens of 5: the first 3 have no position
    o, mag, e = ref.attend(q[:8].double(), *(x.double() for x in keys[0]), ref.seen(8, 5), 64 ** -0.5)
    assert float(out[:3].abs().max()) == 0.0
    ref.is_close(out[:8], o, ref.tolerance(o, mag, e, 5, weight(24)), "8 of 5")
    out = run([5, 40], [0, 5, 9], max_new=2)               # later ones get no readout
    assert bool((out[2:5] == 7.0).all()) and bool((out[7:] == 7.0).all()) and not bool((out[:2] == 7.0).any())
    whole = run([5, 40], [0, 5, 9])
    for b, (at, n, m) in enumerate(((0, 5, 5), (5, 4, 40))):    # (other bounds may take other kernels: the same values, not the same bits)
        o, mag, e = ref.attend(q[at:at + n].double(), *(x.double() for x in keys[b]), ref.seen(n, m), 64 ** -0.5)
        tol = ref.tolerance(o, mag, e, m, weight(24))
        ref.is_close(whole[at:at + n], o, tol, "all")
        ref.is_close(out[at:at + 2], o[:2], tol[:2], "the first two")
    out = run([5, 40], [-7, 5, 900])
    assert torch.equal(out[:5], whole[:5])
    run([5, 40], [9, 3, 1])
    run([-3, 40], [0, 5, 9])
    assert torch.equal(run([5, 40], [0, 5, 9], max_new=0), torch.full_like(out, 7.0))


def test_as_the_attention_of_one_token():
    """One new token each, without a mask: the weights and sums of kv_decode_attention, at the same bounds."""
    lens = [700, 1, 33, 2500]
    gen, kp, vp, table, _ = build(lens, [1] * 4, 2, 128, 16)
    q = torch.randn((4, 8, 128), generator=gen).bfloat16().cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    kd, vd = kp.cuda(), vp.cuda()
    lib.kv_decode_attention(q, kd, vd, table.cuda(), _i32(lens), a)
    lib.kv_tree_attention(q, kd, vd, table.cuda(), _i32(lens), _i32([0, 1, 2, 3, 4]), b, max_new=1)
    assert float((a.float() - b.float()).abs().max()) <= 2 * ref.BF16 * float(a.float().abs().max())


def test_equal_values_come_back():
    for n in (3, 40):
        gen, kp, vp, table, _ = build([900, 60], [n, n], 1, 64, 16, poison=False)
        vp.fill_(1.0)
        q = torch.randn((2 * n, 4, 64), generator=gen).bfloat16().cuda()
        out = torch.zeros_like(q)
        lib.kv_tree_attention(q, kp.cuda(), vp.cuda(), table.cuda(), _i32([900, 60]), _i32([0, n, 2 * n]), out, max_new=n)
        assert bool((out == 1.0).all())


def test_graph_other_stream_and_shared_workspace():
    """Two captured calls share a workspace; replays with other lengths and masks are the eager calls' bits."""
    lens, new = [2600, 900, 3000], [12, 3, 20]
    gen, kp, vp, table, _ = build(lens, new, 2, 128, 16)
    T = sum(new)
    q = torch.randn((T, 8, 128), generator=gen).bfloat16().cuda()
    kd, vd, tab, ln, cu = kp.cuda(), vp.cuda(), table.cuda(), _i32(lens), _i32([0, 12, 15, 35])
    mask = torch.randint(-2 ** 62, 2 ** 62, (T, 1), generator=gen).cuda()
    need = max(lib.kv_tree_attention_workspace_bytes(3, 8, 2, 128, 20, 3200), lib.kv_tree_attention_workspace_bytes(3, 8, 2, 128, 35, 3200))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    assert need > 0
    outs = [torch.zeros_like(q) for _ in range(2)]

    def run(i, w):
        lib.kv_tree_attention(q, kd, vd, tab, ln, cu, outs[i], mask=mask if i else None, max_new=20, max_len=3200, workspace=w)
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(i, ws)
        graphs.append(g)
    for step in range(3):
        ln.copy_(_i32([2600 - 500 * step, 900 - 300 * step, 3000 - 1000 * step]))
        mask.copy_(torch.randint(-2 ** 62, 2 ** 62, (T, 1), generator=gen))
        want = []
        for i in range(2):
            run(i, None)
            want.append(outs[i].clone())
            outs[i].zero_()
        for i in (1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs[0].zero_()
    s.wait_stream(torch.cuda.current_stream())
    lib.kv_tree_attention(q, kd, vd, tab, ln, cu, outs[0], max_new=20, max_len=3200, stream=s)
    s.synchronize()
    assert torch.equal(outs[0], want[0])


def test_refusals():
    gen, kp, vp, table, _ = build([20, 20], [3, 2], 2, 64, 16)
    kd, vd = kp.cuda(), vp.cuda()
    q = torch.zeros((5, 4, 64), dtype=torch.bfloat16, device="cuda")
    args = [q, kd, vd, table.cuda(), _i32([20, 20]), _i32([0, 3, 5]), torch.empty_like(q)]
    lib.kv_tree_attention(*args)
    for i, bad in ((0, q.float()), (0, q[:, :, :32].contiguous()), (1, kd.float()), (2, vd[:1]), (3, _i32([0])), (4, _i32([20])), (5, _i32([0, 3])), (6, q[:3]), (6, q.cpu()),
                   (0, q.transpose(0, 1))):
        with pytest.raises((ValueError, TypeError)):
            lib.kv_tree_attention(*args[:i], bad, *args[i + 1:])
    for mask in (torch.zeros((5, 1), dtype=torch.int32, device="cuda"), torch.zeros((4, 1), dtype=torch.int64, device="cuda"), torch.zeros(5, dtype=torch.int64, device="cuda"),
                 torch.zeros((5, 0), dtype=torch.int64, device="cuda")):
        with pytest.raises((ValueError, TypeError)):
            lib.kv_tree_attention(*args, mask=mask)
    with pytest.raises((ValueError, TypeError)):
        lib.kv_tree_attention(q[:, :3].contiguous(), *args[1:])
    with pytest.raises(lib.DampError):
        lib.kv_tree_attention(q[:, :3].contiguous(), *args[1:6], q[:, :3].contiguous())
    with pytest.raises(lib.DampError):
        lib.kv_tree_attention(*args, max_new=-1)
