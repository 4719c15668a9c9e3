"""The calls on a shared and drafted cache as a server makes them, one after the other: requests are forked,
drafts stored, attended to as trees, kept or dropped, and pages given back, against a model of the
cache in plain lists; latents read in both forms; two threads; caches past 2^32 bytes; least alignment; scores
that rise from tile to tile; values that are not finite beside pages that do not exist.
Bounds: cache_ref.tolerance, as in the tests of the single calls."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import cache_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib  # noqa: E402
from test_gpu_latent import _absorbed  # noqa: E402
from test_gpu_tree import _attend, _i32, build, random_bits, weight  # noqa: E402


class Server:
    """Requests as lists of (key, value) rows on the host, and the paged cache on the device."""

    def __init__(self, B, Hq, Hkv, d, page, pages, blocks, seed):
        self.gen = torch.Generator().manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.d, self.page, self.B = Hq, Hkv, d, page, B
        self.k, self.v = (torch.full((pages, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
        self.shares = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.free = list(self.rng.permutation(pages))
        self.rows = [([], []) for _ in range(B)]

    def lens(self):
        return [len(r[0]) for r in self.rows]

    def random(self, *shape):
        return torch.randn(shape, generator=self.gen).bfloat16()

    def append(self, new):
        """`new[b]` drafted tokens each, stored in pages that are taken where the last one is full."""
        old, T = self.lens(), sum(new)
        slots, used = torch.zeros(T, dtype=torch.int64, device="cuda"), _i32([0])
        lib.kv_build_tables(_i32([a + b for a, b in zip(old, new)]), _i32(new), _i32([int(x) for x in self.free]), self.table, self.page, slots, None, torch.zeros(self.B + 1, dtype=torch.int32, device="cuda"), used)
        del self.free[:used.item()]
        k, v = self.random(T, self.Hkv, self.d), self.random(T, self.Hkv, self.d)
        lib.kv_append(k.cuda(), v.cuda(), slots, self.k, self.v)
        at = 0
        for r, n in zip(self.rows, new):
            r[0].extend(k[at:at + n])
            r[1].extend(v[at:at + n])
            at += n

    def attend(self, new, kind):
        T, most = sum(new), max(new + [1])
        q = self.random(T, self.Hq, self.d)
        bits = [random_bits(n, self.gen, kind) if kind else None for n in new]
        mask = torch.cat([ref.words(x, -(-most // 64)) for x in bits]).cuda() if kind else None
        out = torch.full_like(q, 7.0, device="cuda")
        cu = np.cumsum([0] + new).tolist()
        lib.kv_tree_attention(q.cuda(), self.k, self.v, self.table, _i32(self.lens()), _i32(cu), out, mask=mask, max_new=most)
        for b, n in enumerate(new):
            m = len(self.rows[b][0])
            if n == 0 or m == 0:
                continue
            k, v = (torch.stack(x).double() for x in self.rows[b])
            o, mag, e = ref.attend(q[cu[b]:cu[b + 1]].double(), k, v, ref.seen(n, m, bits[b]), self.d ** -0.5)
            ref.is_close(out[cu[b]:cu[b + 1]], o, ref.tolerance(o, mag, e, m, weight(most * self.Hq // self.Hkv)), f"request {b}: {n} of {m}")

    def keep(self, new):
        """Some of the drafted tokens are kept; the pages behind them are given back."""
        old = self.lens()
        kept = [sorted(self.rng.choice(n, int(self.rng.integers(0, n + 1)), replace=False).tolist()) if n else [] for n in new]
        out = torch.zeros(self.B, dtype=torch.int32, device="cuda")
        lib.kv_compact(_i32(sum(kept, [])), _i32(np.cumsum([0] + [len(x) for x in kept]).tolist()), _i32(old), _i32(new), self.table, self.k, self.v, out)
        for r, n, x in zip(self.rows, new, kept):
            base = len(r[0]) - n
            for side in r:
                side[base:] = [side[base + i] for i in x]
        assert out.tolist() == self.lens()
        self.give_back(out, old)

    def give_back(self, keep, old):
        freed, count = torch.full_like(self.shares, -9), _i32([-9])
        lib.kv_free_pages(keep, _i32(old), self.table, self.shares, self.page, freed, count)
        gone = freed[:count.item()].tolist()
        assert not set(gone) & set(self.free) and len(set(gone)) == len(gone)
        self.free += gone

    def drop(self, b):
        old = [len(r[0]) if i == b else 0 for i, r in enumerate(self.rows)]
        self.rows[b] = ([], [])
        self.give_back(None, old)

    def fork(self, pairs):
        n = len(pairs)
        cs, cd, cr = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(3))
        lens, used = _i32(self.lens()), _i32([0])
        lib.kv_fork_tables(_i32([a for a, _ in pairs]), _i32([b for _, b in pairs]), lens, _i32([int(x) for x in self.free]), self.table, self.shares, self.page, cs, cd, cr, used)
        lib.kv_copy_pages(cs, cd, self.k, self.v, rows=cr)
        del self.free[:used.item()]
        for a, b in pairs:
            self.rows[b] = tuple(list(x) for x in self.rows[a])
        assert lens.tolist() == self.lens()

    def check(self):
        """The cache holds what the lists hold, and no page is lost or held by more than its shares say."""
        table, holders = self.table.cpu(), {}
        k, v = self.k.cpu(), self.v.cpu()
        for b, (ks, vs) in enumerate(self.rows):
            for j in range(-(-len(ks) // self.page)):
                holders[int(table[b, j])] = holders.get(int(table[b, j]), 0) + 1
            for t, (x, y) in enumerate(zip(ks, vs)):
                p = int(table[b, t // self.page])
                assert torch.equal(k[p, :, t % self.page], x) and torch.equal(v[p, :, t % self.page], y), (b, t)
        shares = self.shares.tolist()
        assert all(shares[p] == n - 1 for p, n in holders.items()) and sum(shares) == sum(n - 1 for n in holders.values())
        assert sorted(list(holders) + [int(x) for x in self.free]) == list(range(len(shares)))


@pytest.mark.parametrize("Hq,Hkv,d,page", [(4, 2, 64, 16), (8, 1, 128, 4), (16, 2, 64, 64)])
def test_a_server_s_rounds(Hq, Hkv, d, page):
    s = Server(6, Hq, Hkv, d, page, 900 // page + 60, 400 // page + 2, seed=d + page)
    s.append([130, 1, 0, 64, 0, 0])
    s.check()
    s.fork([(0, 2), (3, 4)])
    s.check()
    for turn in range(4):
        new = [int(x) if len(r[0]) else 0 for x, r in zip(s.rng.integers(0, 14, 6), s.rows)]
        s.append(new)
        s.attend(new, ("tree", "any", None, "tree")[turn])
        s.keep(new)
        s.check()
        if turn == 1:
            s.fork([(2, 5)])
            s.drop(3)
        s.check()
    for b in range(6):
        s.drop(b)
    s.check()
    assert len(s.free) == s.shares.numel() and not s.shares.any()


@pytest.mark.parametrize("n,H", [([5, 1, 64], 2), ([33, 0, 130], 4)])
def test_latents_in_both_forms(n, H):
    """Up-projections that select channels: absorbed queries are the expanded ones in their head's channels, and
    a head's readout is its channels of the latents' (values are the keys' channels here)."""
    dc, d, dr, page = 512, 128, 64, 16
    gen = torch.Generator().manual_seed(sum(n))
    T = sum(n)
    cached = [40, 7, 200]
    c, kr = (torch.randn((T + sum(cached), w), generator=gen).bfloat16().cuda() for w in (dc, dr))
    q = torch.randn((T, H, d + dr), generator=gen).bfloat16().cuda()
    lens = [a + b for a, b in zip(cached, n)]
    blocks = max(-(-x // page) for x in lens)
    table = torch.randperm(3 * blocks, generator=gen).to(torch.int32).reshape(3, blocks).cuda()
    pages = torch.full((3 * blocks, page, dc + dr), float("nan"), dtype=torch.bfloat16, device="cuda")
    cu_k = np.cumsum([0] + lens).tolist()
    slots = torch.cat([table[b, torch.arange(m, device="cuda") // page].long() * page + torch.arange(m, device="cuda") % page for b, m in enumerate(lens)])
    lib.kv_latent_append(c, kr, slots, pages)
    cu = _i32(np.cumsum([0] + n).tolist())
    k = c.view(-1, 4, d)[:, :H].contiguous()
    out = torch.zeros((T, H, d), dtype=torch.bfloat16, device="cuda")
    lib.kv_latent_prompt_attention(q, k, kr, k, cu, out, cu_k=_i32(cu_k))
    absorbed = torch.zeros((T, H, dc + dr), dtype=torch.bfloat16, device="cuda")
    for h in range(H):
        absorbed[:, h, h * d:(h + 1) * d] = q[:, h, :d]
    absorbed[:, :, dc:] = q[:, :, d:]
    wide = torch.zeros((T, H, dc), dtype=torch.bfloat16, device="cuda")
    lib.kv_latent_attention(absorbed, pages, table, _i32(lens), wide, (d + dr) ** -0.5, cu_new=cu, max_new=max(n))
    other = torch.stack([wide[:, h, h * d:(h + 1) * d] for h in range(H)], 1)
    at = 0
    for b, x in enumerate(n):
        if x == 0:
            continue
        kb = k[cu_k[b]:cu_k[b + 1]].cpu().double()
        keys = torch.cat([kb, kr[cu_k[b]:cu_k[b + 1], None].cpu().double().expand(-1, H, -1)], -1)
        live = torch.ones((x, lens[b]), dtype=torch.bool).tril(lens[b] - x)
        o, mag, e = ref.attend(q[at:at + x].cpu().double(), keys, kb, live, (d + dr) ** -0.5)
        for got, what in ((out, "expanded"), (other, "absorbed")):
            ref.is_close(got[at:at + x], o, ref.tolerance(o, mag, e, lens[b], ref.BF16), f"{what}, request {b}")
        at += x


def test_two_threads():
    """Calls of two threads, each on a stream of its own, give the bits of the same calls alone."""
    jobs = []
    for i, (lens, new) in enumerate((([2600, 900, 3000], [12, 3, 20]), ([1500, 4000, 10], [2, 30, 1]))):
        gen, kp, vp, table, _ = build(lens, new, 2, 128, 16, seed=i)
        _, pages, _, lat_table, _ = build(lens, new, 1, 512, 16, seed=i, latent=576)
        T = sum(new)
        q, qa = torch.randn((T, 8, 128), generator=gen).bfloat16().cuda(), torch.randn((T, 16, 576), generator=gen).bfloat16().cuda()
        args = [x.cuda() for x in (kp, vp, table, pages, lat_table)]
        ln, cu = _i32(lens), _i32(np.cumsum([0] + new).tolist())

        def run(q=q, qa=qa, args=args, ln=ln, cu=cu, most=max(new)):
            a, b = torch.empty_like(q), torch.empty((q.shape[0], 16, 512), dtype=torch.bfloat16, device="cuda")
            lib.kv_tree_attention(q, args[0], args[1], args[2], ln, cu, a, max_new=most)
            lib.kv_latent_attention(qa, args[3], args[4], ln, b, 0.05, cu_new=cu, max_new=most)
            return a, b
        jobs.append(run)
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        try:
            for _ in range(20):
                with torch.cuda.stream(stream):
                    got = jobs[i]()
                stream.synchronize()
                if not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                    bad.append(f"thread {i}: other bits")
                    return
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


@pytest.mark.parametrize("page", [64, 8])
@pytest.mark.parametrize("most,Hq", [(1, 8), (5, 8), (20, 32)])
def test_caches_past_32_bits(page, most, Hq):
    """The same pages at the front and at the end of a cache of more than 2^32 bytes: the same bits."""
    lens, new = [777, 64, 1200], [most, 1, most]
    gen, kp, vp, table, _ = build(lens, new, 4, 128, page)
    T, n = sum(new), kp.shape[0]
    q = torch.randn((T, Hq, 128), generator=gen).bfloat16().cuda()
    args = [_i32(lens), _i32(np.cumsum([0] + new).tolist())]
    pages = 2 ** 32 // (4 * page * 128 * 2) + 3 * n
    far, fv = (torch.zeros((pages, 4, page, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for x, y in ((far, kp), (fv, vp)):
        x[:n], x[pages - n:] = y.cuda(), y.cuda()
    shifted = torch.where(table >= 0, table + pages - n, table)
    outs = [torch.zeros_like(q) for _ in range(2)]
    for out, t in zip(outs, (table, shifted)):
        lib.kv_tree_attention(q, far, fv, t.cuda(), *args, out, max_new=most)
    assert bool(outs[0].any()) and torch.equal(*outs)


@pytest.mark.parametrize("page", [64, 8])
@pytest.mark.parametrize("most,H", [(1, 16), (1, 30), (2, 128)])
def test_latent_caches_past_32_bits(page, most, H):
    lens, new = [777, 64, 1200], [most, 1, most]
    gen, kp, _, table, _ = build(lens, new, 1, 512, page, latent=576)
    T, n = sum(new), kp.shape[0]
    q = torch.randn((T, H, 576), generator=gen).bfloat16().cuda()
    pages = 2 ** 32 // (page * 576 * 2) + 3 * n
    far = torch.zeros((pages, page, 576), dtype=torch.bfloat16, device="cuda")
    far[:n], far[pages - n:] = kp.cuda(), kp.cuda()
    shifted = torch.where(table >= 0, table + pages - n, table)
    outs = [torch.zeros((T, H, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for out, t in zip(outs, (table, shifted)):
        lib.kv_latent_attention(q, far, t.cuda(), _i32(lens), out, 0.05, cu_new=_i32(np.cumsum([0] + new).tolist()), max_new=most)
    assert bool(outs[0].any()) and torch.equal(*outs)
    slots = torch.tensor([pages * page - 1, 0, pages * page], device="cuda")
    c, kr = torch.randn((3, 512), generator=gen).bfloat16().cuda(), torch.randn((3, 64), generator=gen).bfloat16().cuda()
    lib.kv_latent_append(c, kr, slots, far)
    assert torch.equal(far[-1, -1], torch.cat([c[0], kr[0]])) and torch.equal(far[0, 0], torch.cat([c[1], kr[1]]))


def _at(t, off):
    """t in memory that begins `off` bytes behind a multiple of 256."""
    raw = torch.empty(t.numel() * t.element_size() + 512, dtype=torch.uint8, device="cuda")
    start = -raw.data_ptr() % 256 + off
    return raw[start:start + t.numel() * t.element_size()].view(t.dtype).view(t.shape).copy_(t)


def test_least_alignment():
    """Arrays at the least alignment that is asked for give the bits of well aligned ones."""
    for most, Hq in ((2, 8), (12, 16)):
        lens, new = [300, 40], [most, 1]
        gen, kp, vp, table, _ = build(lens, new, 2, 64, 8)
        q = torch.randn((most + 1, Hq, 64), generator=gen).bfloat16()
        mask = torch.randint(-2 ** 62, 2 ** 62, (most + 1, 1), generator=gen)
        outs = []
        for big, word, small in ((0, 0, 0), (16, 8, 4)):
            out = _at(torch.zeros_like(q), big)
            lib.kv_tree_attention(_at(q, big), _at(kp, big), _at(vp, big), _at(table, small), _at(_i32(lens), small), _at(_i32([0, most, most + 1]), small), out,
                                  mask=_at(mask, word), max_new=most)
            outs.append(out)
        assert torch.equal(*outs)
    for H in (4, 40):
        gen, pages, _, table, _ = build([300, 40], [1, 1], 1, 256, 8, latent=288)
        q = torch.randn((2, H, 288), generator=gen).bfloat16()
        outs = []
        for big, small in ((0, 0), (16, 4)):
            out = _at(torch.zeros((2, H, 256), dtype=torch.bfloat16), big)
            lib.kv_latent_attention(_at(q, big), _at(pages, big), _at(table, small), _at(_i32([300, 40]), small), out, 0.1)
            outs.append(out)
        assert torch.equal(*outs)
    gen = torch.Generator().manual_seed(1)
    q, k, v, kr = (torch.randn(x, generator=gen).bfloat16() for x in ((90, 3, 96), (90, 3, 64), (90, 3, 64), (90, 32)))
    outs = []
    for big, small in ((0, 0), (16, 4)):
        out = _at(torch.zeros_like(v), big)
        lib.kv_latent_prompt_attention(_at(q, big), _at(k, big), _at(kr, big), _at(v, big), _at(_i32([0, 70, 90]), small), out)
        outs.append(out)
    assert torch.equal(*outs)


def _rising(n, step):
    """Keys along one direction, so that the scores rise by step n times (in units of the exponent)."""
    return (torch.arange(n) * step / 8).bfloat16()


@pytest.mark.parametrize("step", [0.02, 0.5, 3.0, -0.5])
@pytest.mark.parametrize("most,Hq", [(1, 4), (5, 8), (9, 16), (20, 32)])
def test_scores_that_rise(step, most, Hq):
    """Each token scores higher than those before it: the running maximum moves in every tile (or never)."""
    n = 700
    gen, kp, vp, table, keys = build([n], [most], 2, 64, 16)
    k, v = keys[0]
    k[:] = 0
    k[:, :, 5] = _rising(n, step)[:, None]
    pos = torch.arange(n)
    kp[table[0, pos // 16].long(), :, pos % 16] = k
    q = torch.zeros((most, Hq, 64), dtype=torch.bfloat16)
    q[..., 5] = 8.0
    out = torch.zeros((most, Hq, 64), dtype=torch.bfloat16, device="cuda")
    lib.kv_tree_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32([n]), _i32([0, most]), out, scale=1.0)
    o, mag, e = ref.attend(q.double(), k.double(), v.double(), ref.seen(most, n), 1.0)
    ref.is_close(out, o, ref.tolerance(o, mag, e, n, weight(most * Hq // 2)), f"{most} x {Hq}, {step}")


@pytest.mark.parametrize("step", [0.02, 0.5, 3.0, -0.5])
@pytest.mark.parametrize("dc,most,H", [(512, 1, 4), (512, 1, 30), (256, 3, 17), (512, 2, 128), (256, 1, 100)])
def test_latent_scores_that_rise(step, dc, most, H):
    n, W = 700, dc + dc // 8
    gen, pages, _, table, keys = build([n], [most], 1, dc, 16, latent=W)
    k = keys[0]
    k[:, dc:] = 0
    k[:, dc + 3] = _rising(n, step)
    pos = torch.arange(n)
    pages[table[0, pos // 16].long(), pos % 16] = k
    q = torch.zeros((most, H, W), dtype=torch.bfloat16)
    q[..., dc + 3] = 8.0
    q[:, H // 2:, dc + 3] = -1.0                       # (in the same tile some rows' scores fall)
    out = torch.zeros((most, H, dc), dtype=torch.bfloat16, device="cuda")
    lib.kv_latent_attention(q.cuda(), pages.cuda(), table.cuda(), _i32([n]), out, 1.0, cu_new=_i32([0, most]))
    kd = k.double()[:, None]
    o, mag, e = ref.attend(q.double(), kd, kd[..., :dc], ref.seen(most, n), 1.0)
    ref.is_close(out, o, ref.tolerance(o, mag, e, n, ref.BF16), f"{most} x {H}, {step}")


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(scale):
    for most, Hq in ((2, 4), (20, 8)):
        gen, kp, vp, table, keys = build([150], [most], 1, 64, 16)
        q = torch.randn((most, Hq, 64), generator=gen).bfloat16()
        out = torch.zeros_like(q, device="cuda")
        lib.kv_tree_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32([150]), _i32([0, most]), out, scale=scale)
        o, mag, e = ref.attend(q.double(), *(x.double() for x in keys[0]), ref.seen(most, 150), scale)
        ref.is_close(out, o, ref.tolerance(o, mag, e, 150, weight(most * Hq)), f"{most}, {scale}")
    for H in (4, 40):
        gen, pages, _, table, keys = build([150], [2], 1, 256, 16, latent=288)
        q = torch.randn((2, H, 288), generator=gen).bfloat16()
        out = torch.zeros((2, H, 256), dtype=torch.bfloat16, device="cuda")
        lib.kv_latent_attention(q.cuda(), pages.cuda(), table.cuda(), _i32([150]), out, scale, cu_new=_i32([0, 2]))
        k = keys[0].double()[:, None]
        o, mag, e = ref.attend(q.double(), k, k[..., :256], ref.seen(2, 150), scale)
        ref.is_close(out, o, ref.tolerance(o, mag, e, 150, ref.BF16), f"latents, {H}, {scale}")


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_not_finite_beside_a_page_that_does_not_exist(value):
    """Before the drafted tokens, in the tile of a missing page: every row has the value's."""
    n, bad, at = 300, 3, 40
    for most, Hq in ((2, 4), (20, 8)):
        gen, kp, vp, table, keys = build([n], [most], 1, 64, 16)
        vp[int(table[0, at // 16]), 0, at % 16, 7] = value
        table[0, bad] = -1
        q = torch.randn((most, Hq, 64), generator=gen).bfloat16()
        out = torch.zeros_like(q, device="cuda")
        lib.kv_tree_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32([n]), _i32([0, most]), out)
        assert torch.equal(torch.isfinite(out).all(0).all(0).cpu(), torch.arange(64) != 7)
        got = out[..., 7].float()
        assert bool((torch.isnan(got) if value != value else got == value).all())
    for H in (4, 40, 128):
        gen, pages, _, table, keys = build([n], [1], 1, 256, 16, latent=288)
        pages[int(table[0, at // 16]), at % 16, 7] = value
        table[0, bad] = -1
        q = torch.randn((1, H, 288), generator=gen).bfloat16()
        q[..., 7] = 0.0 if value != value else q[..., 7]
        out = torch.zeros((1, H, 256), dtype=torch.bfloat16, device="cuda")
        lib.kv_latent_attention(q.cuda(), pages.cuda(), table.cuda(), _i32([n]), out, 0.1)
        assert not bool(torch.isfinite(out[..., 7]).any())


def test_one_page_twice_and_one_for_all():
    """A table may name a page twice, and requests may read the same pages."""
    gen, kp, vp, table, keys = build([64], [3], 2, 64, 16)
    t = table[:, :4].repeat(2, 1)
    t[1, 2] = t[1, 0]
    k = [keys[0][0], keys[0][0].clone()]
    v = [keys[0][1], keys[0][1].clone()]
    k[1][32:48], v[1][32:48] = k[0][:16], v[0][:16]
    q = torch.randn((6, 4, 64), generator=gen).bfloat16()
    out = torch.zeros_like(q, device="cuda")
    lib.kv_tree_attention(q.cuda(), kp.cuda(), vp.cuda(), t.contiguous().cuda(), _i32([64, 64]), _i32([0, 3, 6]), out, max_new=3)
    for b in range(2):
        o, mag, e = ref.attend(q[3 * b:3 * b + 3].double(), k[b].double(), v[b].double(), ref.seen(3, 64), 0.125)
        ref.is_close(out[3 * b:3 * b + 3], o, ref.tolerance(o, mag, e, 64, weight(12)), f"request {b}")


def _ragged(B, long, at, most, seed):
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(0, 180, B)]
    lens[at % B] = long
    return lens, [int(min(x, y)) for x, y in zip(lens, rng.integers(0, most + 1, B))]


@pytest.mark.parametrize("at", [0, 77, -1])
@pytest.mark.parametrize("B,long,most,Hq,Hkv", [(64, 3001, 2, 4, 2), (65, 2000, 20, 8, 1), (300, 4000, 3, 2, 1), (130, 3500, 40, 4, 1), (512, 2500, 2, 4, 4), (520, 1500, 2, 4, 4)])
def test_one_long_request_among_many(at, B, long, most, Hq, Hkv):
    """Few units and many, one row tile and several, more requests than are cut: every run is taken once."""
    lens, new = _ragged(B, long, at, most, B + most)
    _attend(lens, new, Hq, Hkv, 64, 16, "tree" if most <= 3 else None, max_new=most)


@pytest.mark.parametrize("at", [0, -1])
@pytest.mark.parametrize("B,long,most,H", [(40, 3000, 2, 4), (150, 2500, 3, 40), (300, 2000, 1, 16), (257, 2000, 1, 33)])
def test_one_long_latent_request_among_many(at, B, long, most, H):
    lens, new = _ragged(B, long, at, most, B + H)
    _absorbed(lens, new, H, 256, 16, None)


def test_more_row_tiles_than_are_dealt_at_a_time():
    _attend([2600, 40], [290, 7], 8, 1, 64, 16, None)              # 37 tiles of 64 rows, 19 of 128
    _attend([1300] * 3, [150, 3, 150], 16, 1, 64, 16, None)
    _absorbed([1500, 30], [20, 3], 64, 256, 16, None)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_key_that_is_not_finite_in_one_run(value):
    """A cached key in one of many runs: the formula's NaN in every row, or a weight of 0, as binary64 has it."""
    for most, Hq in ((1, 8), (6, 8), (20, 8)):
        gen, kp, vp, table, keys = build([4000], [most], 1, 64, 16)
        for t in (0, 1990, 2500):
            kp[int(table[0, t // 16]), 0, t % 16, 3] = value
            keys[0][0][t, 0, 3] = value
        q = torch.randn((most, Hq, 64), generator=gen).bfloat16()
        q[..., 3] = q[..., 3].abs() + 1.0
        out = torch.zeros_like(q, device="cuda")
        lib.kv_tree_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32([4000]), _i32([0, most]), out)
        if value == float("-inf"):
            live = ref.seen(most, 4000)
            live[:, [0, 1990, 2500]] = False
            k = torch.nan_to_num(keys[0][0].double(), neginf=0.0)
            o, mag, e = ref.attend(q.double(), k, keys[0][1].double(), live, 0.125)
            ref.is_close(out, o, ref.tolerance(o, mag, e, 4000, weight(most * Hq)), f"{most}")
        else:
            assert bool(torch.isnan(out).all())
    for H in (4, 40):
        gen, pages, _, table, _ = build([3000], [1], 1, 256, 16, latent=288)
        for t in range(1984, 2048):
            pages[int(table[0, t // 16]), t % 16, 260] = float("nan")
        out = torch.zeros((1, H, 256), dtype=torch.bfloat16, device="cuda")
        lib.kv_latent_attention(torch.randn((1, H, 288), generator=gen).bfloat16().cuda(), pages.cuda(), table.cuda(), _i32([3000]), out, 0.1)
        assert bool(torch.isnan(out).all())
