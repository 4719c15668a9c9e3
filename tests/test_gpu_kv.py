"""Block tables, the store of keys and values, and attention of one new token over a paged cache
(kv_build_tables, kv_append, kv_decode_attention) against list and binary64 references.

Bounds of the attention: each softmax weight is off by its score's binary32 error (serving_ref.
score_error, relative) and by its rounding to bf16 (2^-8 relative); sums over the tokens add 2^-24
per tile and join. All are relative to sum p |v| (doubled where the normaliser carries the same
error), and the result's own rounding to bf16 is 2^-8 of it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import serving_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib  # noqa: E402


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- tables ------------------------------------------------------------------------------------
def _tables(seq, new, free, table, page, T, positions=True):
    B, blocks = len(seq), len(table[0]) if table else 4
    tab = _i32(table).reshape(B, blocks)
    slots = torch.full((T,), 12345, dtype=torch.int64, device="cuda")
    pos = _i32([12345] * T) if positions else None
    cu, used = _i32([12345] * (B + 1)), _i32([12345])
    lib.kv_build_tables(_i32(seq), _i32(new), _i32(free), tab, page, slots, pos, cu, used)
    torch.cuda.synchronize()
    want = ref.tables(seq, new, free, table, page, T, blocks)
    assert tab.tolist() == want[0] and slots.tolist() == want[1] and cu.tolist() == want[3] and used.tolist() == [want[4]]
    if positions:
        assert pos.tolist() == want[2]


@pytest.mark.parametrize("B", [1, 2, 63, 64, 65, 511, 512, 513, 1500])
@pytest.mark.parametrize("page", [1, 16, 128])
def test_tables_random(B, page):
    rng = np.random.default_rng([B, page])
    old = rng.integers(0, 6 * page + 1, B) * (rng.random(B) < 0.7)
    new = rng.integers(0, 4 * page + 2, B) * (rng.random(B) < 0.8)
    blocks = 12
    ids = rng.permutation(B * blocks + 50)
    table = [[int(ids[b * blocks + i]) if i < -(-old[b] // page) else -7 for i in range(blocks)] for b in range(B)]
    free = [int(x) for x in rng.permutation(10 ** 6)[: B * blocks]]
    _tables([int(x) for x in old + new], [int(x) for x in new], free, table, page, int(new.sum()) + 5)


def test_tables_edges():
    t = [[3, -1, -1], [5, 6, -1], [-1, -1, -1]]
    _tables([17, 40, 0], [1, 8, 0], [9, 8, 7], t, 16, 9)
    _tables([17, 40, 0], [1, 8, 0], [9, 8, 7], t, 16, 4)               # a slot map shorter than the tokens
    _tables([17, 40, 0], [1, 8, 0], [9], t, 16, 12, positions=False)    # one page too few
    _tables([17, 40, 30], [1, 8, 30], [], t, 16, 50)                    # no free page
    _tables([100, 40, 5], [90, 60, -4], [1, 2, 3, 4, 5, 6], t, 16, 140)  # longer than the table; more new than there are; negative
    _tables([2 ** 20 + 3], [3], [11], [[1, 2]], 32768, 3)               # beyond the table altogether
    _tables([-5, 7], [3, 7], [11], [[1, 2], [-1, -1]], 8, 8)
    _tables([], [], [], [], 16, 3)
    _tables([5], [5], [2 ** 31 - 1], [[-1]], 8, 5)                       # slots past 32 bits


def test_tables_refusals():
    z = _i32([0])
    args = [z, z, z, z.reshape(1, 1), 16, torch.zeros(4, dtype=torch.int64, device="cuda"), _i32([0] * 4), _i32([0, 0]), z.clone()]
    lib.kv_build_tables(*args)
    for i, bad in ((1, _i32([0, 0])), (3, z), (5, torch.zeros(4, dtype=torch.int32, device="cuda")), (6, _i32([0])), (7, z), (8, _i32([0, 0]))):
        with pytest.raises((ValueError, TypeError)):
            lib.kv_build_tables(*args[:i], bad, *args[i + 1:])
    for page in (0, 24, -16, 65536):
        with pytest.raises(lib.DampError) as e:
            lib.kv_build_tables(*args[:4], page, *args[5:])
        assert e.value.status == lib.DAMP_ERR_UNSUPPORTED
    n = 8001
    with pytest.raises(lib.DampError) as e:
        lib.kv_build_tables(_i32([0] * n), _i32([0] * n), z, _i32([0] * n).reshape(n, 1), 16, args[5], None, _i32([0] * (n + 1)), args[8])
    assert e.value.status == lib.DAMP_ERR_UNSUPPORTED
    _tables([1] * 8000, [1] * 8000, list(range(8000)), [[-1]] * 8000, 16, 8000)


@pytest.mark.parametrize("d,H,page", [(64, 1, 16), (128, 3, 1), (128, 8, 32)])
def test_append(d, H, page):
    gen = torch.Generator(device="cuda").manual_seed(d)
    pages, T = 7, 41
    n = pages * page
    kp, vp = (torch.randn((pages, H, page, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn((T, H, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    slots = torch.full((T,), -1, dtype=torch.int64)
    perm = torch.randperm(T)[: min(T - 3, n)]
    slots[perm] = torch.randperm(n)[: perm.numel()]
    bad = [t for t in range(T) if t not in perm.tolist()]
    slots[bad[0]], slots[bad[1]] = n, 2 ** 40
    wk, wv = kp.clone(), vp.clone()
    for t in range(T):
        s = int(slots[t])
        if 0 <= s < n:
            wk[s // page, :, s % page], wv[s // page, :, s % page] = k[t], v[t]
    lib.kv_append(k, v, slots.cuda(), kp, vp)
    torch.cuda.synchronize()
    assert torch.equal(kp, wk) and torch.equal(vp, wv)
    lib.kv_append(k[:0], v[:0], slots[:0].cuda(), kp, vp)
    assert torch.equal(kp, wk)


# ---- attention ---------------------------------------------------------------------------------
def _attend(lens, Hq, Hkv, d, page, new=True, scale=None, max_len=None, seed=0, blocks=None, big=1.0, bad=(), poison=True, extra_len=0):
    gen = torch.Generator().manual_seed(seed + 11 * sum(lens) + d)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    blocks = blocks or max(need + [1]) + 1
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=gen).tolist()
    # whatever lies outside the requests' tokens must not matter
    fill = float("nan") if poison else 0.0
    kp, vp = (torch.full((pages, Hkv, page, d), fill, dtype=torch.bfloat16) for _ in range(2))
    table = torch.full((B, blocks), -1, dtype=torch.int32)
    k_new, v_new = ((torch.randn((B, Hkv, d), generator=gen)).bfloat16() for _ in range(2))
    q = (big * torch.randn((B, Hq, d), generator=gen)).bfloat16()
    keys, at = [], 0
    for b, n in enumerate(lens):
        for i in range(need[b]):
            table[b, i] = ids[at]
            at += 1
        k, v = (torch.randn((n, Hkv, d), generator=gen).bfloat16() for _ in range(2))
        if new and n:
            k[n - 1], v[n - 1] = k_new[b], v_new[b]
        for p in range(n):
            if not (new and p == n - 1):
                kp[table[b, p // page], :, p % page], vp[table[b, p // page], :, p % page] = k[p], v[p]
        keys.append((k, v))
    wk, wv = kp.clone(), vp.clone()
    for b, n in enumerate(lens):
        if new and n and (b, (n - 1) // page) not in bad:
            wk[table[b, (n - 1) // page], :, (n - 1) % page] = k_new[b]
            wv[table[b, (n - 1) // page], :, (n - 1) % page] = v_new[b]
    for b, i in bad:
        table[b, i] = pages + 4 if i % 2 else -2
    kd, vd, out = kp.cuda(), vp.cuda(), torch.full((B, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.kv_decode_attention(q.cuda(), kd, vd, table.cuda(), _i32([n + extra_len for n in lens]), out, scale=scale,
                            k_new=k_new.cuda() if new else None, v_new=v_new.cuda() if new else None, max_len=max_len)
    torch.cuda.synchronize()
    assert torch.equal(kd.cpu().view(torch.int16), wk.view(torch.int16)) and torch.equal(vd.cpu().view(torch.int16), wv.view(torch.int16))
    s = d ** -0.5 if scale is None else scale
    used = 0.0
    for b, n in enumerate(lens):
        live = torch.tensor([(b, p // page) not in bad for p in range(n)], dtype=torch.bool)
        k, v = (x[live].double() for x in keys[b])
        o, mag = ref.attention(q[b].double(), k, v, s)
        e = ref.score_error(q[b].double(), k, s) + 2.0 ** -8 + (len(lens) and (n // 32 + 64)) * ref.EPS32
        used = max(used, ref.is_close(out[b], o, 2.0 ** -8 * o.abs() + 2 * e * mag + 1e-37, f"request {b} of {n} tokens"))
    return used


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 8, 16, 64, 256])
@pytest.mark.parametrize("new", [True, False])
def test_attention_lengths(d, page, new):
    _attend([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300], 4, 2, d, page, new=new)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (3, 1), (7, 1), (16, 1), (17, 1), (40, 1), (64, 2), (32, 8), (10, 5)])
def test_attention_heads(d, Hq, Hkv):
    _attend([129, 5, 260], Hq, Hkv, d, 16)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_long_and_split(d):
    _attend([5000, 1, 0, 2049, 1025], 4, 1, d, 16)
    _attend([3001], 8, 2, d, 32, max_len=3001)
    _attend([100, 3], 2, 1, d, 16, blocks=4000)                 # a table far wider than the requests


def test_attention_many_requests():
    rng = np.random.default_rng(3)
    _attend([int(x) for x in rng.integers(0, 400, 300)], 2, 1, 64, 16)


@pytest.mark.parametrize("B", [40, 64, 65, 300])
def test_attention_many_requests_in_a_wide_table(B):
    """Many requests of which some are cut (the table allows for more than any holds)."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 60, B)]
    lens[0], lens[B // 2], lens[-1] = 2500, 700, 3100
    _attend(lens, 4, 2, 64, 16, blocks=200)


@pytest.mark.parametrize("Hq,Hkv", [(40, 1), (17, 1), (64, 2)])
def test_attention_many_heads_cut(Hq, Hkv):
    _attend([3000, 5, 1100], Hq, Hkv, 128, 16)


@pytest.mark.parametrize("longest", [1023, 1024, 1025, 2048, 2049])
def test_attention_around_the_lengths_that_are_cut(longest):
    _attend([longest, 1, 300], 4, 1, 64, 1)
    _attend([longest] + [3] * 128, 4, 4, 64, 1)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_scales_and_sharp_scores(d):
    _attend([200, 33], 4, 2, d, 16, scale=0.0)
    _attend([200, 33], 4, 2, d, 16, scale=-0.1)
    _attend([700, 33], 4, 2, d, 16, scale=1.0, big=8.0)          # one token takes nearly all the weight


@pytest.mark.parametrize("new", [True, False])
def test_attention_pages_that_do_not_exist_are_left_out(new):
    _attend([100, 40, 16], 4, 2, 64, 16, new=new, bad=((0, 0), (0, 3), (1, 2), (2, 0)))
    _attend([1000, 40], 2, 2, 128, 16, new=new, bad=tuple((0, i) for i in range(8)) + tuple((0, i) for i in range(32, 63)))


def test_attention_lengths_past_the_table_or_the_bound():
    """Tokens past max_len or past the table's width are left out, and nothing is stored there."""
    gen = torch.Generator().manual_seed(5)
    kp, vp = (torch.randn((4, 1, 16, 64), generator=gen).bfloat16() for _ in range(2))
    q, kn = torch.randn((2, 2, 64), generator=gen).bfloat16(), torch.randn((2, 1, 64), generator=gen).bfloat16()
    table = torch.tensor([[0, 1], [3, 2]], dtype=torch.int32)
    for lens, max_len, n in (([70, 2 ** 31 - 1], None, (32, 32)), ([30, 25], 20, (20, 20)), ([-4, 9], 20, (0, 9))):
        kd, vd, out = kp.cuda(), vp.cuda(), torch.empty((2, 2, 64), dtype=torch.bfloat16, device="cuda")
        lib.kv_decode_attention(q.cuda(), kd, vd, table.cuda(), _i32(lens), out, max_len=max_len, k_new=kn.cuda() if n[1] != 9 else None,
                                v_new=kn.cuda() if n[1] != 9 else None)
        torch.cuda.synchronize()
        assert torch.equal(kd.cpu(), kp) and torch.equal(vd.cpu(), vp)
        for b in range(2):
            k, v = (torch.cat([x[i] for i in table[b].tolist()], 1).transpose(0, 1)[: n[b]].double() for x in (kp, vp))
            o, mag = ref.attention(q[b].double(), k, v, 0.125)
            ref.is_close(out[b], o, 2.0 ** -8 * o.abs() + 2 * (2.0 ** -8 + ref.score_error(q[b].double(), k, 0.125) + 70 * ref.EPS32) * mag, f"{lens} {b}")


def test_attention_of_infinities_and_nan_in_the_tokens():
    """A NaN key makes its request's readout NaN and no other's; a -inf score has no weight."""
    kp = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    vp = torch.ones_like(kp)
    vp[1, 0, 3] = 5.0
    kp[0, 0, 2] = float("nan")
    kp[1, 0, 3, 0] = -float("inf")
    q = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    out = torch.empty_like(q)
    lib.kv_decode_attention(q, kp, vp, _i32([[0], [1]]), _i32([9, 9]), out)
    torch.cuda.synchronize()
    assert bool(out[0].isnan().all()) and bool((out[1] == 1.0).all())


def test_attention_cache_past_32_bits():
    """Pages beyond 2^32 bytes, and beyond 2^31 elements, of the cache."""
    d, page, Hkv = 128, 64, 4
    pages = 2 ** 31 // (d * page * Hkv) + 9                      # 2^31 values and more: 4.3 GB of keys
    kp, vp = (torch.zeros((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = [pages - 1, 0, pages - 2]
    for i in ids:
        kp[i].normal_(generator=gen)
        vp[i].normal_(generator=gen)
    q, kn, vn = (torch.randn((1, h, d), generator=gen, device="cuda").bfloat16() for h in (8, Hkv, Hkv))
    n = 3 * page
    k, v = (torch.cat([x[i] for i in ids], 1).transpose(0, 1).cpu().double() for x in (kp, vp))
    k[n - 1], v[n - 1] = kn[0].cpu().double(), vn[0].cpu().double()
    out = torch.empty_like(q)
    lib.kv_decode_attention(q, kp, vp, _i32([ids]), _i32([n]), out, k_new=kn, v_new=vn)
    torch.cuda.synchronize()
    o, mag = ref.attention(q[0].cpu().double(), k, v, d ** -0.5)
    ref.is_close(out[0], o, 2.0 ** -8 * o.abs() + 2 * (2.0 ** -8 + ref.score_error(q[0].cpu().double(), k, d ** -0.5) + 70 * ref.EPS32) * mag, "far pages")
    assert torch.equal(kp[pages - 2, :, page - 1], kn[0])
    slots = torch.tensor([pages * page - 1], dtype=torch.int64, device="cuda")
    lib.kv_append(kn, vn, slots, kp, vp)
    assert torch.equal(kp[pages - 1, :, page - 1], kn[0]) and torch.equal(vp[pages - 1, :, page - 1], vn[0])


def test_attention_refusals():
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    kp = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    t, n, out, new = _i32([[0], [1]]), _i32([1, 1]), torch.empty_like(q), torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    lib.kv_decode_attention(q, kp, kp.clone(), t, n, out, k_new=new, v_new=new)
    bad = [dict(q=q.float()), dict(q=q[:1]), dict(v_pages=kp[:2]), dict(v_pages=kp.float()), dict(block_table=t[0]), dict(block_table=t.long()),
           dict(seq_lens=n[:1]), dict(out=out.float()), dict(k_new=new), dict(k_new=new[:1], v_new=new), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)),
           dict(k_pages=kp[..., :32])]
    for x in bad:
        with pytest.raises((ValueError, TypeError)):
            lib.kv_decode_attention(**{**dict(q=q, k_pages=kp, v_pages=kp, block_table=t, seq_lens=n, out=out), **x})
    q3 = torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lib.DampError) as e:
        lib.kv_decode_attention(q3, kp, kp, t, n, torch.empty_like(q3))      # 3 query heads on 2
    assert e.value.status == lib.DAMP_ERR_INVALID_ARGUMENT
    for shape in ((3, 2, 16, 32), (3, 2, 24, 64)):
        p = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        qq = torch.zeros((2, 4, shape[3]), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(lib.DampError) as e:
            lib.kv_decode_attention(qq, p, p, t, n, torch.empty_like(qq))
        assert e.value.status == lib.DAMP_ERR_UNSUPPORTED
    with pytest.raises(lib.DampError) as e:
        lib.kv_decode_attention(q, kp, kp, t, n, out, max_len=-1)
    assert e.value.status == lib.DAMP_ERR_INVALID_ARGUMENT
    none = q[:0]
    lib.kv_decode_attention(none, kp, kp, t[:0], n[:0], none.clone())


def test_attention_in_a_graph_and_on_two_streams():
    gen = torch.Generator(device="cuda").manual_seed(4)
    B, Hq, Hkv, d, page = 6, 8, 2, 128, 16
    lens = [1, 700, 33, 1500, 0, 640]
    # every page in one place only: the page of a new token is its request's alone
    kp, vp = (torch.randn((B * 100, Hkv, page, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(B * 100, generator=gen, device="cuda").reshape(B, 100).to(torch.int32)
    n = _i32(lens)
    q, kn, vn = (torch.randn((B, h, d), generator=gen, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    oe, og = torch.empty_like(q), torch.empty_like(q)
    lib.kv_decode_attention(q, kp, vp, table, n, oe, k_new=kn, v_new=vn)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.kv_decode_attention(q, kp, vp, table, n, og, k_new=kn, v_new=vn)
    noise = torch.zeros(1 << 20, device="cuda")
    for i in range(4):
        q.copy_(torch.randn((B, Hq, d), generator=gen, device="cuda"))
        n.copy_(_i32([(x + 7 * i) % 1600 for x in lens]))
        lib.kv_decode_attention(q, kp, vp, table, n, oe, k_new=kn, v_new=vn)
        g.replay()
        noise.add_(1.0)
        torch.cuda.synchronize()
        assert torch.equal(oe, og), f"replay {i}"
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(q) for _ in range(2)]
    for _ in range(5):
        for s, o in zip(streams, outs):
            lib.kv_decode_attention(q, kp, vp, table, n, o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], oe) and torch.equal(outs[1], oe)


def test_tables_in_a_graph():
    B, page, T = 40, 16, 60
    seq, new = _i32([33] * B), _i32([1] * B)
    free, table = _i32(list(range(500, 700))), _i32(list(range(B * 6))).reshape(B, 6)
    bufs = [[table.clone(), torch.empty(T, dtype=torch.int64, device="cuda"), _i32([0] * T), _i32([0] * (B + 1)), _i32([0])] for _ in range(3)]

    def call(x):
        lib.kv_build_tables(seq, new, free, x[0], page, *x[1:])

    call(bufs[2])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(bufs[1])
    for i in range(4):
        seq.add_(5 + i)
        new.copy_(_i32([(b + i) % 3 for b in range(B)]))
        call(bufs[0])
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(*bufs[:2]):
            assert torch.equal(x, y), f"replay {i}"
