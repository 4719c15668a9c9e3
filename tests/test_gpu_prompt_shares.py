"""Delta-rule calls of no more tokens than requests: requests of up to 32 tokens run token by token and
longer ones in chunks of 64, within one call.

Bounds as derived for the prompt forms: a state's column is off by (2 d + 156) roundings of its largest norm
per chunk (magnified by the chunk's condition number) or per token, a bf16 readout by 2^-8 of itself and
2^-15 of the norm more where the weights come in two pieces."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import serving_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib  # noqa: E402


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _inputs(seed, T, H, d):
    gen = torch.Generator().manual_seed(seed)
    q, k = (_unit(torch.randn((T, H, d), generator=gen)).bfloat16() for _ in range(2))
    v = torch.randn((T, H, d), generator=gen).bfloat16()
    life = torch.exp2(torch.linspace(1.0, 11.0, H)) if H > 1 else torch.tensor([20.0])
    return q, k, v, torch.exp2(-(0.2 + torch.rand((T, H), generator=gen)) / life), torch.sigmoid(torch.randn((T, H), generator=gen))


def _check(lens, H, d, resume=None, slots=None, num_slots=None, tail=0, seed=0):
    B, T = len(lens), sum(lens)
    assert T + tail <= B
    q, k, v, a, b = _inputs(seed, T + tail, H, d)
    gen = torch.Generator().manual_seed(seed + 5)
    num_slots = num_slots or B + 2
    slots = torch.randperm(num_slots, generator=gen)[:B].to(torch.int32) if slots is None else torch.tensor(slots, dtype=torch.int32)
    pool = torch.randn((num_slots, H, d, d), generator=gen)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    got, out = pool.cuda(), torch.full((T + tail, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.fp32_delta_prefill(got, slots.cuda(), cu.cuda(), q.cuda(), k.cuda(), v.cuda(), a.cuda(), b.cuda(), out,
                           resume=None if resume is None else torch.tensor(resume, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    got, out = got.cpu(), out.cpu()
    assert bool((out[T:] == 7.0).all()), "rows behind the last request were written"
    touched = set()
    for i, n in enumerate(lens):
        s, r = int(slots[i]), slice(int(cu[i]), int(cu[i + 1]))
        if not 0 <= s < num_slots or n == 0:
            assert bool((out[r] == 7.0).all())
            continue
        touched.add(s)
        for h in range(H):
            S = pool[s, h].double() if resume is not None and resume[i] else torch.zeros((d, d), dtype=torch.float64)
            x = [y[r, h].double() for y in (q, k, v)]
            o, X, _, _, top = ref.prompt(S, *x, a[r, h].double(), b[r, h].double())
            chain, kappa = (n, 1.0) if n <= 32 else (-(-n // 64), ref.chunk_condition(x[1], a[r, h].double(), b[r, h].double()))
            e_col = (2 * d + 156) * chain * kappa * ref.EPS32 * top
            assert bool(((got[s, h].double() - X).norm(dim=0) <= e_col).all()), f"state of request {i} ({n} tokens), head {h}"
            ref.is_close(out[r, h], o, 2.0 ** -8 * o.abs() + x[0].norm(dim=-1, keepdim=True) * (e_col + 2.0 ** -15 * kappa * top), f"request {i} ({n} tokens), head {h}")
    rest = [s for s in range(num_slots) if s not in touched]
    assert torch.equal(got[rest], pool[rest]), "a slot without new tokens was written"


def _fill(lens, B):
    """Requests of no tokens spread between the given ones."""
    out = [0] * B
    for i, n in enumerate(lens):
        out[i * B // len(lens)] = n
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[65], [90], [33, 33, 33], [32, 33, 1], [31, 65, 1, 33], [1] * 70, [64, 1, 64, 2, 65], [1, 97, 32, 129], [128, 127, 1, 1],
                                  [1] * 31 + [33] + [1] * 30 + [66], [200]], ids=lambda x: "-".join(map(str, x[:5])) + f"x{len(x)}")
def test_requests_of_few_and_of_many_tokens(d, lens):
    B = sum(lens) + 3
    _check(_fill(lens, B), 2, d, seed=sum(lens))
    _check(lens + [0] * (B - len(lens)), 1, d, resume=[i % 2 for i in range(B)], tail=3, seed=sum(lens) + 1)
    _check([0] * (B - len(lens)) + lens, 1, d, resume=[1] * B, seed=sum(lens) + 2)


def test_many_heads():
    _check(_fill([100, 5, 40, 1, 1, 70], 220), 40, 64, seed=3)


def test_bad_slots_are_skipped():
    lens = _fill([70, 3, 40, 5, 66], 190)
    slots = list(range(190))
    at = [i for i, n in enumerate(lens) if n]
    slots[at[0]], slots[at[1]] = 999, -4
    _check(lens, 2, 64, slots=slots, num_slots=190, seed=4)


def test_lists_that_do_not_ascend_stay_inside():
    H, d, T, B = 2, 64, 100, 120
    q, k, v, a, b = (x.cuda() for x in _inputs(31, T, H, d))
    rng = np.random.default_rng(7)
    for cu in ([-5] * 40 + [60] * 40 + [4000] * 41, [90] * 60 + [20] * 61, [2 ** 31 - 1] * 121, [int(x) for x in rng.integers(-50, 200, B + 1)]):
        pool = torch.zeros((B + 2, H, d, d), device="cuda")
        guard = torch.full((T + 128, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
        ws = torch.full((lib.prefill_workspace_bytes(True, B, T, H, d, torch.bfloat16) + 4096,), 3, dtype=torch.uint8, device="cuda")
        lib.fp32_delta_prefill(pool, torch.arange(1, B + 1, dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                               q, k, v, a, b, guard[64:64 + T], workspace=ws[:-4096])
        torch.cuda.synchronize()
        assert bool((guard[:64] == 3.0).all()) and bool((guard[64 + T:] == 3.0).all()) and bool((ws[-4096:] == 3).all())
        assert bool((pool[[0, B + 1]] == 0).all())


def test_in_a_graph_with_other_lengths():
    H, d, B = 3, 128, 150
    T = B
    q, k, v, a, b = (x.cuda() for x in _inputs(41, T, H, d))
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    sl, one = torch.randperm(B).to(torch.int32).cuda(), torch.ones(B, dtype=torch.int32, device="cuda")
    start = torch.randn((B, H, d, d), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    eager, graphed, oe, og = start.clone(), start.clone(), torch.empty_like(v), torch.empty_like(v)
    lib.fp32_delta_prefill(start, sl, cu, q, k, v, a, b, og, resume=one)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.fp32_delta_prefill(graphed, sl, cu, q, k, v, a, b, og, resume=one)
    noise = torch.zeros(1 << 20, device="cuda")
    for i, lens in enumerate(([1] * B, _fill([B], B), _fill([100, 50], B), _fill([33, 32, 1, 40, 44], B))):
        cu.copy_(torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32))
        lib.fp32_delta_prefill(eager, sl, cu, q, k, v, a, b, oe, resume=one)
        g.replay()
        noise.add_(1.0)
        torch.cuda.synchronize()
        assert torch.equal(oe, og) and torch.equal(eager, graphed), f"replay {i}"
