"""Forms of the prompt kernels that a call takes by its sizes: linear attention in segments with fixed decays,
with requests that are skipped and with segments of more than 256 tokens; requests that start the longest first.
Bounds as for the other prompt tests (serving_ref, test_gpu_linear)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import serving_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib  # noqa: E402
from test_gpu_linear import _alpha, _run, _unit  # noqa: E402

RULES = pytest.mark.parametrize("delta", [False, True], ids=["linear", "delta"])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1500, 700], [513], [0, 1, 900, 257, 255], [256, 512, 64, 1]], ids=str)
def test_long_prompts_with_a_fixed_decay_per_head(d, lens):
    _run(False, lens, 2, d, "bf16", "head", resume=[i % 2 for i in range(len(lens))], seed=d + sum(lens), tail=3)
    _run(False, lens, 1, d, "bf16", "head", seed=d)


@RULES
@pytest.mark.parametrize("form", ["token", "head"])
def test_long_prompts_with_bad_slots(delta, form):
    if delta and form == "head":
        form = "token"
    for d in (64, 128):
        _run(delta, [700, 900, 5, 600], 1, d, "bf16", form, slots=[1, 99, 0, -3], num_slots=3, seed=9)


@RULES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("requests,heads", [(32, 9), (31, 16), (2, 140)])
def test_requests_start_the_longest_first(delta, d, requests, heads):
    """More workgroups than CUs and up to 32 requests; several of the same length, some without tokens."""
    rng = np.random.default_rng([requests, heads, d])
    lens = [int(x) for x in rng.choice([0, 1, 17, 64, 65, 90], requests)]
    _run(delta, lens, heads, d, "bf16", "token", resume=[i % 2 for i in range(requests)], seed=requests + d)


def _some_heads(lens, H, d, form, heads, resume, seed):
    """Linear prompts of many heads, of which some are checked."""
    T, B = sum(lens), len(lens)
    gen = torch.Generator().manual_seed(seed)
    q, k = (_unit(torch.randn((T, H, d), generator=gen)).bfloat16() for _ in range(2))
    v, a = torch.randn((T, H, d), generator=gen).bfloat16(), _alpha(gen, T, H, d, form)
    pool = torch.randn((B + 1, H, d, d), generator=gen)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    slots = torch.arange(B, 0, -1, dtype=torch.int32)
    got, out = pool.cuda(), torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda")
    lib.fp32_linear_prefill(got, slots.cuda(), cu.cuda(), q.cuda(), k.cuda(), v.cuda(), a.cuda(), out, resume=torch.tensor(resume, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.equal(got[0].cpu(), pool[0])
    for b, n in enumerate(lens):
        r, s = slice(int(cu[b]), int(cu[b + 1])), int(slots[b])
        for h in heads:
            S = pool[s, h].double() if resume[b] else torch.zeros((d, d), dtype=torch.float64)
            o, X, mag, A, _ = ref.prompt(S, *(y[r, h].double() for y in (q, k, v)), a[h].double().expand(n) if form == "head" else a[r, h].double())
            chain = -(-n // 64)
            ref.is_close(got[s, h], X, (512 + 8 * chain) * ref.EPS32 * A + 1e-37, f"state {b} {h}")
            ref.is_close(out[r, h], o, 2.0 ** -8 * o.abs() + ((512 + 8 * chain + d) * ref.EPS32 + 2.0 ** -16) * mag + 1e-37, f"readouts {b} {h}")


@pytest.mark.parametrize("form", ["token", "head"])
@pytest.mark.parametrize("lens,H", [([2500], 60), ([321, 1900, 640], 65), ([1, 3000], 100)], ids=str)
def test_segments_of_more_than_256_tokens(lens, H, form):
    """T * H above 131,072: segments of up to 320, 384 and 640 tokens."""
    _some_heads(lens, H, 64, form, (0, H - 1), [i % 2 for i in range(len(lens))], seed=H)


def test_segments_of_more_than_256_tokens_at_128_channels():
    _some_heads([1700, 900], 70, 128, "token", (3, 69), [1, 0], seed=5)


@RULES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,total", [(64, 4.0), (64, 30.0), (64, 90.0), (200, 1.0), (200, 60.0), (1500, 0.3), (1500, 90.0)])
def test_decays_to_their_bound(delta, d, n, total):
    """Only the first token writes (later values are 0, by the delta rule with beta 0), so the last state is the
    product of n - 1 decays times k v^T. An exponent x is a sum of binary32 logarithms (within 2^-23 of each),
    taken as a difference and rounded (2^-23 of it more): 2^-22 |x| in all, over all chunks together, as every
    chunk's is relative to its own share of x. Its power adds 2^-23 and the product with the state 2^-24 a chunk,
    the first chunk's product with three pieces of the value 3 2^-23. Relative to the value, in every element."""
    H = 3
    gen = torch.Generator().manual_seed(n + d)
    q, k = (_unit(torch.randn((n, H, d), generator=gen)).bfloat16() for _ in range(2))
    v = torch.zeros((n, H, d))
    v[0] = torch.randn((H, d), generator=gen)
    v = v.bfloat16()
    w = torch.rand((n, H), generator=gen)
    w[:, 1] = 1.0                                              # even decays, random ones, and a few strong ones
    w[:, 2] = (torch.rand(n, generator=gen) < 0.1).float() + 1e-3
    alpha = torch.exp2(-total * w / w.sum(0))
    beta = torch.zeros((n, H))
    beta[0] = 1.0
    pool, out = torch.zeros((1, H, d, d), device="cuda"), torch.empty((n, H, d), dtype=torch.bfloat16, device="cuda")
    args = (pool, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda"), q.cuda(), k.cuda(), v.cuda(), alpha.cuda())
    if delta:
        lib.fp32_delta_prefill(*args, beta.cuda(), out)
    else:
        lib.fp32_linear_prefill(*args, out)
    torch.cuda.synchronize()
    for h in range(H):
        x = alpha[1:, h].double().log2().sum()
        want = torch.exp2(x) * torch.outer(k[0, h].double(), v[0, h].double())
        bound = (2.0 ** -22 * float(-x) * 0.6931471805599453 + (-(-n // 64) * 1.5 + 4) * 2.0 ** -23) * want.abs()
        ref.is_close(pool[0, h], want, bound, f"head {h}, decay 2^{float(x):.3g}")
