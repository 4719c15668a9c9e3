"""How well the softmax weights of kv_decode_attention enter the product with V.

Bounds. A weight enters as two bf16 pieces: the first is the weight less 2^-12 of it, cut off (below
2^-7 + 2^-12 of the weight is left), the second what is left, rounded (half a step, 2^-8), so together they
are within 2^-15 + 2^-20 of it. Sums over n tokens add n / 32 + 64 roundings of 2^-24 (products and joins), the
normaliser as many, the scores what serving_ref.score_error says on both sides of the quotient, and the
result's own rounding to bf16 is 2^-8 of it."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import serving_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib  # noqa: E402


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(x, page):
    """[n, Hkv, d] as pages [blocks, Hkv, page, d], NaN behind the tokens."""
    n, H, d = x.shape
    blocks = -(-n // page)
    y = torch.full((blocks * page, H, d), float("nan"), dtype=x.dtype)
    y[:n] = x
    return y.reshape(blocks, page, H, d).transpose(1, 2).contiguous()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [700, 8192])
@pytest.mark.parametrize("p", [0.50195, 0.25097, 0.12548, 0.501953125, 0.50585938, 0.2509765625, 0.7519531, 0.9980469, 1.0 / 3.0])
def test_a_plateau_of_equal_weights_under_a_maximum(d, n, p):
    """All weights below the maximum are the same value p, so that nothing of its rounding averages out; the
    maximum stands in the first tile of each wave, however the tokens are cut (a wave's weights go by its own
    maximum). A constant V comes back exactly: the weights sum to 1 within 2^-15 + 2^-20 + 2 (n / 32 + 64) 2^-24
    < 2^-14, relative, and a bf16 value's neighbours are 2^-8 and more away."""
    q = torch.zeros((1, 2, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    k = torch.zeros((n, 1, d), dtype=torch.bfloat16)
    for t in range(0, n, 256):
        k[t:t + 128:32, 0, 0] = 1.0
    v = torch.tensor([1.0, -3.5, 0.0078125, 96.0]).repeat(d // 4).bfloat16().expand(n, 1, d).contiguous()
    out = torch.empty_like(q)
    kp, vp = _pages(k, 16).cuda(), _pages(v, 16).cuda()
    lib.kv_decode_attention(q, kp, vp, torch.arange(kp.shape[0], dtype=torch.int32, device="cuda")[None], _i32([n]), out, scale=-math.log(p))
    torch.cuda.synchronize()
    assert torch.equal(out[0].cpu(), v[0].expand(2, d)), f"{float((out[0].cpu().double() / v[0].double() - 1).abs().max()):.3g} off"


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 4, 1), (128, 6, 2)])
@pytest.mark.parametrize("lens", [[1, 31, 100], [1000, 700], [3000, 40]], ids=str)
def test_random_scores_to_the_pieces_bound(d, Hq, Hkv, lens):
    gen = torch.Generator().manual_seed(sum(lens) + d)
    kv = [[torch.randn((n, Hkv, d), generator=gen).bfloat16() for _ in range(2)] for n in lens]
    q = (2 * torch.randn((len(lens), Hq, d), generator=gen)).bfloat16()
    kp, vp = (torch.cat([_pages(x[i], 16) for x in kv]) for i in range(2))
    table, at = torch.zeros((len(lens), -(-max(lens) // 16)), dtype=torch.int32), 0
    for b, n in enumerate(lens):
        m = -(-n // 16)
        table[b, :m] = torch.arange(at, at + m)
        at += m
    out = torch.empty((len(lens), Hq, d), dtype=torch.bfloat16, device="cuda")
    lib.kv_decode_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32(lens), out)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        k, v = (x.double() for x in kv[b])
        o, mag = ref.attention(q[b].double(), k, v, d ** -0.5)
        e = 2.0 ** -15 + 2.0 ** -20 + 2 * (ref.score_error(q[b].double(), k, d ** -0.5) + (n // 32 + 64) * ref.EPS32)
        ref.is_close(out[b], o, 2.0 ** -8 * o.abs() + e * mag + 1e-37, f"{n} tokens")


@pytest.mark.parametrize("n", [9, 2500])
def test_an_infinite_value_stays_infinite(n):
    """Weights that are bf16 values (1 and 2^-3) leave nothing for a second piece; infinity times nothing
    would be NaN."""
    d = 64
    q = torch.zeros((1, 1, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    k, v = torch.zeros((n, 1, d), dtype=torch.bfloat16), torch.ones((n, 1, d), dtype=torch.bfloat16)
    k[4, 0, 0] = 3.0
    v[4, 0, 1], v[6, 0, 2], v[7, 0, 3] = math.inf, math.inf, -math.inf
    out = torch.empty_like(q)
    kp, vp = _pages(k, 16).cuda(), _pages(v, 16).cuda()
    lib.kv_decode_attention(q, kp, vp, torch.arange(kp.shape[0], dtype=torch.int32, device="cuda")[None], _i32([n]), out, scale=math.log(2.0))
    torch.cuda.synchronize()
    o = out[0, 0].cpu()
    assert float(o[1]) == math.inf and float(o[2]) == math.inf and float(o[3]) == -math.inf
    assert bool((o[4:] == 1.0).all()) and float(o[0]) == 1.0
