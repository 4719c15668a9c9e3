"""Linear attention with a decay and the prompt forms (fp32_linear_step, fp32_linear_prefill,
fp32_delta_prefill) against token-by-token references in binary64.

Bounds. Linear attention is a sum of products, so an element's error is at most (roundings on a
term's way) * 2^-24 * (the same sum by magnitude). A term passes: its product and its share of a
64-token sum (each of up to 3 partial products adds), the decay's power (its logarithm, running sum,
exponential), and 4 more per later chunk (or per token in the token-by-token form); 512 + 8 per step
of the chain covers them. Readouts stored as bf16 add 2^-8 of the value, and two bf16 pieces of the
weights and of the state 2^-17 each of the magnitude. The delta rule's state is held by column
norms: I - beta k k^T with unit k and beta in [0, 1] does not stretch, so the local errors
(d + 70 roundings of a column's norm, magnified by the chunk's condition number) only add up."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import serving_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _alpha(gen, n, H, d, form):
    life = torch.exp2(torch.linspace(1.0, 11.0, H)) if H > 1 else torch.tensor([20.0])
    if form == "head":
        return torch.exp2(-1.0 / life)
    if form == "key":
        return torch.exp2(-(0.2 + torch.rand((n, H, d), generator=gen)) / life[:, None])
    return torch.exp2(-(0.2 + torch.rand((n, H), generator=gen)) / life)


def _inputs(seed, T, H, d, dtype, form):
    gen = torch.Generator().manual_seed(seed)
    q, k = (_unit(torch.randn((T, H, d), generator=gen)).to(DT[dtype]) for _ in range(2))
    v = torch.randn((T, H, d), generator=gen).to(DT[dtype])
    return q, k, v, _alpha(gen, T, H, d, form), torch.sigmoid(torch.randn((T, H), generator=gen))


# ---- the single-token step ---------------------------------------------------------------------
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("form", ["token", "key", "head"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_linear_step(d, form, dtype):
    B, H, slots = 5, 3, 9
    q, k, v, alpha, _ = _inputs(d, B, H, d, dtype, form)
    gen = torch.Generator().manual_seed(1)
    pool = torch.randn((slots, H, d, d), generator=gen)
    idx = torch.tensor([7, 0, 3, 8, 4], dtype=torch.int32)
    got, out = pool.cuda(), torch.full((B, H, d), float("nan"), device="cuda")
    lib.fp32_linear_step(got, idx.cuda(), q.cuda(), k.cuda(), v.cuda(), alpha.cuda(), out)
    torch.cuda.synchronize()
    want = pool.double()
    for b in range(B):
        for h in range(H):
            a = alpha[h] if form == "head" else alpha[b, h]
            S = pool[idx[b], h].double()
            o, X, mag, A, _ = ref.prompt(S, q[b, h].double()[None], k[b, h].double()[None], v[b, h].double()[None],
                                         a.double().reshape(1, -1) if form == "key" else a.double().reshape(1))
            want[idx[b], h] = X
            ref.is_close(got[idx[b], h], X, 3 * ref.EPS32 * A, f"state {b} {h}")
            ref.is_close(out[b, h], o[0], (d + 4) * ref.EPS32 * mag[0], f"readout {b} {h}")
    rest = [s for s in range(slots) if s not in idx.tolist()]
    assert torch.equal(got[rest].cpu(), pool[rest])


def test_linear_step_degenerate():
    """Gates of 0 and 1, zero states, a bad slot (skipped), an empty batch."""
    H, d = 2, 64
    q, k, v, _, _ = _inputs(3, 4, H, d, "bf16", "token")
    pool = torch.randn((4, H, d, d), generator=torch.Generator().manual_seed(2))
    pool[2] = 0
    idx = torch.tensor([0, 9, 2, -1], dtype=torch.int32)
    alpha = torch.tensor([[0.0, 1.0]] * 4)
    got, out = pool.cuda(), torch.full((4, H, d), 7.0, device="cuda")
    lib.fp32_linear_step(got, idx.cuda(), q.cuda(), k.cuda(), v.cuda(), alpha.cuda(), out)
    torch.cuda.synchronize()
    kv = k.float()[..., :, None] * v.float()[..., None, :]
    assert torch.equal(got[0, 0].cpu(), kv[0, 0]) and torch.equal(got[2].cpu(), kv[2])
    assert torch.equal(got[0, 1].cpu(), pool[0, 1] + kv[0, 1])
    assert torch.equal(got[[1, 3]].cpu(), pool[[1, 3]]) and bool((out[[1, 3]] == 7.0).all())
    none = torch.zeros((0, H, d), device="cuda")
    lib.fp32_linear_step(got, torch.zeros(0, dtype=torch.int32, device="cuda"), none, none, none, torch.ones(H, device="cuda"), none)


# ---- prompts -----------------------------------------------------------------------------------
def _run(delta, lens, H, d, dtype, form, resume=None, slots=None, num_slots=None, seed=0, tail=0, alpha=None, beta=None, qkv=None):
    """Runs a prefill and checks every readout, state and untouched place. Returns how much of the bounds was used."""
    B, T = len(lens), sum(lens)
    rows = T + tail
    q, k, v, a, b = _inputs(seed, rows, H, d, dtype, form)
    if qkv is not None:
        q, k, v = qkv
    a = a if alpha is None else alpha
    b = b if beta is None else beta
    gen = torch.Generator().manual_seed(seed + 77)
    num_slots = num_slots or B + 2
    slots = torch.randperm(num_slots, generator=gen)[:B].to(torch.int32) if slots is None else torch.tensor(slots, dtype=torch.int32)
    pool = torch.randn((num_slots, H, d, d), generator=gen)
    if resume is None:
        pool[slots.long().clamp(0, num_slots - 1)] = float("nan")   # a fresh request reads nothing of its slot
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    got, out = pool.cuda(), torch.full((rows, H, d), 7.0, dtype=DT[dtype], device="cuda")
    args = (got, slots.cuda(), cu.cuda(), q.cuda(), k.cuda(), v.cuda(), a.cuda())
    res = None if resume is None else torch.tensor(resume, dtype=torch.int32).cuda()
    if delta:
        lib.fp32_delta_prefill(*args, b.cuda(), out, resume=res)
    else:
        lib.fp32_linear_prefill(*args, out, resume=res)
    torch.cuda.synchronize()
    used = 0.0
    assert bool((out[T:] == 7.0).all()), "rows behind the last request were written"
    for i in range(B):
        r = slice(int(cu[i]), int(cu[i + 1]))
        s = int(slots[i])
        if not 0 <= s < num_slots:
            assert bool((out[r] == 7.0).all()), f"request {i} has no slot"
            continue
        n = lens[i]
        for h in range(H):
            S = pool[s, h].double() if resume is not None and resume[i] else torch.zeros((d, d), dtype=torch.float64)
            if n == 0:
                assert torch.equal(got[s, h].cpu(), pool[s, h]) or bool(pool[s, h].isnan().all()), f"request {i} has no tokens"
                continue
            al = a[h].double().expand(n) if form == "head" else a[r, h].double()
            x = [y[r, h].double() for y in (q, k, v)]
            o, X, mag, A, top = ref.prompt(S, *x, al, b[r, h].double() if delta else None)
            by_token = dtype == "fp32" or form == "key" or d < 64 or (delta and rows <= max(32, B))   # the form the call takes
            chain = n if by_token else -(-n // 64)
            store = 2.0 ** -8 if dtype == "bf16" else ref.EPS32
            if not delta:
                e_state = (512 + 8 * chain) * ref.EPS32 * A
                e_out = store * o.abs() + ((512 + 8 * chain + d) * ref.EPS32 + (2.0 ** -16 if dtype == "bf16" else 0.0)) * mag
                used = max(used, ref.is_close(got[s, h], X, e_state + 1e-37, f"state {i} {h}"))
                used = max(used, ref.is_close(out[r, h], o, e_out + 1e-37, f"readouts {i} {h}"))
            else:
                kappa = ref.chunk_condition(x[1], al, b[r, h].double()) if not by_token else 1.0
                e_col = (2 * d + 140 + 16) * chain * kappa * ref.EPS32 * top
                err = (got[s, h].double().cpu() - X).norm(dim=0)
                assert bool((err <= e_col).all()), f"state {i} {h}: {float((err / e_col).max()):.3g} of the bound"
                e_out = store * o.abs() + x[0].norm(dim=-1, keepdim=True) * (e_col + (2.0 ** -15 * kappa if dtype == "bf16" else d * ref.EPS32) * top)
                used = max(used, float((err / e_col).max()), ref.is_close(out[r, h], o, e_out, f"readouts {i} {h}"))
    rest = [s for s in range(num_slots) if s not in slots.tolist()]
    assert torch.equal(got[rest].cpu().view(torch.int32), pool[rest].view(torch.int32)), "a slot of no request was written"
    return used


RULES = pytest.mark.parametrize("delta", [False, True], ids=["linear", "delta"])


@RULES
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("form", ["token", "key"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_prompts_of_every_form(delta, d, form, dtype):
    _run(delta, [37, 1, 70], 3, d, dtype, form, resume=[1, 0, 1], seed=d)


@RULES
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,form", [("bf16", "key"), ("fp32", "key"), ("fp32", "token")])
def test_token_by_token_lengths(delta, d, dtype, form):
    """Lengths around the blocks of 16 tokens that are staged at a time, rows behind the last request."""
    _run(delta, [300, 17, 16, 0, 15, 1, 33], 3, d, dtype, form, resume=[1, 0, 1, 0, 0, 1, 0], seed=d + 5, tail=2)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_prompts_with_a_fixed_decay_per_head(d):
    _run(False, [130, 5, 64], 3, d, "bf16", "head", seed=d)
    _run(False, [19, 40], 2, d, "fp32", "head", resume=[0, 1], seed=d + 1)


@RULES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63], [64], [65], [127], [128], [129], [193], [0], [0, 1, 0], [64, 64], [1, 0, 63, 200, 2, 65, 128]],
                         ids=lambda x: "-".join(map(str, x)))
def test_prompt_lengths(delta, d, lens):
    _run(delta, lens, 2, d, "bf16", "token", seed=sum(lens) + 1, tail=3)


@RULES
@pytest.mark.parametrize("heads", [1, 5, 33])
def test_prompt_heads_and_resumed_parts(delta, heads):
    _run(delta, [70, 130, 3], heads, 64, "bf16", "token", resume=[1, 0, 1], seed=heads)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[31], [32], [33], [1] * 40, [0] * 45 + [44], [1] * 40 + [2], [3, 0, 29]], ids=lambda x: f"{len(x)}x{sum(x)}")
def test_delta_calls_of_few_tokens(d, lens):
    """Around the sizes up to which a call runs token by token."""
    _run(True, lens, 3, d, "bf16", "token", resume=[i % 2 for i in range(len(lens))], seed=sum(lens))
    _run(True, lens, 1, d, "bf16", "token", seed=len(lens))


@RULES
@pytest.mark.parametrize("d", [64, 128])
def test_long_prompt(delta, d):
    _run(delta, [1500, 700], 1, d, "bf16", "token", resume=[0, 1], seed=4)


@RULES
def test_prompt_bad_slots_are_skipped(delta):
    _run(delta, [20, 66, 5, 7], 2, 64, "bf16", "token", slots=[1, 99, 0, -3], num_slots=3, seed=9)
    _run(delta, [20, 66, 5, 7], 2, 32, "fp32", "token", slots=[1, 99, 0, -3], num_slots=3, seed=9)


@RULES
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_gates_of_zero_and_one(delta, d):
    """Decays of exactly 0 (a state forgotten within a chunk), 1, and strong ones (sums of logarithms in the thousands)."""
    gen = torch.Generator().manual_seed(5)
    T, H = 150, 3
    alpha = torch.ones((T, H))
    alpha[torch.rand((T, H), generator=gen) < 0.1] = 0.0
    alpha[:, 1] = torch.exp2(-60.0 * torch.rand(T, generator=gen))
    alpha[100:, 1] = 1.0
    alpha[:, 2] = 1.0
    _run(delta, [T], H, d, "bf16", "token", resume=[1], alpha=alpha, seed=6)


@pytest.mark.parametrize("d", [64, 128])
def test_delta_prompt_of_equal_keys(d):
    """The same key again and again with beta near 1: the chunk's system is as coupled as it gets."""
    q, k, v, _, _ = _inputs(8, 130, 2, d, "bf16", "token")
    k = k[:1].expand(130, 2, d).contiguous()
    _run(True, [130], 2, d, "bf16", "token", alpha=torch.full((130, 2), 0.999), beta=torch.full((130, 2), 0.97), qkv=(q, k, v), seed=8)
    _run(True, [130], 2, d, "bf16", "token", resume=[1], alpha=torch.ones((130, 2)), beta=torch.zeros((130, 2)), qkv=(q, k, v), seed=8)


@RULES
def test_prompt_in_parts_equals_steps(delta):
    """A prompt taken in two parts and three single tokens gives the state of the whole prompt."""
    H, d, T = 2, 128, 203
    q, k, v, a, b = (x.cuda() for x in _inputs(21, T, H, d, "bf16", "token"))
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    whole, parts = (torch.zeros((1, H, d, d), device="cuda") for _ in range(2))
    out, out2 = torch.empty_like(v), torch.empty_like(v)
    one = torch.ones(1, dtype=torch.int32, device="cuda")

    def prefill(pool, lo, hi, o, resume):
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        x = [y[lo:hi] for y in (q, k, v, a)]
        if delta:
            lib.fp32_delta_prefill(pool, slot, cu, *x, b[lo:hi], o[lo:hi], resume=resume)
        else:
            lib.fp32_linear_prefill(pool, slot, cu, *x, o[lo:hi], resume=resume)

    prefill(whole, 0, T, out, None)
    prefill(parts, 0, 90, out2, None)
    prefill(parts, 90, 200, out2, one)
    for t in range(200, 203):
        y = torch.empty((1, H, d), device="cuda")
        x = [z[t:t + 1] for z in (q, k, v, a)]
        if delta:
            lib.fp32_decode_step(parts, slot, *x, b[t:t + 1], y)
        else:
            lib.fp32_linear_step(parts, slot, *x, y)
        out2[t] = y[0].bfloat16()
    torch.cuda.synchronize()
    assert float((whole - parts).norm() / whole.norm()) < 1000 * ref.EPS32
    assert float((out.float() - out2.float()).abs().max()) <= 2.0 ** -7 * float(out.float().abs().max())


@RULES
@pytest.mark.parametrize("d,heads", [(64, 90), (128, 33)])
def test_prompts_of_many_heads(delta, d, heads):
    """More states than fill the chip: 32 value columns a workgroup in the delta rule's chain (and whole prompts of linear attention)."""
    _run(delta, [70, 130, 3], heads, d, "bf16", "token", resume=[1, 0, 1], seed=heads)


@RULES
@pytest.mark.parametrize("heads", [2, 8])
@pytest.mark.parametrize("requests", [32, 33, 70])
def test_many_prompts(delta, requests, heads):
    """Up to 32 requests start the longest first, more as they come; several of the same length, some without tokens."""
    rng = np.random.default_rng([requests, heads])
    lens = [int(x) for x in rng.choice([0, 1, 17, 64, 65, 90], requests)]
    _run(delta, lens, heads, 64, "bf16", "token", resume=[i % 2 for i in range(requests)], seed=requests)


@RULES
@pytest.mark.parametrize("dtype,d,form", [("bf16", 64, "token"), ("bf16", 128, "token"), ("fp32", 32, "token"), ("bf16", 32, "key")])
def test_nan_in_one_prompt_stays_there(delta, dtype, d, form):
    """A NaN gate, key or value makes the states of its own request NaN and leaves the other requests' results as they were."""
    H, lens = 2, [70, 40, 66]
    T = sum(lens)
    cu = torch.tensor([0, 70, 110, 176], dtype=torch.int32, device="cuda")
    sl = torch.arange(3, dtype=torch.int32, device="cuda")
    x = [y.cuda() for y in _inputs(51, T, H, d, dtype, form)]

    def call(q, k, v, a, b):
        pool, out = torch.zeros((3, H, d, d), device="cuda"), torch.zeros_like(v)
        if delta:
            lib.fp32_delta_prefill(pool, sl, cu, q, k, v, a, b, out)
        else:
            lib.fp32_linear_prefill(pool, sl, cu, q, k, v, a, out)
        torch.cuda.synchronize()
        return pool, out

    pool, out = call(*x)
    for which in (1, 2, 3):                        # k, v, alpha of the middle request's first and last token
        for row in (70, 109):
            y = [z.clone() for z in x]
            y[which][row] = float("nan")
            p, o = call(*y)
            assert bool(p[1].isnan().all()), f"input {which}, row {row}"
            assert torch.equal(p[[0, 2]], pool[[0, 2]]) and torch.equal(o[:70], out[:70]) and torch.equal(o[110:], out[110:])


@RULES
def test_cut_prompts_in_a_graph(delta):
    """Long prompts of few heads (linear attention in segments, over three launches), replayed."""
    H, d, T = 2, 64, 1600
    q, k, v, a, b = (x.cuda() for x in _inputs(61, T, H, d, "bf16", "token"))
    cu = torch.tensor([0, 1300, 1600], dtype=torch.int32, device="cuda")
    sl, one = torch.tensor([1, 0], dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    start = torch.randn((2, H, d, d), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    eager, graphed, oe, og = start.clone(), start.clone(), torch.empty_like(v), torch.empty_like(v)

    def call(pool, out):
        if delta:
            lib.fp32_delta_prefill(pool, sl, cu, q, k, v, a, b, out, resume=one)
        else:
            lib.fp32_linear_prefill(pool, sl, cu, q, k, v, a, out, resume=one)

    call(start, og)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(graphed, og)
    noise = torch.zeros(1 << 20, device="cuda")
    for i in range(4):
        cu.copy_(torch.tensor([0, 1300 - 257 * i, 1600], dtype=torch.int32))
        call(eager, oe)
        g.replay()
        noise.add_(1.0)
        torch.cuda.synchronize()
        assert torch.equal(oe, og) and torch.equal(eager, graphed), f"replay {i}"


def test_prompt_refusals():
    H, d, T = 2, 64, 10
    q, k, v, a, b = (x.cuda() for x in _inputs(1, T, H, d, "bf16", "token"))
    pool = torch.zeros((3, H, d, d), device="cuda")
    sl, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out = torch.empty_like(v)
    with pytest.raises(ValueError):
        lib.fp32_linear_prefill(pool, sl, cu[:1], q, k, v, a, out)
    with pytest.raises(TypeError):
        lib.fp32_linear_prefill(pool, sl, cu, q, k, v, a, out.float())
    with pytest.raises(TypeError):
        lib.fp32_linear_prefill(pool, sl, cu, q.half(), k, v, a, out)
    with pytest.raises(ValueError):
        lib.fp32_linear_prefill(pool, sl, cu, q, k[:5], v, a, out)
    with pytest.raises(ValueError):
        lib.fp32_delta_prefill(pool, sl, cu, q, k, v, a[0], b, out)          # no fixed decays
    with pytest.raises(ValueError):
        lib.fp32_delta_prefill(pool, sl, cu, q, k, v, a, b[:3], out)
    with pytest.raises(ValueError):
        lib.fp32_delta_prefill(pool, sl, cu, q, k, v, a, b, out.transpose(0, 1))
    need = lib.prefill_workspace_bytes(True, 1, T, H, d, torch.bfloat16)
    if need:
        with pytest.raises(ValueError):
            lib.fp32_delta_prefill(pool, sl, cu, q, k, v, a, b, out, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        lib.fp32_linear_step(pool, sl, q[:1], k[:1], v[:1], a[:1], torch.empty((2, H, d), device="cuda"))
    with pytest.raises(lib.DampError) as e:
        p48 = torch.zeros((3, H, 48, 48), device="cuda")
        z = torch.zeros((T, H, 48), device="cuda")
        lib.fp32_linear_prefill(p48, sl, cu, z, z, z, a, z.clone())
    assert e.value.status == lib.DAMP_ERR_UNSUPPORTED
    assert bool((pool == 0).all())


@RULES
def test_prompts_with_lists_that_do_not_ascend_stay_inside(delta):
    """A cu_seqlens that points outside the tokens or goes back: no access leaves the arrays (guard rows keep their values)."""
    H, d, T = 2, 64, 100
    q, k, v, a, b = (x.cuda() for x in _inputs(31, T, H, d, "bf16", "token"))
    for cu in ([-5, 60, 4000], [90, 20, 100], [0, 2 ** 31 - 1, 50], [100, 100, 100]):
        pool = torch.zeros((4, H, d, d), device="cuda")
        guard = torch.full((T + 128, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        sl = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
        if delta:
            lib.fp32_delta_prefill(pool, sl, c, q, k, v, a, b, guard[64:64 + T])
        else:
            lib.fp32_linear_prefill(pool, sl, c, q, k, v, a, guard[64:64 + T])
        torch.cuda.synchronize()
        assert bool((guard[:64] == 3.0).all()) and bool((guard[64 + T:] == 3.0).all())
        assert bool((pool[[0, 3]] == 0).all())


# ---- graphs and streams -----------------------------------------------------------------------
@RULES
def test_prompts_in_a_graph_and_on_two_streams(delta):
    H, d, lens = 4, 128, [130, 70]
    T = sum(lens)
    q, k, v, a, b = (x.cuda() for x in _inputs(41, T, H, d, "bf16", "token"))
    cu = torch.tensor([0, 130, 200], dtype=torch.int32, device="cuda")
    sl = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    one = torch.ones(2, dtype=torch.int32, device="cuda")

    def call(pool, out, stream=None):
        if delta:
            lib.fp32_delta_prefill(pool, sl, cu, q, k, v, a, b, out, resume=one, stream=stream)
        else:
            lib.fp32_linear_prefill(pool, sl, cu, q, k, v, a, out, resume=one, stream=stream)

    start = torch.randn((2, H, d, d), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    eager, graphed = start.clone(), start.clone()
    oe, og = torch.empty_like(v), torch.empty_like(v)
    call(start.clone(), og)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(graphed, og)
    noise = torch.zeros(1 << 20, device="cuda")
    for i in range(4):
        call(eager, oe)
        g.replay()
        noise.add_(1.0)
        torch.cuda.synchronize()
        assert torch.equal(oe, og) and torch.equal(eager, graphed), f"replay {i}"
    pools, outs, streams = [start.clone(), start.clone()], [torch.empty_like(v) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for p, o, s in zip(pools, outs, streams):
            call(p, o, s)
    torch.cuda.synchronize()
    for p, o in zip(pools, outs):
        assert torch.equal(p, eager) and torch.equal(o, oe)
