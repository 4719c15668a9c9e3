"""The serving operators together, as a hybrid model uses them. Two layers: a gated delta rule layer
whose states live in a DAMP pool, and a full-attention layer on a paged cache; and the same with a
linear-attention layer on its fp32 pool. Prompts of a ragged batch go in by the tables of kv_build_tables
(whose running sums are the prompt forms' cu_seqlens), their states are packed, and tokens follow one at
a time, new pages taken as requests grow. Every attention readout and recurrent readout is compared with
binary64 references of the whole history (the packed state's readouts with the fp32 pool's)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import serving_ref as ref  # noqa: E402
from quantized_delta_rule_gdn_amd import lib, synth  # noqa: E402

H, HKV, D, PAGE, STEPS = 4, 2, 128, 16, 5
LENS = [70, 1, 129, 15, 48]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rule", ["delta", "linear"])
def test_prompts_then_tokens(rule):
    gen = torch.Generator().manual_seed(12)
    B, T = len(LENS), sum(LENS)
    total = [n + STEPS for n in LENS]

    def rand(*shape):
        return torch.randn(shape, generator=gen)

    # the whole history of each request, in binary64 copies of what the kernels get
    q = [(x / x.norm(dim=-1, keepdim=True)).bfloat16() for x in (rand(n, H, D) for n in total)]
    k = [(x / x.norm(dim=-1, keepdim=True)).bfloat16() for x in (rand(n, H, D) for n in total)]
    v = [rand(n, H, D).bfloat16() for n in total]
    alpha = [torch.exp2(-torch.rand((n, H), generator=gen) / torch.tensor([4.0, 16.0, 64.0, 512.0])) for n in total]
    beta = [torch.sigmoid(rand(n, H)) for n in total]
    aq = [rand(n, H, D).bfloat16() for n in total]
    ak, av = ([rand(n, HKV, D).bfloat16() for n in total] for _ in range(2))

    def cat(xs, sel):
        return torch.cat([x[s] for x, s in zip(xs, sel)]).cuda()

    prompt = [slice(0, n) for n in LENS]
    pages, blocks = 64, 12
    kp, vp = (torch.full((pages, HKV, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    free = torch.randperm(pages, generator=gen).to(torch.int32).cuda()
    table = torch.full((B, blocks), -1, dtype=torch.int32, device="cuda")
    cu, used = _i32([0] * (B + 1)), _i32([0])
    seq = _i32(LENS)
    slot_map, positions = torch.empty(T + 7, dtype=torch.int64, device="cuda"), _i32([0] * (T + 7))   # a padded batch
    lib.kv_build_tables(seq, seq, free, table, PAGE, slot_map, positions, cu, used)
    pad = torch.full((7, HKV, D), float("inf"), dtype=torch.bfloat16, device="cuda")                # rows of no token
    lib.kv_append(torch.cat([cat(ak, prompt), pad]), torch.cat([cat(av, prompt), pad]), slot_map, kp, vp)
    taken = int(used)
    assert taken == sum(-(-n // PAGE) for n in LENS)

    pool = torch.full((B + 2, H, D, D), float("nan"), device="cuda")
    slots = _i32([3, 0, 6, 2, 5])
    out = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    args = (pool, slots, cu, cat(q, prompt), cat(k, prompt), cat(v, prompt), cat(alpha, prompt))
    if rule == "delta":
        lib.fp32_delta_prefill(*args, cat(beta, prompt), out)
        st = lib.DampState(B + 2, H, D, synth.random_rows(np.random.default_rng(3), H, D, 24))
        st.quantize(pool[slots.long()].contiguous(), slots)
    else:
        lib.fp32_linear_prefill(*args, out)
    rec = [out[sum(LENS[:b]):sum(LENS[: b + 1])] for b in range(B)]
    steps, attn = [], []
    for t in range(STEPS):
        at = [slice(n + t, n + t + 1) for n in LENS]
        x = [cat(y, at) for y in (q, k, v, alpha)]
        y = torch.empty((B, H, D), device="cuda")
        if rule == "delta":
            lib.fp32_decode_step(pool, slots, *x, cat(beta, at), y)
            packed = torch.empty_like(y)
            st.decode_step(slots, *x, cat(beta, at), packed)
            # the packed state's readout stays near the exact state's (INT8 rows: a few percent)
            assert float((packed - y).norm() / y.norm()) < 0.1
        else:
            lib.fp32_linear_step(pool, slots, *x, y)
        steps.append(y)
        lib.kv_build_tables(_i32([n + t + 1 for n in LENS]), _i32([1] * B), free[taken:], table, PAGE, slot_map[:B], positions[:B], cu, used)
        taken += int(used)
        o = torch.empty((B, H, D), dtype=torch.bfloat16, device="cuda")
        lib.kv_decode_attention(cat(aq, at), kp, vp, table, _i32([n + t + 1 for n in LENS]), o, k_new=cat(ak, at), v_new=cat(av, at))
        attn.append(o)
        assert positions[:B].tolist() == [n + t for n in LENS]
    torch.cuda.synchronize()
    assert taken == sum(-(-n // PAGE) for n in total)

    for b in range(B):
        n = LENS[b]
        kappa = 1.0
        for h in range(H):
            z = [y[b][:, h].double() for y in (q, k, v)]
            o, S, mag, A, top = ref.prompt(torch.zeros((D, D), dtype=torch.float64), *z, alpha[b][:, h].double(),
                                           beta[b][:, h].double() if rule == "delta" else None)
            if rule == "delta":
                kappa = ref.chunk_condition(z[1], alpha[b][:, h].double(), beta[b][:, h].double())
            # the bounds of test_gpu_linear.py, with the steps' roundings (d + 8 a token) added
            e_col = ((2 * D + 156) * (-(-n // 64)) * kappa + STEPS * (D + 8)) * ref.EPS32 * (top if rule == "delta" else A.norm(dim=0))
            err = (pool[slots[b], h].double().cpu() - S).norm(dim=0)
            assert bool((err <= e_col + (512 * ref.EPS32 * A.norm(dim=0) if rule == "linear" else 0)).all())
            qn = z[0].norm(dim=-1, keepdim=True)
            inner = qn * (e_col + 2.0 ** -15 * kappa * top) + (0 if rule == "delta" else 2.0 ** -15 * mag)
            ref.is_close(rec[b][:, h], o[:n], 2.0 ** -8 * o[:n].abs() + inner[:n], f"prompt readouts {b} {h}")
            got = torch.stack([s[b, h] for s in steps])
            ref.is_close(got, o[n:], inner[n:], f"step readouts {b} {h}")
        for t in range(STEPS):
            m = n + t + 1
            kk, vv = ak[b][:m].double(), av[b][:m].double()
            o, mag = ref.attention(aq[b][m - 1].double(), kk, vv, D ** -0.5)
            e = ref.score_error(aq[b][m - 1].double(), kk, D ** -0.5) + 2.0 ** -8 + 70 * ref.EPS32
            ref.is_close(attn[t][b], o, 2.0 ** -8 * o.abs() + 2 * e * mag, f"attention {b} after {t} tokens")
    # pages of no request were never written
    idle = [i for i in range(pages) if i not in free[:taken].tolist()]
    assert bool(kp[idle].isnan().all()) and bool(vp[idle].isnan().all())


def test_many_shapes_against_the_token_form():
    """Random ragged batches: the chunked forms against the token-by-token form of the same call (fp32 copies of
    the same bf16 values), which shares no code with them past the entry point."""
    rng = np.random.default_rng(77)
    for case in range(40):
        d = int(rng.choice([64, 128]))
        h = int(rng.integers(1, 9))
        B = int(rng.integers(1, 7))
        lens = [int(x) for x in np.exp(rng.uniform(0, 6.5, B)).astype(int) * (rng.random(B) < 0.9)]
        T = sum(lens)
        if T == 0:
            continue
        gen = torch.Generator(device="cuda").manual_seed(case)
        q, k = (torch.nn.functional.normalize(torch.randn((T, h, d), generator=gen, device="cuda"), dim=-1).bfloat16() for _ in range(2))
        v = torch.randn((T, h, d), generator=gen, device="cuda").bfloat16()
        alpha = torch.exp2(-torch.rand((T, h), generator=gen, device="cuda") * 2.0 ** float(rng.uniform(-10, 1)))
        beta = torch.rand((T, h), generator=gen, device="cuda")
        start = torch.randn((B + 1, h, d, d), generator=gen, device="cuda")
        slots = torch.from_numpy(rng.permutation(B + 1)[:B].astype(np.int32)).cuda()
        cu = _i32([0] + [int(x) for x in np.cumsum(lens)])
        resume = torch.from_numpy(rng.integers(0, 2, B).astype(np.int32)).cuda()
        for delta in (False, True):
            got = []
            for t in (torch.bfloat16, torch.float32):
                pool, out = start.clone(), torch.zeros((T, h, d), dtype=t, device="cuda")
                x = (pool, slots, cu, q.to(t), k.to(t), v.to(t), alpha)
                if delta:
                    lib.fp32_delta_prefill(*x, beta, out, resume=resume)
                else:
                    lib.fp32_linear_prefill(*x, out, resume=resume)
                got.append((pool, out.float()))
            what = f"case {case}: d {d}, heads {h}, lengths {lens}, delta {delta}"
            # two binary32 evaluations: each within (roundings of a chunk) * 2^-24 of the true state per chunk or token
            # of the chain (test_gpu_linear.py), in the norm of the whole; readouts differ by their rounding to bf16
            chain = max(lens)
            tol = 2 ** -24 * (512 + 16 * chain)
            assert float((got[0][0] - got[1][0]).norm() / got[1][0].norm()) <= tol, what
            assert float((got[0][1] - got[1][1]).norm() / got[1][1].norm()) <= 2.0 ** -8 + tol, what
