"""Cases and plain forms of the operators for serving hybrid models: the prompt forms of linear
attention with a decay for each head and of the gated delta rule, the single-token form of the
former, attention of one new token over a paged key-value cache, and the block tables and slot
maps that such a cache goes by.

``run`` computes the plain forms with elementary torch operations (``own`` false) or calls the
library (``own`` true) on what ``prepare`` made; ``exact`` follows the definitions in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64  # tokens per chunk of the plain prompt forms


def listed():
    """Prompts: short ones (a chat turn each), a ragged batch as continuous batching gives it, one
    long document. Steps: a few requests (latency) and a full pool. Attention: one request
    (latency), a large ragged batch, a few long contexts. Tables: a decode step's one page here
    and there, and a batch of prompts whose keys and values are then stored."""
    return [
        {"name": "linear prompts short", "op": "linear_prefill", "requests": 4, "tokens": 203, "heads": 8, "d": 64, "decay": "head", "resume": False},
        {"name": "linear prompts ragged", "op": "linear_prefill", "requests": 12, "tokens": 8191, "heads": 32, "d": 128, "decay": "token", "resume": True},
        {"name": "linear step few", "op": "linear_step", "requests": 3, "slots": 16, "heads": 32, "d": 128, "dtype": "bf16"},
        {"name": "linear step pool", "op": "linear_step", "requests": 1024, "slots": 1152, "heads": 32, "d": 128, "dtype": "bf16"},
        {"name": "delta prompts short", "op": "delta_prefill", "requests": 4, "tokens": 203, "heads": 8, "d": 64, "decay": "token", "resume": False},
        {"name": "delta prompts ragged", "op": "delta_prefill", "requests": 16, "tokens": 8191, "heads": 32, "d": 128, "decay": "token", "resume": True},
        {"name": "delta prompt long", "op": "delta_prefill", "requests": 1, "tokens": 16384, "heads": 32, "d": 128, "decay": "token", "resume": False},
        {"name": "attention one request", "op": "attention", "requests": 1, "longest": 700, "q_heads": 16, "kv_heads": 2, "d": 128, "page": 16},
        {"name": "attention batch", "op": "attention", "requests": 64, "longest": 8192, "q_heads": 32, "kv_heads": 8, "d": 128, "page": 16},
        {"name": "attention long", "op": "attention", "requests": 5, "longest": 65536, "q_heads": 32, "kv_heads": 4, "d": 64, "page": 64},
        {"name": "tables of a decode step", "op": "tables", "requests": 48, "tokens": 48, "cached": 4000, "page": 16, "kv_heads": 0, "d": 0},
        {"name": "tables and cache of prompts", "op": "tables", "requests": 300, "tokens": 32000, "cached": 0, "page": 32, "kv_heads": 8, "d": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_prefill", "linear_step", "delta_prefill", "attention", "tables"])
    d = rng.choice([64, 128])
    if op == "linear_prefill" or op == "delta_prefill":
        heads = rng.randint(1, 40)
        most = 8192 * 32 * 128 // (heads * d)
        return {"op": op, "requests": _log(rng, 1, 24), "tokens": _log(rng, 1, min(16384, most)), "heads": heads, "d": d,
                "decay": rng.choice(["token", "token", "head"]) if op == "linear_prefill" else "token", "resume": rng.random() < 0.5}
    if op == "linear_step":
        heads = rng.randint(1, 40)
        n = _log(rng, 1, min(1024, 1024 * 32 // heads))
        return {"op": op, "requests": n, "slots": n + _log(rng, 1, 128), "heads": heads, "d": d, "dtype": rng.choice(["bf16", "fp32"])}
    if op == "attention":
        kv, group = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
        n = _log(rng, 1, 64)
        most = 64 * 8192 * 8 // (n * kv * 2)
        return {"op": op, "requests": n, "longest": _log(rng, 1, min(65536, most)), "q_heads": kv * group, "kv_heads": kv, "d": d,
                "page": rng.choice([16, 32, 64, 128])}
    n = _log(rng, 1, 1000)
    kv = rng.choice([0, 1, 3, 8])
    return {"op": op, "requests": n, "tokens": _log(rng, n, 32000), "cached": rng.choice([0, rng.randint(1, 64000 // n if kv else 8000)]), "page": rng.choice([16, 32, 64, 128]),
            "kv_heads": kv, "d": d if kv else 0}


def _spread(n, total, gen, least=0):
    """n lengths of a wide spread with the given sum, in an order of the generator's."""
    w = [math.exp(3.0 * i / max(1, n - 1)) for i in range(n)]
    got = [least + int((total - least * n) * x / sum(w)) for x in w]
    got[-1] += total - sum(got)
    order = torch.randperm(n, generator=gen).tolist()
    return [got[i] for i in order]


def _gates(shape, heads, gen, dev):
    """Decays whose half-lives run from 4 to 4,096 tokens over the heads."""
    life = torch.exp2(torch.linspace(2.0, 12.0, heads, device=dev)) if heads > 1 else torch.full((1,), 64.0, device=dev)
    if shape is None:
        return torch.exp2(-1.0 / life)
    return torch.exp2(-(0.5 + torch.rand(shape, generator=gen, device=dev)) / life)


def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def prepare(case, seed):
    dev = "cuda"
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    c, s = case, {"op": case["op"]}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if c["op"] in ("linear_prefill", "delta_prefill"):
        n, T, H, d = c["requests"], c["tokens"], c["heads"], c["d"]
        lens = _spread(n, T, cpu)
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
        s["cu"], s["longest"] = cu.to(dev, torch.int32), max(lens)
        s["q"], s["k"] = _unit(normal(T, H, d)).bfloat16(), _unit(normal(T, H, d)).bfloat16()
        s["v"] = normal(T, H, d).bfloat16()
        s["alpha"] = _gates(None if c["decay"] == "head" else (T, H), H, gen, dev)
        s["beta"] = torch.sigmoid(normal(T, H))
        slots = torch.randperm(n + 3, generator=cpu)[:n]
        s["slots"] = slots.to(dev, torch.int32)
        s["pool"] = 0.1 * normal(n + 3, H, d, d)
        s["resume"] = torch.randint(0, 2, (n,), generator=cpu, dtype=torch.int32).to(dev) if c["resume"] else None
        s["out"] = torch.zeros((T, H, d), dtype=torch.bfloat16, device=dev)
    elif c["op"] == "linear_step":
        n, H, d = c["requests"], c["heads"], c["d"]
        t = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["q"], s["k"], s["v"] = _unit(normal(n, H, d)).to(t), _unit(normal(n, H, d)).to(t), normal(n, H, d).to(t)
        s["alpha"] = _gates((n, H), H, gen, dev)
        s["slots"] = torch.randperm(c["slots"], generator=cpu)[:n].to(dev, torch.int32)
        s["pool"] = normal(c["slots"], H, d, d)
        s["out"] = torch.empty((n, H, d), device=dev)
    elif c["op"] == "attention":
        n, page, Hq, Hk, d = c["requests"], c["page"], c["q_heads"], c["kv_heads"], c["d"]
        most = c["longest"]
        # lengths spread evenly from one token to the longest
        lens = torch.tensor([max(1, most * (i + 1) // n) for i in range(n)])[torch.randperm(n, generator=cpu)]
        blocks = -(-most // page)
        used = -(-lens // page)
        pages = int(used.sum()) + 5
        ids = torch.randperm(pages, generator=cpu)
        first = used.cumsum(0) - used
        at = first[:, None] + torch.arange(blocks)
        table = torch.where(torch.arange(blocks) < used[:, None], ids[at.clamp(max=pages - 1)], torch.tensor(-1))
        s["table"], s["lens"] = table.to(dev, torch.int32), lens.to(dev, torch.int32)
        s["longest"], s["scale"] = most, d ** -0.5
        s["kp"] = torch.empty((pages, Hk, page, d), dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        s["vp"] = torch.empty((pages, Hk, page, d), dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        s["q"] = (2.0 * normal(n, Hq, d)).bfloat16()
        s["k_new"], s["v_new"] = normal(n, Hk, d).bfloat16(), normal(n, Hk, d).bfloat16()
        s["out"] = torch.empty((n, Hq, d), dtype=torch.bfloat16, device=dev)
    else:
        n, T, page = c["requests"], c["tokens"], c["page"]
        new = torch.tensor(_spread(n, T, cpu, 1))
        old = torch.randint(0, c["cached"] + 1, (n,), generator=cpu)
        total = old + new
        have = -(-old // page)
        most = -(-(c["cached"] + new) // page)
        blocks, pages = int(most.max()) + 2, int(most.sum()) + 7
        ids = torch.randperm(pages, generator=cpu)
        first = have.cumsum(0) - have
        at = first[:, None] + torch.arange(blocks)
        table = torch.where(torch.arange(blocks) < have[:, None], ids[at.clamp(max=pages - 1)], torch.tensor(-1))
        s["free"] = ids[int(have.sum()):].to(dev, torch.int32)
        s["table"], s["page"] = table.to(dev, torch.int32), page
        s["lens"], s["new"] = total.to(dev, torch.int32), new.to(dev, torch.int32)
        s["slot_map"] = torch.empty(T + 3, dtype=torch.int64, device=dev)  # a padded batch: three rows behind the last token
        s["positions"] = torch.empty(T + 3, dtype=torch.int32, device=dev)
        s["cu"] = torch.empty(n + 1, dtype=torch.int32, device=dev)
        s["used"] = torch.empty(1, dtype=torch.int32, device=dev)
        s["k"] = None
        if c["kv_heads"]:
            s["k"], s["v"] = normal(T + 3, c["kv_heads"], c["d"]).bfloat16(), normal(T + 3, c["kv_heads"], c["d"]).bfloat16()
            s["kp"] = torch.zeros((pages, c["kv_heads"], page, c["d"]), dtype=torch.bfloat16, device=dev)
            s["vp"] = torch.zeros_like(s["kp"])
    return s


# ---- plain forms ----------------------------------------------------------------------------
def _padded(s):
    """Row numbers of each request's tokens [requests, chunks * CHUNK], and which of them are tokens."""
    cu = s["cu"].long()
    rows = max(1, -(-s["longest"] // CHUNK)) * CHUNK
    at = torch.arange(rows, device=cu.device)
    live = at < (cu[1:] - cu[:-1])[:, None]
    return torch.where(live, cu[:-1, None] + at, torch.zeros_like(cu[:-1, None])), live


def _chunks(x, idx, live, fill=0.0):
    """x [T, H, ...] as float32 [requests, H, chunks, CHUNK, ...], padding rows `fill`."""
    y = x.float()[idx]
    y = torch.where(live.reshape(live.shape + (1,) * (y.dim() - 2)), y, torch.full_like(y, fill))
    y = y.transpose(1, 2)
    return y.reshape(y.shape[0], y.shape[1], -1, CHUNK, *y.shape[3:]).contiguous()


def _start_state(s):
    S0 = s["pool"][s["slots"].long()]
    return torch.zeros_like(S0) if s["resume"] is None else torch.where(s["resume"][:, None, None, None] != 0, S0, torch.zeros_like(S0))


def _finish(s, idx, live, o, S):
    """Stores the readouts [requests, H, rows, d] and the states; a request of no tokens keeps its state."""
    s["out"][idx[live]] = o.transpose(1, 2)[live].to(s["out"].dtype)
    slots = s["slots"].long()
    s["pool"][slots] = torch.where(live[:, 0, None, None, None], S, s["pool"][slots])
    return {"out": s["out"], "pool": s["pool"]}


def _decays(G):
    """exp of G_t - G_s over t >= s for running sums G [..., n] of logarithms (float64), as float32."""
    diff = G[..., :, None] - G[..., None, :]
    n = G.shape[-1]
    lower = torch.ones((n, n), dtype=torch.bool, device=G.device).tril()
    return torch.where(lower, diff, torch.full_like(diff, -math.inf)).exp().float()


def _log_alpha(s, idx, live):
    a = s["alpha"]
    T, H = s["q"].shape[:2]
    return _chunks(a.expand(T, H) if a.dim() == 1 else a, idx, live, 1.0).double().log()


def _plain_linear_prefill(s):
    idx, live = _padded(s)
    q, k, v = (_chunks(s[x], idx, live) for x in "qkv")
    G = _log_alpha(s, idx, live).cumsum(-1)
    P = torch.matmul(q, k.transpose(-1, -2).contiguous()) * _decays(G)
    kw = k * (G[..., -1:] - G).exp().float()[..., None]
    own_state = torch.matmul(kw.transpose(-1, -2).contiguous(), v)          # what each chunk adds
    S0 = _start_state(s)
    all_states = torch.cat([S0[:, :, None], own_state], 2)                  # [requests, H, 1 + chunks, d, d]
    ends = torch.cat([torch.zeros_like(G[..., 0, -1:]), G[..., -1].cumsum(-1)], -1)
    n = all_states.shape[2]
    mixed = torch.matmul(_decays(ends), all_states.flatten(3)).reshape(all_states.shape)
    o = torch.matmul(P, v) + torch.matmul(q * G.exp().float()[..., None], mixed[:, :, : n - 1])
    return _finish(s, idx, live, o.flatten(2, 3), mixed[:, :, n - 1])


def _plain_linear_step(s):
    slots = s["slots"].long()
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    S = s["pool"][slots] * s["alpha"][..., None, None] + k[..., :, None] * v[..., None, :]
    s["pool"][slots] = S
    s["out"].copy_((S * q[..., :, None]).sum(-2))
    return {"out": s["out"], "pool": s["pool"]}


def _inverse(A):
    """(I + A)^-1 for strictly lower triangular A [..., n, n], n a power of two: the diagonal blocks'
    inverses are joined two by two, [[X, 0], [Y, Z]]^-1 = [[X', 0], [-Z' Y X', Z']]."""
    n = A.shape[-1]
    X = torch.ones(A.shape[:-2] + (n, 1, 1), dtype=A.dtype, device=A.device)
    m = 1
    while m < n:
        blocks = A.reshape(A.shape[:-2] + (n // (2 * m), 2 * m, n // (2 * m), 2 * m)).diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
        Y = blocks[..., m:, :m]
        X, Z = X[..., 0::2, :, :], X[..., 1::2, :, :]
        low = -torch.matmul(torch.matmul(Z.contiguous(), Y.contiguous()), X.contiguous())
        X = torch.cat([torch.cat([X, torch.zeros_like(X)], -1), torch.cat([low, Z], -1)], -2)
        m *= 2
    return X[..., 0, :, :]


def _plain_delta_prefill(s):
    idx, live = _padded(s)
    q, k, v = (_chunks(s[x], idx, live) for x in "qkv")
    beta = _chunks(s["beta"], idx, live)
    G = _log_alpha(s, idx, live).cumsum(-1)
    D = _decays(G)
    kt = k.transpose(-1, -2).contiguous()
    A = (torch.matmul(k, kt) * D * beta[..., None]).tril(-1)
    P = torch.matmul(q, kt) * D
    X = _inverse(A)
    eG = G.exp().float()[..., None]
    U = torch.matmul(X, v * beta[..., None])
    W = torch.matmul(X, k * (eG * beta[..., None]))
    qe = q * eG
    kw = kt * (G[..., -1:] - G).exp().float()[..., None, :]
    last = eG[..., -1:, :]
    S, o = _start_state(s), torch.empty_like(q)
    for c in range(q.shape[2]):  # the state goes from chunk to chunk
        delta = U[:, :, c] - torch.matmul(W[:, :, c], S)
        o[:, :, c] = torch.matmul(qe[:, :, c], S) + torch.matmul(P[:, :, c], delta)
        S = S * last[:, :, c] + torch.matmul(kw[:, :, c], delta)
    return _finish(s, idx, live, o.flatten(2, 3), S)


def _plain_attention(s):
    page, d = s["kp"].shape[2], s["kp"].shape[3]
    n, Hk = s["k_new"].shape[:2]
    lens, table = s["lens"].long(), s["table"].long()
    at = (lens - 1).clamp(min=0)
    to = table.gather(1, (at // page)[:, None])[:, 0]
    s["kp"][to, :, at % page] = s["k_new"]
    s["vp"][to, :, at % page] = s["v_new"]
    rows = table.shape[1] * page
    live = torch.arange(rows, device=lens.device) < lens[:, None]
    ids = table.clamp(min=0)
    k = s["kp"][ids].transpose(1, 2).reshape(n, Hk, rows, d).float()
    q = s["q"].float().reshape(n, Hk, -1, d) * s["scale"]
    x = torch.matmul(q, k.transpose(-1, -2).contiguous())
    del k
    x = torch.where(live[:, None, None], x, torch.full_like(x, -math.inf))
    p = (x - x.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    v = s["vp"][ids].transpose(1, 2).reshape(n, Hk, rows, d).float()
    v = torch.where(live[:, None, :, None], v, torch.zeros_like(v))
    s["out"].copy_(torch.matmul(p, v).reshape(s["out"].shape))
    return {"out": s["out"], "k_pages": s["kp"], "v_pages": s["vp"]}


def _plain_tables(s):
    page, table, free = s["page"], s["table"].long(), s["free"].long()
    lens, new = s["lens"].long(), s["new"].long()
    old = lens - new
    have = (old + page - 1) // page
    need = (lens + page - 1) // page - have
    first = need.cumsum(0) - need
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    j = torch.arange(table.shape[1], device=table.device)
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None])
    at = (first - have)[:, None] + j
    table = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table)
    t = torch.arange(s["slot_map"].numel(), device=table.device)
    live = t < cu[-1]
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=new.numel() - 1)
    pos = torch.where(live, old[b] + t - cu[b], torch.zeros_like(t))
    slots = table[b, pos // page] * page + pos % page
    s["table"].copy_(table)
    s["slot_map"].copy_(torch.where(live, slots, torch.full_like(slots, -1)))
    s["positions"].copy_(torch.where(live, pos, torch.full_like(pos, -1)))
    s["cu"].copy_(cu)
    s["used"].copy_(need.sum(0, keepdim=True))
    got = {x: s[x] for x in ("table", "slot_map", "positions", "cu", "used")}
    if s["k"] is not None:
        row = t[: t.numel() - 3]
        to = s["slot_map"][row]
        s["kp"][to // page, :, to % page] = s["k"][row]
        s["vp"][to // page, :, to % page] = s["v"][row]
        got |= {"k_pages": s["kp"], "v_pages": s["vp"]}
    return got


# ---- the library's calls --------------------------------------------------------------------
def _own(s):
    from quantized_delta_rule_gdn_amd import lib
    if s["op"] == "linear_prefill":
        lib.fp32_linear_prefill(s["pool"], s["slots"], s["cu"], s["q"], s["k"], s["v"], s["alpha"], s["out"], resume=s["resume"])
        return {"out": s["out"], "pool": s["pool"]}
    if s["op"] == "delta_prefill":
        lib.fp32_delta_prefill(s["pool"], s["slots"], s["cu"], s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["out"], resume=s["resume"])
        return {"out": s["out"], "pool": s["pool"]}
    if s["op"] == "linear_step":
        lib.fp32_linear_step(s["pool"], s["slots"], s["q"], s["k"], s["v"], s["alpha"], s["out"])
        return {"out": s["out"], "pool": s["pool"]}
    if s["op"] == "attention":
        lib.kv_decode_attention(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["out"], scale=s["scale"], k_new=s["k_new"], v_new=s["v_new"],
                                max_len=s["longest"])
        return {"out": s["out"], "k_pages": s["kp"], "v_pages": s["vp"]}
    lib.kv_build_tables(s["lens"], s["new"], s["free"], s["table"], s["page"], s["slot_map"], s["positions"], s["cu"], s["used"])
    got = {x: s[x] for x in ("table", "slot_map", "positions", "cu", "used")}
    if s["k"] is not None:
        lib.kv_append(s["k"], s["v"], s["slot_map"], s["kp"], s["vp"])
        got |= {"k_pages": s["kp"], "v_pages": s["vp"]}
    return got


def run(state):
    if own:
        return _own(state)
    return {"linear_prefill": _plain_linear_prefill, "linear_step": _plain_linear_step, "delta_prefill": _plain_delta_prefill,
            "attention": _plain_attention, "tables": _plain_tables}[state["op"]](state)


def work(case):
    c = case
    if c["op"] in ("linear_prefill", "delta_prefill"):
        n, T, H, d = c["requests"], c["tokens"], c["heads"], c["d"]
        delta = c["op"] == "delta_prefill"
        # q, k, v in and out, the gates, each request's state written (about half read where some resume);
        # per token: the update and the readout of a d x d state, and for the delta rule its projection
        return {"bytes": 8 * T * H * d + 4 * T * H * (2 if delta else 1 if c["decay"] == "token" else 0) + n * H * d * d * (6 if c["resume"] else 4),
                "flops": (6 if delta else 4) * T * H * d * d}
    if c["op"] == "linear_step":
        n, H, d = c["requests"], c["heads"], c["d"]
        return {"bytes": n * H * (8 * d * d + 3 * d * (2 if c["dtype"] == "bf16" else 4) + 4 * d + 4), "flops": 5 * n * H * d * d}
    if c["op"] == "attention":
        n, most = c["requests"], c["longest"]
        tokens = sum(max(1, most * (i + 1) // n) for i in range(n))
        Hq, Hk, d = c["q_heads"], c["kv_heads"], c["d"]
        return {"bytes": 4 * tokens * Hk * d + 4 * n * Hq * d + 8 * n * Hk * d, "flops": 4 * tokens * Hq * d}
    T, n = c["tokens"], c["requests"]
    fresh = T // c["page"] + 1
    return {"bytes": 12 * T + 12 * n + 8 * fresh + 8 * T * c["kv_heads"] * c["d"], "flops": 0}


# ---- the definitions in 64 bits -------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("linear_prefill", "delta_prefill"):
        return _exact_prompts(s, case["op"] == "delta_prefill")
    if case["op"] == "linear_step":
        pool, out = s["pool"].double(), torch.empty_like(s["out"], dtype=torch.float64)
        for i, slot in enumerate(s["slots"].tolist()):
            S = s["alpha"][i].double()[:, None, None] * pool[slot] + s["k"][i].double()[:, :, None] * s["v"][i].double()[:, None, :]
            pool[slot] = S
            out[i] = torch.matmul(s["q"][i].double()[:, None, :], S)[:, 0]
        return {"out": out, "pool": pool}
    if case["op"] == "attention":
        return _exact_attention(s)
    return _exact_tables(s)


def _exact_prompts(s, delta):
    """Token by token: S <- a S, then S <- S + k e^T with e = v, or beta (v - S^T k) for the delta rule; o = S^T q."""
    cu = s["cu"].tolist()
    T, H, d = s["q"].shape
    pool, out = s["pool"].double(), torch.zeros((T, H, d), dtype=torch.float64, device="cuda")
    # longest first: at token t the requests still running are the first ones
    order = sorted(range(len(cu) - 1), key=lambda b: cu[b] - cu[b + 1])
    lens = [cu[b + 1] - cu[b] for b in order]
    slots = s["slots"].long()[torch.tensor(order, device="cuda")]
    S = pool[slots]
    if s["resume"] is None:
        S.zero_()
    else:
        S[s["resume"][torch.tensor(order, device="cuda")] == 0] = 0.0
    begin = torch.tensor([cu[b] for b in order], device="cuda")
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    a = s["alpha"].double()
    n = len(order)
    for t in range(lens[0]):
        while lens[n - 1] <= t:
            n -= 1
        rows, X = begin[:n] + t, S[:n]
        X *= (a if a.dim() == 1 else a[rows])[..., None, None]
        kt, e = k[rows], v[rows]
        if delta:
            e = s["beta"][rows].double()[..., None] * (e - torch.matmul(kt[..., None, :], X)[..., 0, :])
        X += kt[..., :, None] * e[..., None, :]
        out[rows] = torch.matmul(q[rows][..., None, :], X)[..., 0, :]
    some = torch.tensor([x > 0 for x in lens], device="cuda")
    pool[slots[some]] = S[some]
    return {"out": out, "pool": pool}


def _exact_attention(s):
    page, d = s["kp"].shape[2:]
    n, Hq = s["q"].shape[:2]
    Hk = s["k_new"].shape[1]
    out = torch.zeros((n, Hq, d), dtype=torch.float64, device="cuda")
    kp, vp = s["kp"].clone(), s["vp"].clone()
    for b, m in enumerate(s["lens"].tolist()):
        at = torch.arange(m, device="cuda")
        ids, off = s["table"][b].long()[at // page], at % page
        kp[ids[m - 1], :, off[m - 1]] = s["k_new"][b]
        vp[ids[m - 1], :, off[m - 1]] = s["v_new"][b]
        k, v = kp[ids, :, off].double(), vp[ids, :, off].double()           # [m, Hk, d]
        q = s["q"][b].double().reshape(Hk, Hq // Hk, d)
        p = torch.softmax(torch.matmul(q, k.permute(1, 2, 0).contiguous()) * s["scale"], -1)
        out[b] = torch.matmul(p, v.transpose(0, 1).contiguous()).reshape(Hq, d)
    return {"out": out, "k_pages": None, "v_pages": None}


def _exact_tables(s):
    """Request by request, in lists: pages that are missing come from the free list in order."""
    page, table, free = s["page"], s["table"].tolist(), s["free"].tolist()
    slots, positions, cu, used = [], [], [0], 0
    for b, (total, new) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        for i in range(-(-(total - new) // page), -(-total // page)):
            table[b][i] = free[used]
            used += 1
        for pos in range(total - new, total):
            slots.append(table[b][pos // page] * page + pos % page)
            positions.append(pos)
        cu.append(cu[-1] + new)
    rest = [-1] * (s["slot_map"].numel() - len(slots))
    got = {"table": torch.tensor(table), "slot_map": torch.tensor(slots + rest), "positions": torch.tensor(positions + rest),
           "cu": torch.tensor(cu), "used": torch.tensor([used])}
    if s["k"] is not None:
        for x, y in (("k_pages", "k"), ("v_pages", "v")):
            pages = torch.zeros(s["kp"].shape, dtype=torch.float64, device="cuda").transpose(1, 2).contiguous()
            pages.view(-1, *pages.shape[2:])[torch.tensor(slots, device="cuda")] = s[y][: len(slots)].double()
            got[x] = pages.transpose(1, 2)
    return got
