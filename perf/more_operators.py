"""Cases and plain forms of the operators that a paged cache needs once requests draft tokens, share
pages and keep latents: attention of a tree of drafted tokens, forked tables with copied pages, kept
tokens moved together with pages given back, and latent attention in its absorbed and expanded forms.

``run`` computes the plain forms with elementary torch operations (``own`` false) or calls the
library (``own`` true) on what ``prepare`` made; ``exact`` follows the definitions in 64 bits.
"""
import math

import torch

own = False


def listed():
    """Tree: one request's short draft (latency), a batch that drafts 32 tokens each at the widest, a
    few long contexts with 64 drafted tokens. Fork: a handful of requests sampled several times, beams
    of a large batch. Keep: the accepted drafts of a few requests, of a large batch, and tokens
    dropped from long caches. Latent: one request (latency), a large ragged batch with the heads of one
    device of eight, all heads with drafted tokens. Latent prompts: short ones, ragged ones of which
    some go on from cached tokens."""
    return [
        {"name": "tree one request", "op": "tree", "requests": 1, "longest": 900, "drafted": 8, "q_heads": 16, "kv_heads": 2, "d": 128, "page": 16},
        {"name": "tree batch", "op": "tree", "requests": 48, "longest": 4096, "drafted": 32, "q_heads": 32, "kv_heads": 8, "d": 128, "page": 16},
        {"name": "tree long", "op": "tree", "requests": 4, "longest": 65536, "drafted": 64, "q_heads": 32, "kv_heads": 4, "d": 64, "page": 64},
        {"name": "fork samples", "op": "fork", "parents": 6, "children": 3, "longest": 1000, "page": 16, "kv_heads": 8, "d": 128},
        {"name": "fork beams", "op": "fork", "parents": 192, "children": 3, "longest": 2048, "page": 128, "kv_heads": 8, "d": 128},
        {"name": "keep drafts few", "op": "keep", "requests": 5, "longest": 1000, "drafted": 12, "page": 16, "kv_heads": 8, "d": 128},
        {"name": "keep of long caches", "op": "keep", "requests": 32, "longest": 8192, "drafted": 0, "page": 16, "kv_heads": 8, "d": 128},
        {"name": "latent one request", "op": "latent", "requests": 1, "longest": 700, "drafted": 1, "heads": 16, "dc": 512, "page": 64},
        {"name": "latent batch", "op": "latent", "requests": 64, "longest": 8192, "drafted": 1, "heads": 16, "dc": 512, "page": 64},
        {"name": "latent all heads", "op": "latent", "requests": 24, "longest": 4096, "drafted": 4, "heads": 128, "dc": 512, "page": 64},
        {"name": "latent prompts short", "op": "prompt", "requests": 4, "tokens": 203, "cached": 0, "heads": 8, "d": 64},
        {"name": "latent prompts ragged", "op": "prompt", "requests": 8, "tokens": 12288, "cached": 1024, "heads": 16, "d": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "fork", "keep", "latent", "prompt"])
    d = rng.choice([64, 128])
    if op == "tree":
        kv, group = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
        n, drafted = _log(rng, 1, 64), _log(rng, 1, 150)
        most = 48 * 4096 * 32 * 128 * 32 // (n * kv * group * 128 * max(drafted, 256 // group))
        return {"op": op, "requests": n, "longest": _log(rng, 1, max(1, min(65536, most))), "drafted": drafted, "q_heads": kv * group, "kv_heads": kv, "d": d,
                "page": rng.choice([16, 32, 64, 128])}
    if op == "fork":
        parents, children = _log(rng, 1, 400), rng.randint(1, 4)
        page = rng.choice([16, 32, 64, 128])
        if parents * children * page > 192 * 3 * 128:
            page = 16
        return {"op": op, "parents": parents, "children": children, "longest": _log(rng, 1, 4096), "page": page, "kv_heads": rng.randint(1, 8), "d": d}
    if op == "keep":
        n, drafted = _log(rng, 1, 512), rng.choice([0, _log(rng, 1, 64)])
        most = 32 * 8192 // n
        return {"op": op, "requests": n, "longest": _log(rng, 1, max(1, min(16384, most))), "drafted": drafted, "page": rng.choice([16, 32, 64, 128]),
                "kv_heads": rng.randint(1, 8), "d": d}
    if op == "latent":
        n, heads, drafted = _log(rng, 1, 64), rng.choice([1, 5, 8, 16, 20, 32, 64, 128]), rng.choice([1, 1, _log(rng, 1, 70)])
        most = min(64 * 8192 // n, 24 * 4096 * 4 * 128 // (n * heads * drafted))
        return {"op": op, "requests": n, "longest": _log(rng, 1, max(1, min(65536, most))), "drafted": drafted, "heads": heads, "dc": rng.choice([256, 512]),
                "page": rng.choice([16, 64, 128])}
    n, heads = _log(rng, 1, 16), rng.randint(1, 16)
    return {"op": op, "requests": n, "tokens": _log(rng, n, 12288 if n >= 8 else 4096 * n // 4 + 2048), "cached": rng.choice([0, _log(rng, 1, 1024)]), "heads": heads, "d": d}


def _spread(n, total, gen, least=1):
    """n lengths of a wide spread with the given sum, in an order of the generator's."""
    w = [math.exp(2.0 * i / max(1, n - 1)) for i in range(n)]
    got = [least + int((total - least * n) * x / sum(w)) for x in w]
    got[-1] += total - sum(got)
    order = torch.randperm(n, generator=gen).tolist()
    return [got[i] for i in order]


def _ladder(n, most):
    """Lengths spread evenly from one token to the longest."""
    return [max(1, most * (i + 1) // n) for i in range(n)]


def _drafts(c):
    """Drafted tokens of each request: the most for every second one, fewer for the others; never more than its tokens."""
    lens = _ladder(c["requests"], c["longest"])
    return lens, [min(x, c["drafted"] if i % 2 == 0 else max(1, c["drafted"] * (i % 7 + 1) // 8)) for i, x in enumerate(lens)]


def _tables(lens, page, spare, gen):
    """A block table over pages in random order: [requests, blocks] (-1 behind a request's pages), the other pages, and how many there are."""
    used = -(-lens // page)
    blocks = max(1, int(used.max()))
    pages = int(used.sum()) + spare
    ids = torch.randperm(pages, generator=gen)
    first = used.cumsum(0) - used
    at = first[:, None] + torch.arange(blocks)
    table = torch.where(torch.arange(blocks) < used[:, None], ids[at.clamp(max=pages - 1)], torch.tensor(-1))
    return table, ids[int(used.sum()):], pages


def _trees(new, gen):
    """Which drafted tokens of its request a drafted token sees: itself and its ancestors in a random tree, as bits of 64-bit words [sum(new), words]."""
    n, most = len(new), max(new)
    words = -(-most // 64)
    # a token's parent is one of the few before it, or the last token of the context (-1)
    back = torch.randint(1, 5, (n, most), generator=gen)
    parent = (torch.arange(most) - back).clamp(min=-1)
    bits = torch.zeros((n, most, words), dtype=torch.int64)
    rows = torch.arange(n)
    for i in range(most):
        p = parent[:, i]
        bits[:, i] = torch.where((p >= 0)[:, None], bits[rows, p.clamp(min=0)], torch.zeros((n, words), dtype=torch.int64))
        bits[:, i, i // 64] |= -(1 << 63) if i % 64 == 63 else 1 << (i % 64)
    return torch.cat([bits[b, :m] for b, m in enumerate(new)])


def prepare(case, seed):
    dev = "cuda"
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    c, s = case, {"op": case["op"]}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def pages_of(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=gen)

    def ints(x):
        return torch.as_tensor(x).to(dev, torch.int32)

    if c["op"] in ("tree", "latent"):
        lens, new = _drafts(c)
        order = torch.randperm(c["requests"], generator=cpu).tolist()
        lens, new = [lens[i] for i in order], [new[i] for i in order]
        table, _, pages = _tables(torch.tensor(lens), c["page"], 5, cpu)
        s["table"], s["lens"], s["longest"], s["most"] = ints(table), ints(lens), c["longest"], max(new)
        T = sum(new)
        s["cu"] = ints(torch.tensor([0] + new).cumsum(0))
        s["mask"] = _trees(new, cpu).to(dev) if c["drafted"] > 1 else None
        if c["op"] == "tree":
            s["scale"] = c["d"] ** -0.5
            s["kp"], s["vp"] = pages_of(pages, c["kv_heads"], c["page"], c["d"]), pages_of(pages, c["kv_heads"], c["page"], c["d"])
            s["q"] = (2.0 * normal(T, c["q_heads"], c["d"])).bfloat16()
            s["out"] = torch.empty_like(s["q"])
        else:
            dc, dr = c["dc"], c["dc"] // 8
            s["scale"] = (dc // 4 + dr) ** -0.5   # of the expanded heads' d + d / 2 channels
            s["kp"] = pages_of(pages, c["page"], dc + dr)
            s["q"] = normal(T, c["heads"], dc + dr).bfloat16()
            s["out"] = torch.empty((T, c["heads"], dc), dtype=torch.bfloat16, device=dev)
    elif c["op"] == "fork":
        n, k = c["parents"], c["children"]
        lens = torch.tensor(_ladder(n, c["longest"]))[torch.randperm(n, generator=cpu)]
        table, free, pages = _tables(lens, c["page"], n * k + 4, cpu)
        rows = torch.randperm(n * (k + 1), generator=cpu)                # parents and children lie anywhere in the batch
        whole = torch.full((n * (k + 1), table.shape[1] + 2), -1)
        whole[rows[:n], : table.shape[1]] = table
        all_lens = torch.zeros(n * (k + 1), dtype=torch.int64)
        all_lens[rows[:n]] = lens
        s["table"], s["lens"], s["page"], s["free"] = ints(whole), ints(all_lens), c["page"], ints(free)
        s["src"], s["dst"] = ints(rows[:n].repeat_interleave(k)), ints(rows[n:])
        s["shares"] = torch.zeros(pages, dtype=torch.int32, device=dev)
        s["copy_src"], s["copy_dst"], s["copy_rows"] = (torch.empty(n * k, dtype=torch.int32, device=dev) for _ in range(3))
        s["used"] = torch.empty(1, dtype=torch.int32, device=dev)
        s["kp"], s["vp"] = (pages_of(pages, c["kv_heads"], c["page"], c["d"]) for _ in range(2))
    elif c["op"] == "keep":
        n = c["requests"]
        lens = torch.tensor(_ladder(n, c["longest"]))[torch.randperm(n, generator=cpu)]
        table, _, pages = _tables(lens, c["page"], 5, cpu)
        new = lens.clamp(max=c["drafted"]) if c["drafted"] else lens     # drafted tokens, or the whole cache
        cu_new = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
        owner = torch.repeat_interleave(torch.arange(n), new)
        offset = torch.arange(int(cu_new[-1])) - cu_new[owner]
        stays = torch.rand(offset.shape, generator=cpu) < (0.3 if c["drafted"] else 0.5)
        counts = torch.zeros(n, dtype=torch.int64).index_add_(0, owner, stays.long())
        s["kept"], s["cu"] = ints(offset[stays]), ints(torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]))
        s["lens"], s["new"], s["table"], s["page"] = ints(lens), ints(new), ints(table), c["page"]
        s["out_lens"] = torch.empty(n, dtype=torch.int32, device=dev)
        s["shares"] = torch.zeros(pages, dtype=torch.int32, device=dev)
        s["freed"] = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        s["count"] = torch.empty(1, dtype=torch.int32, device=dev)
        s["kp"], s["vp"] = (pages_of(pages, c["kv_heads"], c["page"], c["d"]) for _ in range(2))
    else:
        n, T, H, d = c["requests"], c["tokens"], c["heads"], c["d"]
        dr = d // 2
        q_lens = _spread(n, T, cpu)
        before = [c["cached"] * (i % 3) // 2 for i in range(n)]         # none, half of it, or all
        k_lens = [a + b for a, b in zip(q_lens, before)]
        s["cu_q"], s["cu_k"] = (ints(torch.tensor([0] + x).cumsum(0)) for x in (q_lens, k_lens))
        s["longest_q"], s["longest_k"], s["scale"] = max(q_lens), max(k_lens), (d + dr) ** -0.5
        s["q"] = normal(T, H, d + dr).bfloat16()
        kv = normal(sum(k_lens), H, 2 * d).bfloat16()                    # as the up-projection of the latents leaves them
        s["k"], s["v"] = kv[..., :d], kv[..., d:]
        s["kr"] = normal(sum(k_lens), dr).bfloat16()
        s["out"] = torch.empty((T, H, d), dtype=torch.bfloat16, device=dev)
    return s


# ---- plain forms ----------------------------------------------------------------------------
def _softmax(x, live):
    """Softmax over the last axis of what is live; all zero where nothing is."""
    x = torch.where(live, x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    p = (x - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total)


def _padded(cu, most):
    """Row numbers of each request's tokens [requests, most], and which of them are tokens."""
    cu = cu.long()
    at = torch.arange(most, device=cu.device)
    live = at < (cu[1:] - cu[:-1])[:, None]
    return torch.where(live, cu[:-1, None] + at, torch.zeros_like(cu[:-1, None])), live


def _seen(s, idx, rows):
    """[requests, drafted, positions]: which positions of its request a drafted token sees."""
    lens = s["lens"].long()
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    at = torch.arange(rows, device=lens.device)
    rel = at - (lens - new)[:, None]                                     # of the drafted tokens: 0, 1, ...
    live = at < lens[:, None]
    if s["mask"] is None:
        drafted = rel[:, None] <= torch.arange(idx.shape[1], device=lens.device)[:, None]
    else:
        words = s["mask"][idx]                                           # [requests, drafted, words]
        w = (rel.clamp(min=0) // 64).clamp(max=words.shape[2] - 1)
        drafted = words.gather(2, w[:, None].expand(-1, words.shape[1], -1)) >> (rel.clamp(min=0) % 64)[:, None] & 1 == 1
    return live[:, None] & ((rel < 0)[:, None] | drafted)


def _plain_tree(s):
    page, d = s["kp"].shape[2:]
    T, Hq = s["q"].shape[:2]
    n, Hk = s["lens"].numel(), s["kp"].shape[1]
    idx, mine = _padded(s["cu"], s["most"])
    rows = s["table"].shape[1] * page
    ids = s["table"].long().clamp(min=0)
    q = s["q"].float()[idx].reshape(n, -1, Hk, Hq // Hk, d).permute(0, 2, 3, 1, 4).reshape(n, Hk, -1, d) * s["scale"]
    k = s["kp"][ids].transpose(1, 2).reshape(n, Hk, rows, d).float()
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()).reshape(n, Hq, -1, rows)
    del k
    p = _softmax(x, _seen(s, idx, rows)[:, None]).reshape(n, Hk, -1, rows)
    del x
    live = torch.arange(rows, device=p.device) < s["lens"][:, None]
    v = s["vp"][ids].transpose(1, 2).reshape(n, Hk, rows, d).float()
    v = torch.where(live[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p, v).reshape(n, Hq, -1, d).transpose(1, 2)
    s["out"][idx[mine]] = o[mine].to(s["out"].dtype)
    return s["out"]


def _plain_latent(s):
    page, width = s["kp"].shape[1:]
    T, H, dc = s["out"].shape
    n = s["lens"].numel()
    idx, mine = _padded(s["cu"], s["most"])
    rows = s["table"].shape[1] * page
    k = s["kp"][s["table"].long().clamp(min=0)].reshape(n, rows, width).float()
    live = torch.arange(rows, device=k.device) < s["lens"][:, None]
    k = torch.where(live[..., None], k, torch.zeros_like(k))
    q = s["q"].float()[idx].reshape(n, -1, width) * s["scale"]
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()).reshape(n, -1, H, rows)
    p = _softmax(x, _seen(s, idx, rows)[:, :, None]).reshape(n, -1, rows)
    o = torch.matmul(p, k[..., :dc].contiguous()).reshape(n, -1, H, dc)
    s["out"][idx[mine]] = o[mine].to(s["out"].dtype)
    return s["out"]


def _plain_prompt(s):
    H, d = s["v"].shape[1:]
    iq, mine = _padded(s["cu_q"], s["longest_q"])
    ik, live = _padded(s["cu_k"], s["longest_k"])
    before = (s["cu_k"][1:] - s["cu_k"][:-1] - s["cu_q"][1:] + s["cu_q"][:-1]).long()
    q = s["q"].float()[iq].transpose(1, 2).contiguous() * s["scale"]
    k = torch.cat([s["k"].float(), s["kr"].float()[:, None].expand(-1, H, -1)], -1)[ik]
    x = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous())
    del k
    seen = torch.arange(ik.shape[1], device=x.device) <= before[:, None, None] + torch.arange(iq.shape[1], device=x.device)[:, None]
    p = _softmax(x, (seen & live[:, None])[:, None])
    del x
    o = torch.matmul(p, s["v"].float()[ik].transpose(1, 2).contiguous()).transpose(1, 2)
    s["out"][iq[mine]] = o[mine].to(s["out"].dtype)
    return s["out"]


def _plain_fork(s):
    page, table, free = s["page"], s["table"].long(), s["free"].long()
    src, dst = s["src"].long(), s["dst"].long()
    lens = s["lens"].long()[src]
    part = lens % page
    need = (part > 0).long()
    at = need.cumsum(0) - need
    fresh = torch.where(need > 0, free[at.clamp(max=free.numel() - 1)], torch.full_like(at, -1))
    full = lens // page
    j = torch.arange(table.shape[1], device=table.device)
    rows = table[src]
    last = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    shared = j < full[:, None]
    mine = torch.where(shared, rows, torch.where((j == full[:, None]) & (need > 0)[:, None], fresh[:, None], table[dst]))
    s["shares"].index_add_(0, rows.clamp(min=0).flatten(), shared.flatten().int())
    s["table"][dst] = mine.int()
    s["lens"][dst] = lens.int()
    s["copy_src"].copy_(torch.where(need > 0, last, torch.full_like(last, -1)))
    s["copy_dst"].copy_(fresh)
    s["copy_rows"].copy_(part)
    s["used"].copy_(need.sum(0, keepdim=True))
    # the copies of one layer
    inner = torch.arange(page, device=table.device) < s["copy_rows"][:, None]
    i, r = (inner & (s["copy_dst"] >= 0)[:, None]).nonzero(as_tuple=True)
    a, b = s["copy_src"].long()[i], s["copy_dst"].long()[i]
    for x in ("kp", "vp"):
        s[x][b, :, r] = s[x][a, :, r]
    return {x: s[x] for x in ("table", "lens", "shares", "copy_src", "copy_dst", "copy_rows", "used", "kp", "vp")}


def _plain_keep(s):
    page, table = s["page"], s["table"].long()
    cu, lens = s["cu"].long(), s["lens"].long()
    base = lens - s["new"].long()
    t = torch.arange(s["kept"].numel(), device=table.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    old, new = base[b] + s["kept"].long(), base[b] + t - cu[b]
    old_page, new_page = table[b, old // page], table[b, new // page]
    for x in ("kp", "vp"):
        s[x][new_page, :, new % page] = s[x][old_page, :, old % page]
    s["out_lens"].copy_(base + cu[1:] - cu[:-1])
    # pages behind what is kept
    j = torch.arange(table.shape[1], device=table.device)
    gone = (j >= ((s["out_lens"].long() + page - 1) // page)[:, None]) & (j < ((lens + page - 1) // page)[:, None])
    drops = torch.zeros_like(s["shares"]).index_add_(0, table.clamp(min=0).flatten(), gone.flatten().int())
    released = drops > s["shares"]
    s["shares"].copy_((s["shares"] - drops).clamp(min=0))
    ids = released.nonzero()[:, 0]
    s["freed"][: ids.numel()] = ids.int()
    s["count"].copy_(released.sum(0, keepdim=True))
    return {x: s[x] for x in ("kp", "vp", "out_lens", "shares", "freed", "count")}


# ---- the library's calls --------------------------------------------------------------------
def _own(s):
    from quantized_delta_rule_gdn_amd import lib
    if s["op"] == "tree":
        lib.kv_tree_attention(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["cu"], s["out"], mask=s["mask"], max_new=s["most"], scale=s["scale"],
                              max_len=s["longest"])
        return s["out"]
    if s["op"] == "latent":
        lib.kv_latent_attention(s["q"], s["kp"], s["table"], s["lens"], s["out"], s["scale"], cu_new=s["cu"], mask=s["mask"], max_new=s["most"], max_len=s["longest"])
        return s["out"]
    if s["op"] == "prompt":
        lib.kv_latent_prompt_attention(s["q"], s["k"], s["kr"], s["v"], s["cu_q"], s["out"], cu_k=s["cu_k"], scale=s["scale"])
        return s["out"]
    if s["op"] == "fork":
        lib.kv_fork_tables(s["src"], s["dst"], s["lens"], s["free"], s["table"], s["shares"], s["page"], s["copy_src"], s["copy_dst"], s["copy_rows"], s["used"])
        lib.kv_copy_pages(s["copy_src"], s["copy_dst"], s["kp"], s["vp"], rows=s["copy_rows"])
        return {x: s[x] for x in ("table", "lens", "shares", "copy_src", "copy_dst", "copy_rows", "used", "kp", "vp")}
    lib.kv_compact(s["kept"], s["cu"], s["lens"], s["new"], s["table"], s["kp"], s["vp"], s["out_lens"])
    lib.kv_free_pages(s["out_lens"], s["lens"], s["table"], s["shares"], s["page"], s["freed"], s["count"])
    return {x: s[x] for x in ("kp", "vp", "out_lens", "shares", "freed", "count")}


def run(state):
    if own:
        return _own(state)
    return {"tree": _plain_tree, "latent": _plain_latent, "prompt": _plain_prompt, "fork": _plain_fork, "keep": _plain_keep}[state["op"]](state)


def work(case):
    c = case
    if c["op"] == "tree":
        lens, new = _drafts(c)
        T, Hq, Hk, d = sum(new), c["q_heads"], c["kv_heads"], c["d"]
        # the cache once, queries and readouts; every drafted token against its request's tokens
        return {"bytes": 4 * sum(lens) * Hk * d + 4 * T * Hq * d, "flops": 4 * Hq * d * sum(a * b for a, b in zip(lens, new))}
    if c["op"] == "latent":
        lens, new = _drafts(c)
        T, H, dc = sum(new), c["heads"], c["dc"]
        dr = dc // 8
        return {"bytes": 2 * sum(lens) * (dc + dr) + 2 * T * H * (2 * dc + dr), "flops": 2 * H * (2 * dc + dr) * sum(a * b for a, b in zip(lens, new))}
    if c["op"] == "prompt":
        n, T, H, d = c["requests"], c["tokens"], c["heads"], c["d"]
        q_lens = _spread(n, T, torch.Generator().manual_seed(0))
        before = [c["cached"] * (i % 3) // 2 for i in range(n)]
        keys = T + sum(before)
        pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(sorted(q_lens), before))
        return {"bytes": 2 * T * H * (2 * d + d // 2) + keys * (4 * H * d + d), "flops": 2 * H * (2 * d + d // 2) * pairs}
    lens = _ladder(c["parents"] if c["op"] == "fork" else c["requests"], c["longest"])
    row = 4 * c["kv_heads"] * c["d"]                                     # a token's key and value
    if c["op"] == "fork":
        k, page = c["children"], c["page"]
        return {"bytes": k * sum(2 * row * (x % page) + 8 * -(-x // page) + 24 for x in lens), "flops": 0}
    kept = sum(0.3 * min(x, c["drafted"]) if c["drafted"] else 0.5 * x for x in lens)
    return {"bytes": int(kept * (2 * row + 4)) + sum(16 + 4 * -(-x // c["page"]) for x in lens), "flops": 0}


# ---- the definitions in 64 bits -------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(s)
    if case["op"] in ("tree", "latent"):
        return _exact_cached(s, case["op"] == "latent")
    return (_exact_fork if case["op"] == "fork" else _exact_keep)(s)


def _attend(q, k, v, seen, scale):
    """q [heads, n, d], k [heads, m, d], v [heads, m, e] in 64 bits, seen [n, m] (every row sees something)."""
    x = torch.matmul(q, k.transpose(1, 2).contiguous()) * scale
    x.masked_fill_(~seen, -math.inf)
    return torch.matmul(torch.softmax(x, -1), v)


def _exact_cached(s, latent):
    """Request by request and key head by key head; a drafted token's row of `seen` from its bits."""
    cu, out = s["cu"].tolist(), torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    page = s["kp"].shape[1 if latent else 2]
    masks = None if s["mask"] is None else s["mask"].tolist()
    for b, m in enumerate(s["lens"].tolist()):
        n = cu[b + 1] - cu[b]
        at = torch.arange(m, device="cuda")
        ids, off = s["table"][b].long()[at // page], at % page
        own_bits = [[i >= j if masks is None else masks[cu[b] + i][j // 64] >> (j % 64) & 1 == 1 for j in range(n)] for i in range(n)]
        seen = torch.cat([torch.ones((n, m - n), dtype=torch.bool), torch.tensor(own_bits, dtype=torch.bool).reshape(n, n)], 1).cuda()
        q = s["q"][cu[b]:cu[b + 1]].double()                              # [n, Hq, width]
        if latent:
            k = s["kp"][ids, off].double()[None]
            got = _attend(q.reshape(1, -1, q.shape[2]), k, k[..., : out.shape[2]].contiguous(), seen.repeat_interleave(q.shape[1], 0), s["scale"])
            out[cu[b]:cu[b + 1]] = got.reshape(n, q.shape[1], -1)
            continue
        group = q.shape[1] // s["kp"].shape[1]
        for h in range(s["kp"].shape[1]):
            k, v = (s[x][ids, h, off].double()[None].expand(group, -1, -1).contiguous() for x in ("kp", "vp"))
            got = _attend(q[:, h * group:(h + 1) * group].transpose(0, 1).contiguous(), k, v, seen, s["scale"])
            out[cu[b]:cu[b + 1], h * group:(h + 1) * group] = got.transpose(0, 1)
    return out


def _exact_prompt(s):
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for b in range(len(cq) - 1):
        n, m = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        seen = torch.ones((n, m), dtype=torch.bool, device="cuda").tril(m - n)
        rope = s["kr"][ck[b]:ck[b + 1]].double()
        for h in range(s["q"].shape[1]):
            k = torch.cat([s["k"][ck[b]:ck[b + 1], h].double(), rope], 1)[None]
            out[cq[b]:cq[b + 1], h] = _attend(s["q"][cq[b]:cq[b + 1], h].double()[None], k, s["v"][ck[b]:ck[b + 1], h].double()[None], seen, s["scale"])[0]
    return out


def _exact_fork(s):
    """Fork by fork, in lists: full pages are shared, the rest goes into the next free page. (The pages' values are copies.)"""
    page, table, lens, free = s["page"], s["table"].tolist(), s["lens"].tolist(), s["free"].tolist()
    shares, copies, used = s["shares"].tolist(), [], 0
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        lens[b] = lens[a]
        for i in range(lens[a] // page):
            table[b][i] = table[a][i]
            shares[table[a][i]] += 1
        if lens[a] % page:
            table[b][lens[a] // page] = free[used]
            copies.append((table[a][lens[a] // page], free[used], lens[a] % page))
            used += 1
        else:
            copies.append((-1, -1, 0))
    a, b, r = (torch.tensor(x) for x in zip(*copies))
    return {"table": torch.tensor(table), "lens": torch.tensor(lens), "shares": torch.tensor(shares), "copy_src": a, "copy_dst": b, "copy_rows": r,
            "used": torch.tensor([used]), "kp": None, "vp": None}


def _exact_keep(s):
    page, table, shares, cu = s["page"], s["table"].tolist(), s["shares"].tolist(), s["cu"].tolist()
    out_lens, freed = [], []
    for b, (m, n) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        out_lens.append(m - n + cu[b + 1] - cu[b])
        for i in range(-(-out_lens[b] // page), -(-m // page)):
            if shares[table[b][i]]:
                shares[table[b][i]] -= 1
            else:
                freed.append(table[b][i])
    rest = [-1] * (s["freed"].numel() - len(freed))
    return {"kp": None, "vp": None, "out_lens": torch.tensor(out_lens), "shares": torch.tensor(shares), "freed": torch.tensor(sorted(freed) + rest),
            "count": torch.tensor([len(freed)])}
