"""Plain 64-bit references of the operators of a shared and drafted cache (attention of several tokens,
latent attention, forked tables, kept tokens, pages given back), written from the definitions request
by request, and the error bounds that the GPU tests hold the kernels to."""
from __future__ import annotations

import torch

EPS32 = 2.0 ** -24
BF16 = 2.0 ** -8          # a rounding to bf16, relative to the value


def seen(n, m, bits=None):
    """[n, m]: which of m positions each of the last n tokens sees; bits [n, n] among them, or in order."""
    s = torch.ones((n, m), dtype=torch.bool)
    if m < n:                                     # the first new tokens have no position
        own = torch.ones((n, n), dtype=torch.bool).tril() if bits is None else bits
        return own[:, n - m:].clone()
    s[:, m - n:] = torch.ones((n, n), dtype=torch.bool).tril() if bits is None else bits
    return s


def words(bits, count=None):
    """Rows of truth values as 64-bit words [rows, count]."""
    n, m = bits.shape
    count = count or -(-m // 64)
    out = torch.zeros((n, count), dtype=torch.int64)
    for i in range(n):
        for j in torch.nonzero(bits[i])[:, 0].tolist():
            out[i, j // 64] |= -(1 << 63) if j % 64 == 63 else 1 << (j % 64)
    return out


def attend(q, k, v, live, scale):
    """q [n, Hq, d], k [m, Hkv, d], v [m, Hkv, e], live [n, m], in 64 bits: readouts [n, Hq, e], the same
    with |v|, and a bound of a binary32 score's relative effect on its weight."""
    n, Hq, d = q.shape
    m, Hk = k.shape[:2]
    out, mag = torch.zeros((n, Hq, v.shape[2]), dtype=torch.float64), torch.zeros((n, Hq, v.shape[2]), dtype=torch.float64)
    worst = 0.0
    if m == 0 or n == 0:
        return out, mag, worst
    for h in range(Hq):
        kh, vh = k[:, h * Hk // Hq], v[:, h * Hk // Hq]
        x = (q[:, h] @ kh.T) * scale
        x = torch.where(live, x, torch.full_like(x, -torch.inf))
        top = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        total = p.sum(1, keepdim=True)
        p = torch.where(live, p / torch.where(total == 0, torch.ones_like(total), total), torch.zeros_like(p))
        for i in range(n):                         # (a value that a token does not see does not matter, whatever it is)
            out[i, h], mag[i, h] = p[i, live[i]] @ vh[live[i]], p[i, live[i]] @ vh[live[i]].abs()
        worst = max(worst, float((q[:, h].abs() @ torch.nan_to_num(kh.abs(), posinf=0.0).T).max()) * abs(scale))
    # d products and sums, the scaling, and the base-2 exponential of the difference from the maximum
    return out, mag, 2 * (d + 8) * EPS32 * worst


def tolerance(o, mag, score, m, weight, splits=64):
    """A readout's bound: its own rounding, and for numerator and normaliser each the score's error, the
    weight's rounding and binary32 sums (a tile at a time, and over the parts)."""
    return BF16 * o.abs() + 2 * (score + weight + (m // 16 + splits) * EPS32) * mag + 1e-37


def is_close(got, want, tol, what):
    got = got.double().cpu()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: not finite at other places"
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    err = torch.where(fine, (got - want).abs(), torch.zeros_like(want))
    over = err > torch.where(fine, tol, torch.zeros_like(tol))
    assert not bool(over.any()), f"{what}: {int(over.sum())} of {err.numel()} beyond the bound, worst {float((err / tol.clamp(min=1e-300))[fine].max()):.3g} of it"
    return float((err / tol)[fine].max()) if fine.any() else 0.0


def fork(src, dst, lens, free, table, shares, page, pages):
    """kv_fork_tables in lists."""
    table, lens, shares = [list(r) for r in table], list(lens), list(shares)
    blocks, copies, used = len(table[0]) if table else 0, [], 0
    for a, b in zip(src, dst):
        if not (0 <= a < len(lens) and 0 <= b < len(lens)):
            copies.append((-1, -1, 0))
            continue
        n = max(lens[a], 0)
        lens[b] = lens[a]
        full, part = min(n // page, blocks), n % page if n // page < blocks else 0
        for j in range(full):
            table[b][j] = table[a][j]
            if 0 <= table[a][j] < pages:
                shares[table[a][j]] += 1
        got = (-1, -1, 0)
        if part:
            fresh = free[used] if used < len(free) else -1
            table[b][full] = fresh
            if 0 <= table[a][full] < pages and 0 <= fresh < pages:
                got = (table[a][full], fresh, part)
            used += 1
        copies.append(got)
    return table, lens, shares, copies, used


def release(keep, lens, table, shares, page):
    """kv_free_pages in lists: the shares left and the pages that no one holds."""
    shares, gone = list(shares), []
    for b, n in enumerate(lens):
        first, stop = (min(-(-max(x, 0) // page), len(table[b])) for x in (keep[b] if keep else 0, n))
        for j in range(first, stop):
            p = table[b][j]
            if not 0 <= p < len(shares) or p in gone:
                continue
            if shares[p] > 0:
                shares[p] -= 1
            else:
                gone.append(p)
    return shares, sorted(gone)
