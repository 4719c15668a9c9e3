"""Plain 64-bit references of the serving operators (linear attention, prompt forms, block tables,
paged attention), written from the definitions token by token and request by request, and the error
bounds that the GPU tests hold the kernels to."""
from __future__ import annotations

import math

import torch

EPS32 = 2.0 ** -24
EPS_BF16 = 2.0 ** -9      # half a step of bf16, relative to the binade's lower end; 2^-8 covers any value


def prompt(S, q, k, v, alpha, beta=None):
    """One request and head: S [d, d]; q, k, v [n, d]; alpha [n] or [n, d]; beta [n] or None. Returns the
    readouts, the last state, the same with every term taken by magnitude (linear attention only: what
    any summation order's error is relative to), and the largest column norms met."""
    S, A = S.clone(), S.abs()
    out, mag = torch.zeros_like(v), torch.zeros_like(v)
    top = S.norm(dim=0)
    for t in range(q.shape[0]):
        a = alpha[t].reshape(-1, 1)
        S, A = a * S, a * A
        e = v[t] if beta is None else beta[t] * (v[t] - k[t] @ S)
        S = S + torch.outer(k[t], e)
        A = A + torch.outer(k[t].abs(), e.abs())
        out[t], mag[t] = q[t] @ S, q[t].abs() @ A
        top = torch.maximum(top, S.norm(dim=0) + e.abs())
    return out, S, mag, A, top


def chunk_condition(k, alpha, beta, chunk=64):
    """The largest row sum of |X| |I + A| |X| over the chunks, X = (I + A)^-1 and A the delta rule's
    coupling of a chunk's tokens: how much the chunked solution magnifies a relative rounding."""
    worst = 1.0
    for c in range(0, k.shape[0], chunk):
        kc, bc = k[c:c + chunk], beta[c:c + chunk]
        n = kc.shape[0]
        A = torch.zeros((n, n), dtype=torch.float64)
        for t in range(n):
            w = 1.0
            for s in range(t - 1, -1, -1):
                w *= float(alpha[c + s + 1])
                A[t, s] = bc[t] * (kc[t] @ kc[s]) * w
        M = torch.eye(n, dtype=torch.float64) + A
        X = torch.linalg.inv(M)
        worst = max(worst, float((X.abs() @ M.abs() @ X.abs()).sum(1).max()))
    return worst


def tables(seq, new, free, table, page, T, blocks):
    """kv_build_tables in lists."""
    table = [list(r) for r in table]
    slots, pos, cu, used = [], [], [0], 0
    for b, (n, m) in enumerate(zip(seq, new)):
        n = max(n, 0)
        m = min(max(m, 0), n)
        have, need = (min(-(-x // page), blocks) for x in (n - m, n))
        for i in range(have, need):
            table[b][i] = free[used] if used < len(free) else -1
            used += 1
        for p in range(n - m, n):
            i = p // page
            ok = i < blocks and table[b][i] >= 0
            slots.append(table[b][i] * page + p % page if ok else -1)
            pos.append(p)
        cu.append(cu[-1] + m)
    return table, (slots + [-1] * T)[:T], (pos + [-1] * T)[:T], cu, used


def attention(q, k, v, scale):
    """One request: q [Hq, d], k, v [n, Hkv, d] (binary64). Zero where there is no token."""
    Hq, d = q.shape
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    g = Hq // k.shape[1]
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    for h in range(Hq):
        x = (k[:, h // g] @ q[h]) * scale
        p = torch.exp(x - x.max())
        p = p / p.sum()
        out[h], mag[h] = p @ v[:, h // g], p @ v[:, h // g].abs()
    return out, mag


def score_error(q, k, scale):
    """Bound of a binary32 score's error times log2(e): d products and sums, the scaling, and the base-2
    exponential of the difference from the maximum, each relative to the terms' magnitude."""
    g = q.shape[0] // k.shape[1]
    most = 0.0
    for h in range(q.shape[0]):
        most = max(most, float((k[:, h // g].abs() @ q[h].abs()).max()) * scale if k.shape[0] else 0.0)
    return 2 * (q.shape[1] + 8) * EPS32 * most


def is_close(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    over = err - tol
    assert bool((over <= 0).all()), f"{what}: {int((over > 0).sum())} of {err.numel()} beyond the bound, worst {float(err.max()):.3g} " \
                                    f"(bound there {float((tol if torch.is_tensor(tol) else torch.full_like(err, tol)).flatten()[int(err.argmax())]):.3g})"
    return float((err / (tol + 1e-300)).max()) if err.numel() else 0.0
