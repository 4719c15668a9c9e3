"""Calls that the header allows and that a program makes now and then: arrays at their least alignment,
one workspace for two captured graphs, the debug checks."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from quantized_delta_rule_gdn_amd import lib  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _off(t, n):
    """The same values n elements into a buffer (its allocation is 512-byte aligned)."""
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    buf[n:].copy_(t.flatten())
    out = buf[n:].view(t.shape)
    assert out.data_ptr() % 16 == n * t.element_size() % 16
    return out


def _prompt(T, H, d, dtype, key, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    a = 0.8 + 0.2 * torch.rand((T, H, d) if key else (T, H), generator=gen, device="cuda")
    return _unit(normal(T, H, d)).to(dtype), _unit(normal(T, H, d)).to(dtype), normal(T, H, d).to(dtype), a, torch.rand((T, H), generator=gen, device="cuda")


@pytest.mark.parametrize("dtype,d,key", [(torch.bfloat16, 64, False), (torch.bfloat16, 128, True), (torch.float32, 32, True), (torch.float32, 16, False)])
@pytest.mark.parametrize("by", [1, 3])
def test_prompts_with_gates_at_their_least_alignment(dtype, d, key, by):
    """alpha, beta, slots, lengths 4 (and 12) bytes off a 16-byte border; q, k, v and out on one only."""
    T, H = 100, 3
    q, k, v, a, b = _prompt(T, H, d, dtype, key)
    cu, sl = torch.tensor([0, 37, T], dtype=torch.int32, device="cuda"), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    half = 8 if dtype == torch.bfloat16 else 4
    for delta in (False, True):
        got = []
        for move in (lambda t, n: t, _off):
            pool, out = torch.ones((2, H, d, d), device="cuda"), torch.zeros_like(v)
            out = move(out, half)
            args = (pool, move(sl, by), move(cu, by), move(q, half), move(k, half), move(v, half), move(a, by))
            res = move(torch.ones(2, dtype=torch.int32, device="cuda"), by)
            if delta:
                lib.fp32_delta_prefill(*args, move(b, by), out, resume=res)
            else:
                lib.fp32_linear_prefill(*args, out, resume=res)
            torch.cuda.synchronize()
            got.append((pool, out))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("dtype,d,key", [(torch.bfloat16, 128, True), (torch.bfloat16, 16, False), (torch.float32, 64, True)])
def test_linear_step_at_its_least_alignment(dtype, d, key):
    B, H = 3, 2
    q, k, v, a, _ = _prompt(B, H, d, dtype, key)
    sl = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    got = []
    for move in (lambda t, n: t, _off):
        pool, out = torch.ones((3, H, d, d), device="cuda"), torch.zeros((B, H, d), device="cuda")
        lib.fp32_linear_step(pool, move(sl, 1), move(q, 1), move(k, 3), move(v, 1), move(a, 1), out)
        torch.cuda.synchronize()
        got.append((pool, out))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_attention_and_tables_at_their_least_alignment():
    gen = torch.Generator(device="cuda").manual_seed(3)
    B, Hq, Hkv, d, page, blocks = 3, 4, 2, 64, 16, 90
    kp, vp = (torch.randn((B * blocks, Hkv, page, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    q, kn, vn = (torch.randn((B, h, d), generator=gen, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    table = torch.arange(B * blocks, dtype=torch.int32, device="cuda").reshape(B, blocks)
    lens = torch.tensor([1400, 1, 640], dtype=torch.int32, device="cuda")
    got = []
    for move in (lambda t, n: t, _off):
        k2, v2, out = move(kp.clone(), 8), move(vp.clone(), 8), move(torch.zeros_like(q), 8)
        lib.kv_decode_attention(move(q, 8), k2, v2, move(table, 1), move(lens, 3), out, k_new=move(kn, 8), v_new=move(vn, 8))
        slots = move(torch.empty(5, dtype=torch.int64, device="cuda"), 1)
        tab, pos, cu, used = (move(torch.full(n, -1, dtype=torch.int32, device="cuda"), 1) for n in ((B, blocks), (5,), (B + 1,), (1,)))
        new = torch.tensor([1, 1, 2], dtype=torch.int32, device="cuda")
        lib.kv_build_tables(move(lens, 1), move(new, 3), move(table.flatten()[:9].contiguous(), 1), tab, page, slots, pos, cu, used)
        lib.kv_append(move(kn, 8), move(vn, 8), move(torch.tensor([40, 99, -1], device="cuda"), 1), k2, v2)
        torch.cuda.synchronize()
        got.append([k2, v2, out, slots, tab, pos, cu, used])
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_one_workspace_for_two_captured_graphs():
    """Nothing in a workspace is kept: graphs of different calls share one, replayed in turn on one stream."""
    H, d, T = 3, 128, 900
    q, k, v, a, b = _prompt(T, H, d, torch.bfloat16, False)
    cu, sl = torch.tensor([0, 600, T], dtype=torch.int32, device="cuda"), torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(9)
    kp, vp = (torch.randn((200, 2, 16, 128), generator=gen, device="cuda").bfloat16() for _ in range(2))
    table, lens = torch.randperm(200, device="cuda", generator=gen).to(torch.int32).reshape(2, 100), torch.tensor([1600, 900], dtype=torch.int32, device="cuda")
    qa = torch.randn((2, 8, 128), generator=gen, device="cuda").bfloat16()
    n = max(lib.prefill_workspace_bytes(True, 2, T, H, d, torch.bfloat16), lib.prefill_workspace_bytes(False, 2, T, H, d, torch.bfloat16),
            lib.kv_decode_attention_workspace_bytes(2, 8, 2, 128, 1600))
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def calls(w):
        pool, out, oa = torch.zeros((2, H, d, d), device="cuda"), torch.zeros_like(v), torch.zeros_like(qa)
        pool2, out2 = torch.zeros_like(pool), torch.zeros_like(out)
        return [(lambda: (pool.zero_(), lib.fp32_delta_prefill(pool, sl, cu, q, k, v, a, b, out, workspace=w)), (pool, out)),
                (lambda: (pool2.zero_(), lib.fp32_linear_prefill(pool2, sl, cu, q, k, v, a, out2, workspace=w)), (pool2, out2)),
                (lambda: lib.kv_decode_attention(qa, kp, vp, table, lens, oa, workspace=w), (oa,))]

    eager, shared = calls(None), calls(ws)
    graphs = []
    for (f, _), (g, _) in zip(eager, shared):
        f()
        g()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g()
        graphs.append(graph)
    for i in range(4):
        for t in (q, qa):
            t.copy_(t.flip(0))
        for (f, _), graph in zip(eager, graphs):
            f()
            graph.replay()
            if i % 2:
                ws.fill_(255)
        torch.cuda.synchronize()
        for (_, x), (_, y) in zip(eager, shared):
            for s, t in zip(x, y):
                assert torch.equal(s, t), f"replay {i}"


DEBUG = """
import torch
from quantized_delta_rule_gdn_amd import lib
H, d, T = 2, 64, 80
z = torch.zeros((T, H, d), dtype=torch.bfloat16, device="cuda")
pool, a = torch.zeros((3, H, d, d), device="cuda"), torch.ones((T, H), device="cuda")
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
lib.fp32_delta_prefill(pool, i32(0, 2), i32(0, 40, 80), z, z, z, a, a, z.clone())
lib.fp32_linear_prefill(pool, i32(0, 2), i32(0, 40, 40), z, z, z, a, z.clone())
lib.fp32_linear_step(pool, i32(0, 2), z[:2], z[:2], z[:2], a[:2], torch.zeros((2, H, d), device="cuda"))
bad = 0
for slots, cu in ((i32(0, 3), i32(0, 40, 80)), (i32(1, 1), i32(0, 40, 80)), (i32(0, 2), i32(0, 81, 80)), (i32(0, 2), i32(0, 40, 81)), (i32(0, 2), i32(1, 40, 80)), (i32(0, 2), i32(0, -1, 80))):
    for call in (lambda: lib.fp32_delta_prefill(pool, slots, cu, z, z, z, a, a, z.clone()), lambda: lib.fp32_linear_prefill(pool, slots, cu, z, z, z, a, z.clone())):
        try:
            call()
        except lib.DampError as e:
            bad += e.status == lib.DAMP_ERR_SLOT_INDEX
try:
    lib.fp32_linear_step(pool, i32(0, 7), z[:2], z[:2], z[:2], a[:2], torch.zeros((2, H, d), device="cuda"))
except lib.DampError as e:
    bad += e.status == lib.DAMP_ERR_SLOT_INDEX
torch.cuda.synchronize()
print("refused", bad)
"""


def test_debug_checks_of_slots_and_lengths():
    r = subprocess.run([sys.executable, "-c", DEBUG], cwd=ROOT, env={**os.environ, "DAMP_DEBUG": "1"}, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "refused 13" in r.stdout, r.stdout + r.stderr
