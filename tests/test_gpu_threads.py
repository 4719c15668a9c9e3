"""Calls that make their own workspace, from two threads at once on one stream (and on a stream each):
every result is that of the same call alone, bit for bit, while each thread also allocates, fills and
frees memory of its own between the calls."""
import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from quantized_delta_rule_gdn_amd import lib  # noqa: E402


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _calls(seed):
    """The three calls that take a workspace, each as a function of its outputs, and the outputs' makers."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    H, d, T = 4, 128, 1500
    q, k, v = _unit(normal(T, H, d)).bfloat16(), _unit(normal(T, H, d)).bfloat16(), normal(T, H, d).bfloat16()
    a, b = torch.rand((T, H), generator=gen, device="cuda") * 0.1 + 0.9, torch.rand((T, H), generator=gen, device="cuda")
    cu = torch.tensor([0, 1100, T], dtype=torch.int32, device="cuda")
    sl = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    B, Hq, Hkv, page, blocks = 3, 8, 2, 16, 200
    kp, vp = normal(B * blocks, Hkv, page, d).bfloat16(), normal(B * blocks, Hkv, page, d).bfloat16()
    table = torch.arange(B * blocks, dtype=torch.int32, device="cuda").reshape(B, blocks)
    lens = torch.tensor([3100, 7, 1500], dtype=torch.int32, device="cuda")
    qa = normal(B, Hq, d).bfloat16()

    def prompts():
        return torch.zeros((2, H, d, d), device="cuda"), torch.zeros_like(v)

    return [(prompts, lambda o, s: lib.fp32_delta_prefill(o[0], sl, cu, q, k, v, a, b, o[1], stream=s)),
            (prompts, lambda o, s: lib.fp32_linear_prefill(o[0], sl, cu, q, k, v, a, o[1], stream=s)),
            (lambda: (torch.zeros_like(qa),), lambda o, s: lib.kv_decode_attention(qa, kp, vp, table, lens, o[0], stream=s))]


@pytest.mark.parametrize("own_streams", [False, True])
def test_two_threads_at_once(own_streams):
    calls = [_calls(seed) for seed in (1, 2)]
    alone = []
    for one in calls:
        alone.append([])
        for make, call in one:
            o = make()
            call(o, None)
            alone[-1].append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() if own_streams else torch.cuda.current_stream() for _ in calls]
    got, errors, start = [[], []], [], threading.Barrier(2)

    def work(i):
        try:
            start.wait(30)
            with torch.cuda.stream(streams[i]):
                for n in range(12):
                    for make, call in calls[i]:
                        o = make()
                        call(o, streams[i] if n % 2 else None)
                        got[i].append(o)
                        torch.full((1 << (18 + n % 5),), float("nan"), device="cuda")
        except Exception as e:   # shown by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i in range(2):
        assert len(got[i]) == 36
        for n, o in enumerate(got[i]):
            for x, y in zip(o, alone[i][n % 3]):
                assert torch.equal(x, y), f"thread {i}, call {n}"
