"""CPU-only: what a delta-rule call of many requests sets aside for those of them that run in chunks."""
import pytest

from quantized_delta_rule_gdn_amd import lib

CHUNK = 5 * 64 * 64 * 2 + 2 * 64 * 4     # bytes of a chunk and head: five bf16 pieces [64][64], two gates a token


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,T", [(65, 65), (512, 512), (512, 100), (1000, 1000), (8000, 129)])
def test_no_call_of_many_tokens_has_room_for_single_tokens_only(B, T, d):
    """One request may hold all T tokens: ceil(T / 64) chunks, and no arrangement of the tokens has more
    than T / 32 (a request that runs in chunks has 33 tokens or more)."""
    n = lib.load().fp32_prefill_workspace_bytes(1, B, T, 4, d, lib.DAMP_BF16, lib.DAMP_DECAY_SCALAR)
    assert n == T // 32 * 4 * CHUNK >= -(-T // 64) * 4 * CHUNK


@pytest.mark.parametrize("B,T,chunks", [(1, 32, 0), (100, 32, 0), (64, 64, 0), (200, 50, 0), (1, 33, 1), (32, 33, 32), (63, 64, 64), (64, 65, 65)])
def test_sizes_around_the_rule(B, T, chunks):
    n = lib.load().fp32_prefill_workspace_bytes(1, B, T, 1, 64, lib.DAMP_BF16, lib.DAMP_DECAY_SCALAR)
    assert n == chunks * CHUNK


def test_chunk_numbers_of_long_requests_do_not_meet():
    """The numbering by begin / 32 over random lists: every chunk of a request of more than 32 tokens has a
    number of its own below T / 32, and the last request that begins at or before 32 (number + 1) - 1 owns it."""
    import random
    rng = random.Random(1)
    for _ in range(2000):
        lens = [rng.choice([0, 1, 2, 31, 32, 33, 34, 63, 64, 65, 66, 96, 97, 128, 129, 300]) for _ in range(rng.randint(1, 30))]
        begin = [sum(lens[:b]) for b in range(len(lens) + 1)]
        seen = {}
        for b, n in enumerate(lens):
            for j in range(-(-n // 64) if n > 32 else 0):
                i = begin[b] // 32 + j
                assert i not in seen and i < begin[-1] // 32
                seen[i] = b
                assert max(x for x in range(len(lens)) if begin[x] // 32 <= i) == b
