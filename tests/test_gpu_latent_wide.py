"""Prompts by latents with enough queries and heads for row tiles of 128 (more than 512 full tiles of 64 with d = 128, 768 with
d = 64): the bounds and references of test_gpu_latent."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from test_gpu_latent import LENGTHS, _prompt  # noqa: E402

# heads with which the lengths' 1,084 queries make that many
WIDE = pytest.mark.parametrize("d,H", [(64, 46), (128, 31)])


@WIDE
@pytest.mark.parametrize("form", ["side", "heads"])
def test_lengths(d, H, form):
    assert sum(LENGTHS) * H > 64 * (768 if d == 64 else 512)
    _prompt(LENGTHS, LENGTHS, H, d, form=form)


@WIDE
def test_after_cached_tokens(d, H):
    _prompt(LENGTHS, [n + x for n, x in zip(LENGTHS, [0, 5, 1, 63, 64, 65, 200, 0, 129, 1, 7, 300, 64, 31])], H, d)
    _prompt([400, 100, 64, 520], [200, 40, 0, 540], H, d)          # fewer keys than queries: the first see nothing


@WIDE
@pytest.mark.parametrize("value", [float("inf")])
def test_not_finite_values(d, H, value):
    def spoil(k, v, kr):
        v[50, :, 3:9], v[130, :, 20] = value, value
    n = [120, 77, 900]
    _prompt(n, n, H, d, spoil=spoil)


@WIDE
@pytest.mark.parametrize("scale", [-0.1])
def test_scales(d, H, scale):
    _prompt([1084], [1084], H, d, scale=scale)
