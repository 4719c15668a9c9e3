"""CPU-only: how much workspace the attentions of several tokens ask for, and up to which sizes they take a call."""
import pytest

from quantized_delta_rule_gdn_amd import lib


@pytest.mark.parametrize("name,head,rows,width", [
    ("kv_tree_attention_workspace_bytes", (32, 8, 128), 128, 130), ("kv_tree_attention_workspace_bytes", (16, 2, 64), 128, 66),
    ("kv_latent_attention_workspace_bytes", (128, 512), 64, 514), ("kv_latent_attention_workspace_bytes", (64, 256), 64, 258)])
def test_the_workspace_is_what_one_round_of_workgroups_leaves(name, head, rows, width):
    """No more units of work, and no wider bound of a request's new tokens, ask for more: a partial readout, a maximum and a sum
    of the rows of at most 768 workgroups (3 a CU), and 8 bytes a request."""
    size = getattr(lib.load(), name)
    for B in (48, 64, 256, 512):
        for most in (32, 512):
            got = size(B, *head, most, 4096) - 8 * B
            assert 0 < got <= min(768 * rows * width * 4, 2 ** 26), (B, most, got)
            assert got == size(48, *head, 32, 4096) - 8 * 48
