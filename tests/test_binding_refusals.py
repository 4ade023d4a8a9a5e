"""Calls that the binding refuses before anything is launched (no GPU needed)."""
import pytest
import torch

import rotation_ptq_b200 as sq
from tests.test_kv_paged_validation import attend_ok


def test_rope_tables_are_made_on_the_gpu_only():
    """A CPU device: its memory is no kernel's to write."""
    with pytest.raises(ValueError, match="no CPU path"):
        sq.rope_tables(1e6, 4, device="cpu")


@pytest.mark.parametrize("bad,msg", [
    (dict(window=1 << 32), "window must be a whole number from 0 to 1073741824"),    # 0 in 32 bits: no window
    (dict(window=(1 << 32) + 5), "window must be"), (dict(window=-1), "window must be"),
    (dict(window=0.5), "window must be"),
    (dict(max_q=1 << 32), "max_q must be a whole number from 0 to 2147483647"),      # 0: nothing to do
    (dict(max_q=-1), "max_q must be"), (dict(max_q=1.5), "max_q must be"),
])
def test_numbers_that_32_bits_do_not_hold(bad, msg):
    args = {**attend_ok(), **bad}
    with pytest.raises(ValueError, match=msg):
        sq.kv_paged_attention(**args)
    with pytest.raises(ValueError, match=msg):
        sq.kv_prefix_attention(**args, prefix_table=torch.zeros(2, dtype=torch.int32), prefix_len=20)


def test_token_counts_that_32_bits_do_not_hold():
    a = attend_ok()
    for n in (-1, 1 << 31, 2.5):
        with pytest.raises(ValueError, match="num_tokens must be a whole number"):
            sq.kv_paged_dequant(a["pages"], a["block_table"], a["cu_seqlens"], a["lengths"], n)
    with pytest.raises(ValueError, match="max_q must be a whole number"):
        sq.kv_attention_workspace_bytes(4, 4, a["pages"], 2, 2, 1 << 32)
