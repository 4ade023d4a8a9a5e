"""Calls that the binding refuses before anything is launched (no GPU needed)."""
import pytest

import rotation_ptq_b200 as sq


def test_rope_tables_are_made_on_the_gpu_only():
    """A CPU device: its memory is no kernel's to write."""
    with pytest.raises(ValueError, match="no CPU path"):
        sq.rope_tables(1e6, 4, device="cpu")
