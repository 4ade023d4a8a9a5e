"""kv_paged_append refuses queries' output over its inputs (host checks only: no GPU needed)."""
import ctypes

import pytest

import rotation_ptq_b200 as sq
from rotation_ptq_b200 import binding as bd

SQ_ERR_INVALID_ARG, T, HQ, HKV = 1, 3, 4, 2
ROW = (HQ + 2 * HKV) * 256               # bytes of a token of one fused projection
_buf = ctypes.create_string_buffer(16 * ROW + 16)
P = (ctypes.addressof(_buf) + 15) // 16 * 16
Q, K, V, END = P + 4 * ROW, P + 4 * ROW + HQ * 256, P + 4 * ROW + (HQ + HKV) * 256, P + (4 + T) * ROW


def append(q_out):
    pg = bd._PagesStruct(k_codes=P, k_scale=P, k_zero=P, v_codes=P, v_scale=P, v_zero=P, num_pages=2, page_size=16,
                         hkv=HKV, d=128, bits=4)
    st = sq.lib.sq_kv_paged_append(Q, K, V, ROW // 2, ROW // 2, ROW // 2, T, HQ, ctypes.addressof(pg), P, 2, P, P, 1,
                                   None, None, 0, 0, 0, None, None, 1e-6, q_out, None)
    return st, sq.lib.sq_last_error().decode()


@pytest.mark.parametrize("q_out", [Q, K, V, Q - T * HQ * 256 + 16, END - 16])
def test_output_over_the_inputs(q_out):
    assert append(q_out) == (SQ_ERR_INVALID_ARG, "q_out may not overlap q, k or v")


@pytest.mark.parametrize("q_out", [Q - T * HQ * 256, END])
def test_output_beside_the_inputs(q_out):
    """Passes the check: what stops the call here, if anything, is that there is no device."""
    if sq_has_device():
        pytest.skip("the buffers are host memory")
    assert "overlap" not in append(q_out)[1]


def sq_has_device():
    import torch
    return torch.cuda.is_available()
