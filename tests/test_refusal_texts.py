"""What the C calls say when they refuse misaligned pointers: each names what it takes itself (no GPU needed:
the checks come before any launch)."""
import ctypes

import pytest

import rotation_ptq_b200 as sq
from rotation_ptq_b200 import binding as bd

SQ_ERR_MISALIGNED = 3
_buf = ctypes.create_string_buffer(64)
P = (ctypes.addressof(_buf) + 15) // 16 * 16
OFF = P + 4                              # 4-byte aligned only


def text():
    return sq.lib.sq_last_error().decode()


@pytest.mark.parametrize("call", [
    lambda: sq.lib.sq_w4a4_linear(OFF, P, P, P, 1, 16, 128, P, 0, None, 0, None),
    lambda: sq.lib.sq_w4a8_linear(OFF, P, P, P, 1, 16, 128, P, 0, None, 0, None),
    lambda: sq.lib.sq_kv_rotate_quant(P, P, P, 1, 4, 2, 128, OFF, None, None, 0, P + 16, P, P, P, P, P, P, None),
    lambda: sq.lib.sq_kv_dequant(OFF, P, P, 1, 2, 128, P, None),
    lambda: sq.lib.sq_cayley_update(P, P, 0.1, 8, 1, P, OFF, P, 1 << 30, None),
    lambda: sq.lib.sq_rope_tables(1e6, 4, 128, OFF, P, None),
], ids=["w4a4_linear", "w4a8_linear", "kv_rotate_quant", "kv_dequant", "cayley_update", "rope_tables"])
def test_calls_whose_pointers_all_need_16_bytes(call):
    assert call() == SQ_ERR_MISALIGNED
    assert text() == "device pointers must be 16-byte aligned"


def test_paged_calls_name_their_own_arrays():
    pg = bd._PagesStruct(k_codes=P, k_scale=P, k_zero=P, v_codes=P, v_scale=P, v_zero=P, num_pages=2, page_size=16,
                         hkv=2, d=128, bits=4)
    rule = bd._ScoreRule(scale=0.1, softcap=0.0, window=0, slopes=None)
    at, ru = ctypes.addressof(pg), ctypes.addressof(rule)
    assert sq.lib.sq_kv_paged_dequant(at, P, 2, P, P, 1, 1, OFF, P, None) == SQ_ERR_MISALIGNED
    assert text() == "device pointers must be 16-byte aligned (int32 arrays: 4-byte)"
    assert sq.lib.sq_kv_paged_append(OFF, P, P, 512, 256, 256, 1, 4, at, P, 2, P, P, 1, None, None, 0, 0, 0, None,
                                     None, 1e-6, P, None) == SQ_ERR_MISALIGNED
    assert text() == "device pointers must be 16-byte aligned (int32 arrays: 4-byte)"
    assert sq.lib.sq_kv_paged_attention(OFF, 512, 1, 4, at, P, 2, P, P, 1, 1, ru, P, None, None, 0, None) == SQ_ERR_MISALIGNED
    assert text() == "device pointers must be 16-byte aligned (int32 arrays, slopes and lse: 4-byte)"
