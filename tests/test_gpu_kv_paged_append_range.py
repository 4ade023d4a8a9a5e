"""kv_paged_append over the whole range of bf16: a norm's mean square that float32 does not hold."""
import numpy as np
import pytest
import torch

import rotation_ptq_b200 as sq
from oracle import oracle as O
from tests.test_gpu_kv_paged import append_case, bf16, pages_of, run_append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, False), (64, True), (0, False)])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("power,eps", [(62, 1e-6), (75, 1e-6), (110, 1e-6), (-60, 0.0), (-100, 0.0), (-100, 1e-6)])
def test_normalised_heads_of_any_size(power, eps, bits, rot, interleaved):
    c = append_case(70, [5, 9], [3, 0], 8, 2, 16, bits, rot, interleaved, True, pad=1)
    x = c["qkv"]
    x[:, :10] *= 2.0 ** power                     # queries and keys: exact in bf16
    x[3, 1] /= 2.0 ** power                       # one head vector of ordinary size among them
    t = bf16(x)
    c["q"], c["k"], c["v"] = t[:, :8], t[:, 8:10], t[:, 10:]
    pages = pages_of(c["pool"])
    n, args = c["n"], (c["pos"], c["cos"], c["sin"], interleaved)
    q = run_append(c, pages, eps=eps)[:n].double().cpu().numpy()
    ref = O.head_forward(x[:n, :8], c["w"][0], eps, *args)
    size = np.abs(O.rms_norm(x[:n, :8], c["w"][0], eps)).sum(-1, keepdims=True)
    # as for ordinary sizes: 14 float32 operations a term at most, then bf16
    bound = 2.0 ** -8 * np.abs(ref) + 14 * 2.0 ** -24 * 2 * size / np.sqrt(128)
    assert (np.abs(q - ref) <= bound).all()
    # keys are exact up to the float32 rounding: what the pages give back is within half a step of them
    k = O.head_forward(x[:n, 8:10], c["w"][1], eps, *args)
    page, row = c["pool"].table[c["seq"], c["pos"] // 16], c["pos"] % 16
    scale = pages.k_scale.cpu().numpy()[page, :, row].astype(np.float64)[..., None]
    zero = pages.k_zero.cpu().numpy()[page, :, row].astype(np.float64)[..., None]
    raw = pages.k_codes.cpu().numpy()[page, :, row]
    codes = O.unpack_int4(raw, signed=False) if bits == 4 else raw
    # (half a step, and as much again where the zero point's rounding meets the end of the codes)
    assert (np.abs((codes - zero) * scale - k) <= scale * (1 + 2.0 ** -20)).all()
    assert sq.device_status() == 0
