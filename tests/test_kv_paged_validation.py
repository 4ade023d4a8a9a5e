"""The paged cache's calls refuse malformed operands before any launch (no GPU needed), and the oracle's
head map and causal attention are the path's own where they overlap."""
import ctypes

import numpy as np
import pytest
import torch

import rotation_ptq_b200 as sq
from oracle import oracle as O

u8, f32, bf16, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


def z(shape, dt):
    return torch.zeros(shape, dtype=dt)


def pool(n=4, hkv=2, ps=16, rb=64, **bad):
    parts = {}
    for key in "kv":
        parts.update({key + "_codes": z((n, hkv, ps, rb), u8), key + "_scale": z((n, hkv, ps), f32),
                      key + "_zero": z((n, hkv, ps), u8)})
    return {**parts, **bad}


@pytest.mark.parametrize("bad,msg", [
    (dict(k_codes=z((4, 2, 16, 32), u8)), "64 bytes"),
    (dict(k_codes=z((4, 2, 24, 64), u8)), "power of two"),
    (dict(k_codes=z((4, 65, 16, 64), u8)), "1..64 KV heads"),
    (dict(k_scale=z((4, 16, 2), f32)), "k_scale must have shape"),
    (dict(v_scale=z((4, 2, 16), torch.float16)), "v_scale must be torch.float32"),
    (dict(v_codes=z((4, 2, 16, 128), u8)[..., ::2]), "v_codes must be contiguous"),
    (dict(k_zero=z((4, 2, 16), i32)), "k_zero must be torch.uint8"),
])
def test_pages_reject(bad, msg):
    with pytest.raises(ValueError, match=msg):
        sq.KVPages(**pool(**bad))
    with pytest.raises(ValueError, match="4 or 8"):
        sq.KVPages.empty(4, 16, 2, bits=5, device="cpu")


def append_ok(T=3, hq=4, hkv=2, B=2):
    return dict(q=z((T, hq, 128), bf16), k=z((T, hkv, 128), bf16), v=z((T, hkv, 128), bf16),
                pages=sq.KVPages(**pool()), block_table=z((B, 2), i32), cu_seqlens=z((B + 1,), i32),
                cached=z((B,), i32), cos=z((9, 64), f32), sin=z((9, 64), f32))


@pytest.mark.parametrize("bad,msg", [
    (dict(q=z((3, 4, 128), f32)), "q must be a bf16"),
    (dict(q=z((3, 4, 64), bf16)), "q must have shape"),
    (dict(q=z((3, 5, 128), bf16)), "multiple of the 2 KV heads"),
    (dict(k=z((2, 2, 128), bf16)), "same number of tokens"),
    (dict(k=z((3, 1, 128), bf16)), "k must have shape"),
    (dict(v=z((3, 4, 128), bf16)[:, ::2]), "contiguous heads"),
    (dict(q=z((3, 4 * 128 + 4), bf16).as_strided((3, 4, 128), (4 * 128 + 4, 128, 1))), "multiple of 8"),
    (dict(q=z((1, 4, 128), bf16).expand(3, 4, 128)), "holds its heads"),
    (dict(cos=None), "both be given or both"),
    (dict(cos=z((9, 60), f32), sin=z((9, 60), f32)), "multiple of 16"),
    (dict(sin=z((8, 64), f32)), "sin must have shape"),
    (dict(q_norm=z((64,), f32)), "q_norm must have shape"),
    (dict(k_norm=z((128,), bf16)), "k_norm must be torch.float32"),
    (dict(cu_seqlens=z((2,), i32)), "cu_seqlens must have shape"),
    (dict(cached=z((2,), torch.int64)), "cached must be torch.int32"),
    (dict(block_table=z((2,), i32)), "block_table must be"),
    (dict(q_out=z((3, 4, 128), f32)), "q_out must be torch.bfloat16"),
    (dict(), "no CPU path"),
])
def test_append_rejects(bad, msg):
    with pytest.raises(ValueError, match=msg):
        sq.kv_paged_append(**{**append_ok(), **bad})


def attend_ok(T=3, hq=4, B=2):
    return dict(q=z((T, hq, 128), bf16), pages=sq.KVPages(**pool()), block_table=z((B, 2), i32),
                cu_seqlens=z((B + 1,), i32), lengths=z((B,), i32), max_q=1)


@pytest.mark.parametrize("bad,msg", [
    (dict(q=z((3, 3, 128), bf16)), "multiple of the 2 KV heads"),
    (dict(slopes=z((2,), f32)), "slopes must have shape"),
    (dict(out=z((3, 4, 64), bf16)), "out must have shape"),
    (dict(lse=z((3, 4), bf16)), "lse must be torch.float32"),
    (dict(lengths=z((3,), i32)), "lengths must have shape"),
    (dict(workspace=z((8,), f32)), "workspace must be a contiguous uint8"),
    (dict(), "no CPU path"),
])
def test_attention_rejects(bad, msg):
    with pytest.raises(ValueError, match=msg):
        sq.kv_paged_attention(**{**attend_ok(), **bad})
    prefix = dict(prefix_table=z((2,), i32), prefix_len=20)
    with pytest.raises(ValueError, match=msg):
        sq.kv_prefix_attention(**{**attend_ok(), **prefix, **bad})


@pytest.mark.parametrize("bad,msg", [
    (dict(prefix_len=0), "prefix_len must be 1 .. 32"), (dict(prefix_len=33), "prefix_len must be 1 .. 32"),
    (dict(prefix_table=z((2, 1), i32)), "prefix_table must be int32"),
    (dict(prefix_table=z((2,), torch.int64)), "prefix_table must be torch.int32")])
def test_prefix_rejects(bad, msg):
    with pytest.raises(ValueError, match=msg):
        sq.kv_prefix_attention(**{**attend_ok(), "prefix_table": z((2,), i32), "prefix_len": 20, **bad})
    with pytest.raises(TypeError, match="KVPages"):
        sq.kv_paged_attention(**{**attend_ok(), "pages": None})


def test_read_back_rejects():
    a = attend_ok()
    args = (a["pages"], a["block_table"], a["cu_seqlens"], a["lengths"], 5)
    with pytest.raises(ValueError, match="k_out must have shape"):
        sq.kv_paged_dequant(*args, k_out=z((5, 2, 64), bf16))
    with pytest.raises(ValueError, match="no CPU path"):
        sq.kv_paged_dequant(*args)


def test_c_calls_refuse_on_the_host():
    """The C entry points' own checks: they return before anything is launched or read."""
    from rotation_ptq_b200 import binding as bd
    lib = sq.lib
    buf = ctypes.create_string_buffer(64 + 16)
    p = (ctypes.addressof(buf) + 15) // 16 * 16

    def pages(**bad):
        f = dict(k_codes=p, k_scale=p, k_zero=p, v_codes=p, v_scale=p, v_zero=p, num_pages=2, page_size=16,
                 hkv=2, d=128, bits=4)
        f.update(bad)
        return bd._PagesStruct(**f)

    def rule(**bad):
        return bd._ScoreRule(**{**dict(scale=0.1, softcap=0.0, window=0, slopes=None), **bad})

    def attention(pg=None, ru=None, T=1, hq=4, B=1, width=2, max_q=1, stride=512, q=p, out=p, table=p, ws=None):
        pg, ru = pages() if pg is None else pg, rule() if ru is None else ru
        return lib.sq_kv_paged_attention(q, stride, T, hq, ctypes.addressof(pg), table, width, p, p, B, max_q,
                                         ctypes.addressof(ru), out, None, ws, 0, None)

    for kw, want in [
            (dict(pg=pages(bits=5)), 2), (dict(pg=pages(d=64)), 2), (dict(pg=pages(page_size=8)), 2),
            (dict(pg=pages(page_size=48)), 2), (dict(pg=pages(page_size=8192)), 2), (dict(pg=pages(hkv=0)), 2),
            (dict(pg=pages(num_pages=0)), 2), (dict(pg=pages(v_zero=None)), 1), (dict(pg=pages(k_scale=p + 4)), 3),
            (dict(hq=3), 2), (dict(hq=512), 2), (dict(T=-1), 1), (dict(B=-1), 1), (dict(width=0), 1),
            (dict(T=1 << 31), 2), (dict(width=1 << 27), 2), (dict(B=(1 << 20) + 1), 2),
            (dict(ru=rule(scale=float("nan"))), 1), (dict(ru=rule(scale=float("inf"))), 1),
            (dict(ru=rule(softcap=-1.0)), 1), (dict(ru=rule(softcap=float("nan"))), 1),
            (dict(ru=rule(window=-1)), 1), (dict(ru=rule(window=(1 << 30) + 1)), 1),
            (dict(max_q=-1), 1), (dict(stride=500), 2), (dict(stride=516), 2),
            (dict(q=None), 1), (dict(out=None), 1), (dict(q=p + 2), 3), (dict(table=p + 2), 3), (dict(ws=p + 4), 3),
            (dict(T=0), 0), (dict(B=0), 0), (dict(max_q=0), 0)]:
        assert attention(**kw) == want, (kw, lib.sq_last_error())
    pg, ru = pages(), rule()
    for n in (0, -1, 1 << 30):
        assert lib.sq_kv_prefix_attention(p, 512, 1, 4, ctypes.addressof(pg), p, n, p, 2, p, p, 1, 1,
                                          ctypes.addressof(ru), p, None, None, 0, None) == 1

    def append(T=1, hq=4, B=1, width=2, cos=None, sin=None, max_pos=0, rot=0, inter=0, eps=1e-6, norm=None, q=p, qs=512):
        return lib.sq_kv_paged_append(q, p, p, qs, 256, 256, T, hq, ctypes.addressof(pg), p, width, p, p, B, cos,
                                      sin, max_pos, rot, inter, norm, None, eps, p, None)

    for kw, want in [(dict(cos=p), 1), (dict(cos=p, sin=p, max_pos=0, rot=128), 1),
                     (dict(cos=p, sin=p, max_pos=9, rot=8), 2), (dict(cos=p, sin=p, max_pos=9, rot=144), 2),
                     (dict(cos=p, sin=p, max_pos=9, rot=40), 2), (dict(inter=2), 1), (dict(eps=-1.0), 1),
                     (dict(eps=float("nan")), 1), (dict(qs=511), 2), (dict(q=None), 1), (dict(norm=p + 4), 3),
                     (dict(T=0), 0), (dict(B=0), 0), (dict(hq=5), 2)]:
        assert append(**kw) == want, (kw, lib.sq_last_error())


def test_oracle_head_map_is_the_contiguous_path():
    rng = np.random.default_rng(3)
    x, pos = rng.standard_normal((5, 2, 128)), np.array([0, 1, 7, 3, 2])
    cos, sin = O.rope_tables(1e6, 8, 128)
    want = O.headwise_hadamard(O.rope(x, pos, cos, sin))
    assert np.allclose(O.head_forward(x, None, 0.0, pos, cos, sin, False), want, atol=1e-13)
    # interleaved pairs are the half layout's under a permutation of channels, and a norm gives unit mean square
    perm = np.arange(128).reshape(2, 64).T.reshape(-1)
    y = np.empty_like(x)
    y[..., :] = O.rope_part(x[..., perm], pos, cos, sin, True)
    back = np.empty_like(y)
    back[..., perm] = y
    assert np.allclose(back, O.rope_part(x, pos, cos, sin, False), atol=1e-13)
    assert np.allclose(np.mean(O.rms_norm(x, np.ones(128), 0.0) ** 2, -1), 1.0)
    # channels behind the rotated part pass
    part = O.rope_part(x, pos, cos[:, :16], sin[:, :16], False)
    assert np.array_equal(part[..., 32:], x[..., 32:])


def test_oracle_causal_attention_is_decode_attention_at_the_last_row():
    rng = np.random.default_rng(4)
    q, K, V = rng.standard_normal((3, 4, 128)), rng.standard_normal((9, 2, 128)), rng.standard_normal((9, 2, 128))
    out, lse, spread, _ = O.causal_attention(q, K, V, np.array([6, 7, 8]), np.arange(9))
    for i, n in enumerate((7, 8, 9)):
        want = O.decode_attention(q[i:i + 1], K, V, np.array([n]), 9)
        assert np.allclose(out[i], want[0], atol=1e-12)
    assert (spread >= np.abs(out) - 1e-12).all() and np.isfinite(lse).all()
    out, lse, _, _ = O.causal_attention(q, K, V, np.array([-1, 0, 5]), np.arange(9), window=1)
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all()
    assert np.allclose(out[1], np.repeat(V[0], 2, axis=0)) and np.allclose(out[2], np.repeat(V[5], 2, axis=0))
