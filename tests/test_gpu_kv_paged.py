"""The paged KV cache on the GPU against the float64 oracle: append, read-back, attention over pages and
behind a shared prefix, and the calls one after another as a server makes them."""
import pathlib
import subprocess
import sys

import numpy as np
import pytest
import torch

import rotation_ptq_b200 as sq
from oracle import oracle as O
from tests import paged as G
from tests import parity as P

pytestmark = pytest.mark.gpu
D = 128
STREAM_EPS = 2.0 ** -19      # weights held as two fp16 halves (2^-22) and ex2 (2^-22), sums of both
# the tile kernel holds weights (times the value's scale) in one fp16 number: half a step is 2^-11 of it
TILE_EPS = 2.0 ** -11 + STREAM_EPS
TILE_STEP = 2.0 ** -32


def cu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float64)).to(torch.bfloat16).cuda()


def pages_of(pool):
    return sq.KVPages(**{k: cu(v) for k, v in pool.arrays.items()})


def attend(prob, pages=None, q=None, **kw):
    pages = pages_of(prob.pool) if pages is None else pages
    out = torch.full((prob.T, prob.hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((prob.T, prob.hq), 7.0, device="cuda")
    args = dict(max_q=max(prob.new, default=1), out=out, lse=lse,
                slopes=None if prob.slopes is None else cu(prob.slopes), **prob.rule)
    args.update(kw)
    q = bf16(prob.q) if q is None else q
    batch = (cu(prob.table()), cu(prob.cu), cu(np.array(prob.own, np.int32)))
    if prob.prefix:
        got = sq.kv_prefix_attention(q, pages, cu(prob.prefix_table()), prob.prefix, *batch, **args)
    else:
        got = sq.kv_paged_attention(q, pages, *batch, **args)
    assert got is out
    return out, lse


def weight_eps(prob):
    """By the kernel that a call's longest sequence, or a prefix read for the whole batch, goes to."""
    rows = max(prob.new) * (prob.hq // prob.hkv)
    return TILE_EPS if rows > 16 or (prob.prefix and len(prob.new) > 1) else STREAM_EPS


def check(prob, out, lse):
    ref = prob.reference()
    eps = weight_eps(prob)
    b_out, b_lse = prob.bounds(ref, eps, *([TILE_STEP] if eps == TILE_EPS else []))
    o, m = out.double().cpu().numpy(), lse.double().cpu().numpy()
    n = sum(prob.new)
    assert (o[n:] == 7).all() and (m[n:] == 7).all(), "rows behind the last sequence were written"
    empty = np.isneginf(ref[1][:n])
    assert np.array_equal(np.isneginf(m[:n]), empty)
    assert (o[:n][empty] == 0).all()
    err = np.abs(o[:n] - ref[0][:n])
    assert (err <= b_out[:n]).all(), "out: %.3g times its bound" % (err / b_out[:n]).max()
    live = ~empty
    err = np.abs(m[:n] - np.where(live, ref[1][:n], 0))[live]
    assert (err <= b_lse[:n][live]).all(), "lse: %.3g times its bound" % (err / b_lse[:n][live]).max()
    assert sq.device_status() == 0


# ------------------------------------------------------------------ append


def append_case(seed, new, cached, hq, hkv, page, bits, rot, interleaved, norm, pad=0, strided=True):
    rng = np.random.default_rng(seed)
    total = [n + c for n, c in zip(new, cached)]
    pool = G.Pool(rng, total, page, hkv, bits)
    T = sum(new) + pad
    qkv = rng.standard_normal((T, hq + 2 * hkv, D)) * np.exp(rng.standard_normal((T, hq + 2 * hkv, 1)))
    qkv[:, hq:hq + hkv, ::37] *= 8
    qkv = G.round_bf16(qkv)
    t = bf16(qkv)
    q, k, v = t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cos = sin = None
    if rot:
        ang = np.arange(max(total) + 1)[:, None] * 1e6 ** (-np.arange(0, rot, 2) / rot)
        cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    w = [(1 + 0.2 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)] if norm else [None, None]
    pos = np.concatenate([c + np.arange(n) for n, c in zip(new, cached)]).astype(int)
    seq = np.repeat(np.arange(len(new)), new)
    return dict(pool=pool, T=T, n=sum(new), qkv=qkv, q=q, k=k, v=v, cos=cos, sin=sin, w=w, pos=pos, seq=seq,
                cu=np.concatenate([[0], np.cumsum(new)]).astype(np.int32), cached=np.array(cached, np.int32),
                hq=hq, hkv=hkv, bits=bits, page=page, interleaved=interleaved)


def run_append(c, pages, **kw):
    opt = lambda a: None if a is None else cu(a)  # noqa: E731
    args = dict(interleaved=c["interleaved"], q_norm=opt(c["w"][0]), k_norm=opt(c["w"][1]), eps=1e-6)
    args.update(kw)
    return sq.kv_paged_append(c["q"], c["k"], c["v"], pages, cu(c["pool"].table), cu(c["cu"]), cu(c["cached"]),
                              opt(c["cos"]), opt(c["sin"]), **args)


@pytest.mark.parametrize("new,cached,hq,hkv,page,bits,rot,interleaved,norm,pad", [
    ([1], [0], 1, 1, 16, 4, 128, False, False, 0),
    ([1, 1, 1], [15, 16, 17], 4, 1, 16, 4, 128, False, True, 2),
    ([5, 0, 33, 1], [0, 9, 31, 100], 8, 2, 32, 4, 64, False, True, 3),
    ([40, 17], [3, 0], 6, 3, 16, 8, 32, True, True, 1),
    ([9, 70], [60, 1], 7, 7, 64, 8, 96, False, False, 0),
    ([11], [5], 10, 5, 128, 4, 112, True, False, 4),
    ([130], [1000], 32, 8, 256, 4, 128, True, True, 0),
    ([6, 6], [0, 2], 8, 8, 16, 8, 0, False, True, 0),
    ([6, 6], [0, 2], 4, 2, 16, 4, 0, False, False, 0),
    ([64], [0], 256, 64, 16, 4, 16, False, True, 0),
])
def test_append_and_read_back(new, cached, hq, hkv, page, bits, rot, interleaved, norm, pad):
    c = append_case(11, new, cached, hq, hkv, page, bits, rot, interleaved, norm, pad)
    pages = pages_of(c["pool"])
    before = {k: getattr(pages, k).clone() for k in c["pool"].arrays}
    q_out = torch.full((c["T"], hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    assert run_append(c, pages, q_out=q_out) is q_out
    n, x = c["n"], c["qkv"][:c["n"]]
    # queries: float32 norm, rotary map and butterflies.  Each of the 128 terms of an output takes part in
    # at most 14 float32 operations, each off by 2^-24 of the vector's 1-norm / sqrt(128); then bf16
    ref = O.head_forward(x[:, :hq], c["w"][0], 1e-6, c["pos"], c["cos"], c["sin"], interleaved)
    got = q_out.double().cpu().numpy()
    size = np.abs(O.rope_part(O.rms_norm(x[:, :hq], c["w"][0], 1e-6), c["pos"], None, None, False)).sum(-1, keepdims=True)
    bound = 2.0 ** -8 * np.abs(ref) + 14 * 2.0 ** -24 * 2 * size / np.sqrt(D) + 1e-30
    assert (np.abs(got[:n] - ref) <= bound).all()
    assert (got[n:] == 7).all()
    # caches: the exact rotation rounded once to float32, then the contiguous caches' rule
    k = O.head_forward(x[:, hq:hq + hkv], c["w"][1], 1e-6, c["pos"], c["cos"], c["sin"], interleaved).astype(np.float32)
    page_of, row = c["pool"].table[c["seq"], c["pos"] // page], c["pos"] % page
    touched = np.zeros((pages.num_pages, page), bool)
    touched[page_of, row] = True
    back = sq.kv_paged_dequant(pages, cu(c["pool"].table), cu(c["cu"]), cu(c["cached"]), c["T"],
                               k_out=torch.full((c["T"], hkv, D), 7.0, dtype=torch.bfloat16, device="cuda"),
                               v_out=torch.full((c["T"], hkv, D), 7.0, dtype=torch.bfloat16, device="cuda"))
    for key, val, rb in (("k", k, back[0]), ("v", x[:, hq + hkv:].astype(np.float32), back[1])):
        codes, scale, zero, v = G.quantize(val, bits)
        raw = getattr(pages, key + "_codes").cpu().numpy()[page_of, :, row]
        mine = O.unpack_int4(raw, signed=False) if bits == 4 else raw
        P.check_codes(mine, codes, v, key)
        got_s = getattr(pages, key + "_scale").cpu().numpy()[page_of, :, row]
        got_z = getattr(pages, key + "_zero").cpu().numpy()[page_of, :, row]
        P.check_scales(got_s, scale)
        assert np.array_equal(got_z, zero)
        # read-back: one float32 product of exact factors, then bf16: the exact rounding but at double ties
        want = torch.from_numpy((mine.astype(np.float32) - got_z[..., None].astype(np.float32)) * got_s[..., None])
        assert torch.equal(rb[:n].cpu(), want.to(torch.bfloat16))
        assert (rb[n:] == 7).all()
        # nothing else in the pool moved
        for part in ("_codes", "_scale", "_zero"):
            a, b = getattr(pages, key + part).cpu().numpy(), before[key + part].cpu().numpy()
            keep = ~np.broadcast_to(touched[:, None, :], a.shape[:3])
            assert np.array_equal(a[keep], b[keep], equal_nan=part == "_scale")
    assert sq.device_status() == 0


def test_append_matches_the_contiguous_cache():
    """Without a norm and with the whole head rotated, the codes are those of kv_rotate_quant, bit for bit."""
    c = append_case(12, [200], [0], 32, 8, 64, 4, 128, False, False, strided=False)
    pages = pages_of(c["pool"])
    q_out = run_append(c, pages)
    ref = sq.kv_rotate_quant(c["q"], c["k"], c["v"], cu(c["pos"].astype(np.int32)), cu(c["cos"]), cu(c["sin"]))
    t, r = c["pool"].table[0, c["pos"] // 64], c["pos"] % 64
    for key in ("k", "v"):
        assert torch.equal(getattr(pages, key + "_codes")[t, :, r], ref[key + "_cache"])
        assert torch.equal(getattr(pages, key + "_scale")[t, :, r], ref[key + "_scale"])
        assert torch.equal(getattr(pages, key + "_zero")[t, :, r], ref[key + "_zero"])
    assert torch.allclose(q_out.float(), ref["q_out"].float(), rtol=2.0 ** -7, atol=2.0 ** -16)


def test_append_reports_what_is_out_of_range():
    c = append_case(13, [4, 4, 4], [0, 0, 0], 4, 2, 16, 4, 128, False, False)
    pages = pages_of(c["pool"])
    ok = {k: v.copy() for k, v in (("table", c["pool"].table), ("cu", c["cu"]), ("cached", c["cached"]))}

    def call(**bad):
        a = {**ok, **bad}
        q_out = torch.full((c["T"], 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
        sq.kv_paged_append(c["q"], c["k"], c["v"], pages, cu(a["table"]), cu(a["cu"]), cu(a["cached"]),
                           cu(c["cos"]), cu(c["sin"]), q_out=q_out)
        assert sq.device_status() == 1          # SQ_ERR_INVALID_ARG
        return (q_out == 7).all(-1).all(-1).cpu().numpy()

    table = ok["table"].copy()
    table[1, 0] = pages.num_pages
    assert call(table=table).tolist() == [False] * 4 + [True] * 4 + [False] * 4
    table[1, 0] = -1
    assert call(table=table).tolist() == [False] * 4 + [True] * 4 + [False] * 4
    assert call(cached=np.array([0, -3, 0], np.int32)).tolist() == [False] * 4 + [True] * 4 + [False] * 4
    width = 16 * ok["table"].shape[1]
    got = call(cached=np.array([0, width - 2, 0], np.int32), table=np.zeros_like(ok["table"]))
    assert got.tolist() == [False] * 4 + [True] * 4 + [False] * 4      # positions behind the rope tables
    got = call(cu=np.array([0, 4, 3, 12], np.int32))
    assert got[:3].tolist() == [False] * 3


# --------------------------------------------------------------- attention


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new,own,hq,hkv,page", [
    ([1], [1], 4, 1, 16),
    ([1], [16], 1, 1, 16),
    ([1, 1, 1, 1], [17, 64, 65, 300], 8, 2, 16),
    ([1] * 9, [1, 2, 15, 31, 33, 63, 127, 128, 129], 32, 8, 32),
    ([1, 1], [1500, 700], 14, 2, 64),               # 7 query heads per KV head
    ([1, 1], [333, 90], 16, 1, 16),                 # 16
    ([1], [200], 48, 1, 256),                       # more rows than one block
    ([2, 0, 3, 1], [2, 40, 100, 7], 8, 2, 16),      # drafts beside an idle sequence
    ([5, 8], [5, 400], 4, 4, 32),
    ([40, 17], [40, 90], 8, 2, 16),                 # whole prompts and chunks
    ([3, 2], [1, 0], 4, 2, 16),                     # fewer cached tokens than new ones: empty rows
])
def test_attention(new, own, hq, hkv, page, bits):
    prob = G.Attention(21, new, own, hq, hkv, page, bits, pad=2)
    check(prob, *attend(prob))


@pytest.mark.parametrize("rule", [
    dict(softcap=20.0), dict(softcap=0.5), dict(window=1), dict(window=33), dict(slopes=True),
    dict(scale=0.31), dict(scale=-0.1), dict(scale=0.0), dict(softcap=30.0, window=70, slopes=True),
    dict(window=1 << 30)])
@pytest.mark.parametrize("prefix", [0, 45])
def test_score_rules(rule, prefix):
    prob = G.Attention(22, [1, 4, 20], [150, 81, 20], 8, 2, 16, 4, prefix=prefix, pad=1, **rule)
    check(prob, *attend(prob))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("prefix,new,own,hq,hkv,page", [
    (1, [1], [1], 4, 1, 16),
    (64, [1, 1], [0, 5], 8, 2, 16),                 # a sequence with nothing of its own but the prefix
    (129, [1] * 7, [1, 2, 3, 16, 17, 64, 65], 32, 8, 32),
    (700, [2, 5, 1], [2, 30, 200], 14, 2, 64),
    (50, [30, 3], [30, 100], 8, 2, 16),
])
def test_prefix(prefix, new, own, hq, hkv, page, bits):
    prob = G.Attention(23, new, own, hq, hkv, page, bits, prefix=prefix, pad=1)
    check(prob, *attend(prob))


@pytest.mark.parametrize("kw", [dict(k_size=30.0, q_size=4.0), dict(k_size=1e-3, q_size=1e-3),
                                dict(v_size=1e4), dict(v_size=1e-6), dict(q_size=1e4, k_size=1e-4)])
def test_sizes_of_values(kw):
    prob = G.Attention(24, [1, 3], [400, 77], 8, 2, 16, 4, **kw)
    check(prob, *attend(prob))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new,own,hq,hkv,page", [
    ([129], [129], 1, 1, 16),                       # the second half's first row
    ([257], [300], 1, 1, 16),                       # the second block's
    ([200, 130], [200, 500], 8, 2, 64),
    ([33], [3000], 16, 2, 128),                     # keys of a few rows, split
    ([1, 64, 2, 5, 0], [50, 64, 900, 5, 77], 8, 2, 32),     # both kernels in one call
    ([300, 41, 500], [1200, 41, 640], 6, 1, 256),
    ([9, 20, 70], [4, 10, 60], 4, 1, 16),           # fewer cached tokens than new ones
    ([100], [100], 128, 2, 16),                     # 64 query heads per KV head
])
def test_many_rows(new, own, hq, hkv, page, bits):
    prob = G.Attention(33, new, own, hq, hkv, page, bits, pad=3)
    check(prob, *attend(prob))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rule", [
    dict(softcap=20.0), dict(window=1), dict(window=130), dict(slopes=True), dict(scale=-0.1), dict(scale=0.0),
    dict(softcap=30.0, window=300, slopes=True), dict(v_size=1e4), dict(v_size=1e-6), dict(k_size=30.0, q_size=4.0),
    dict(q_size=1e4, k_size=1e-4)])
@pytest.mark.parametrize("prefix", [0, 200])
def test_many_rows_score_rules(rule, prefix, bits):
    prob = G.Attention(34, [150, 40], [520, 40], 8, 2, 16, bits, prefix=prefix, pad=1, **rule)
    check(prob, *attend(prob))


@pytest.mark.parametrize("rule", [{}, dict(softcap=20.0), dict(window=700), dict(slopes=True)])
@pytest.mark.parametrize("prefix,batch,new,page,bits", [
    (1000, 3, 1, 16, 4), (129, 40, 1, 32, 8), (1500, 70, 1, 64, 4), (300, 9, 8, 16, 8), (128, 5, 32, 64, 4)])
def test_prefix_of_a_batch(prefix, batch, new, page, bits, rule):
    own = [new + (7 * b) % 90 for b in range(batch)]
    count = [max(0, new - b % 3) for b in range(batch)]
    prob = G.Attention(35, count, own, 8, 2, page, bits, prefix=prefix, pad=2, **rule)
    check(prob, *attend(prob))


@pytest.mark.parametrize("rule", [{}, dict(softcap=20.0), dict(window=700), dict(slopes=True), dict(v_size=1e4)])
@pytest.mark.parametrize("prefix,batch,new,hq,hkv,page,bits", [
    (1000, 160, 1, 8, 4, 16, 4),                    # two blocks of rows per KV head
    (1793, 40, 8, 16, 4, 64, 8),                    # five, of ragged drafts
    (3001, 24, 17, 8, 2, 32, 4)])                   # more rows than the streaming kernel takes by itself
def test_prefix_read_once(prefix, batch, new, hq, hkv, page, bits, rule):
    """Batches whose prefix is long enough for a pass of its own, on any device of at least 148 SMs' worth
    of streaming tiles (30 an SM)."""
    own = [new + (11 * b) % 50 for b in range(batch)]
    count = [max(0, new - b % 3) for b in range(batch)]
    rows = new * hq // hkv
    per = 4 if rows <= 4 else 8 if rows <= 8 else 16
    assert batch * -(-rows // per) * hkv * -(-prefix // 128) >= 30 * 148
    prob = G.Attention(39, count, own, hq, hkv, page, bits, prefix=prefix, pad=2, **rule)
    check(prob, *attend(prob))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new,own,hq,hkv,page", [
    ([5, 8, 1, 0], [300, 200, 90, 5], 16, 4, 16),   # 20 and 32 rows: two units of 16
    ([1] * 40, [(37 * i) % 900 for i in range(40)], 8, 8, 16),       # more units than CTAs: ragged pieces
    ([1] * 60, [(13 * i) % 40 for i in range(60)], 32, 8, 32),       # units of one tile or none
    ([1, 1], [2000, 1], 256, 64, 128),
    ([1], [700], 256, 1, 64),                       # 256 rows for one token
])
def test_units(new, own, hq, hkv, page, bits):
    prob = G.Attention(40, new, own, hq, hkv, page, bits, pad=1)
    check(prob, *attend(prob))


def problems_of_all_kinds():
    """One of each path: split streaming, units in pieces, split tiles, tiles, both kernels, a prefix in line,
    a prefix in a pass of its own."""
    return [G.Attention(41, [1, 1], [5000, 70], 4, 1, 64, 4), G.Attention(42, [1] * 40, [200 + i for i in range(40)], 8, 8, 16, 8),
            G.Attention(43, [40], [2500], 8, 2, 64, 4), G.Attention(44, [300, 200], [300, 500], 8, 2, 32, 8),
            G.Attention(45, [1, 90], [800, 90], 8, 2, 16, 4), G.Attention(46, [1, 3], [20, 90], 8, 2, 16, 8, prefix=300),
            G.Attention(47, [1] * 160, [1 + i % 30 for i in range(160)], 8, 4, 16, 4, prefix=1000)]


def test_calls_of_all_kinds_share_a_workspace():
    """One stream's calls use one workspace: what each leaves in it is what the next expects, in any order."""
    probs = problems_of_all_kinds()
    pages = [pages_of(p.pool) for p in probs]
    first = [attend(p, g) for p, g in zip(probs, pages)]
    rng = np.random.default_rng(48)
    for i in rng.integers(0, len(probs), 60):
        out, lse = attend(probs[i], pages[i])
        n = sum(probs[i].new)
        assert torch.equal(out[:n], first[i][0][:n]) and torch.equal(lse[:n], first[i][1][:n])
    assert sq.device_status() == 0


def test_two_streams_at_once():
    probs = problems_of_all_kinds()
    pages = [pages_of(p.pool) for p in probs]
    first = [attend(p, g)[0] for p, g in zip(probs, pages)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for k in range(20):
        with torch.cuda.stream(streams[k & 1]):
            i = (3 * k + k // 2) % len(probs)
            got.append((i, attend(probs[i], pages[i])[0]))
    torch.cuda.synchronize()
    for i, out in got:
        n = sum(probs[i].new)
        assert torch.equal(out[:n], first[i][:n])


def test_captured_calls_of_all_kinds_side_by_side():
    probs = problems_of_all_kinds()
    held, eager = [], []
    for p in probs:
        pages, q = pages_of(p.pool), bf16(p.q)
        args = (cu(p.table()), cu(p.cu), cu(np.array(p.own, np.int32)), max(p.new))
        if p.prefix:
            table = cu(p.prefix_table())
            call = lambda out, a=args, g=pages, q=q, t=table, n=p.prefix: sq.kv_prefix_attention(q, g, t, n, *a, out=out)  # noqa: E731
        else:
            call = lambda out, a=args, g=pages, q=q: sq.kv_paged_attention(q, g, *a, out=out)  # noqa: E731
        out = torch.zeros_like(q)
        call(out)
        eager.append(out.clone())
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            call(out)
        held.append((graph, out, call))
    streams = [torch.cuda.Stream() for _ in probs]
    for _ in range(5):
        for (graph, out, _), s in zip(held, streams):
            with torch.cuda.stream(s):
                out.zero_()
                graph.replay()
    torch.cuda.synchronize()
    for (_, out, _), e in zip(held, eager):
        assert torch.equal(out, e)


def test_a_first_call_may_be_captured():
    """In a process that has made no call yet: nothing that the first call sets up is in the way of capture."""
    code = """
import torch, rotation_ptq_b200 as sq
pages = sq.KVPages.empty(64, 16, 2, 4)
table = torch.arange(64, dtype=torch.int32, device="cuda").view(2, 32)
q = torch.randn(41, 8, 128, device="cuda").bfloat16()
kv = q[:, :2].contiguous()
cu = torch.tensor([0, 1, 41], dtype=torch.int32, device="cuda")
cached, lengths = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([300, 60], [301, 100]))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    r = sq.kv_paged_append(q, kv, kv, pages, table, cu, cached)
    out = sq.kv_paged_attention(r, pages, table, cu, lengths, 40)
g.replay()
torch.cuda.synchronize()
want = sq.kv_paged_attention(r, pages, table, cu, lengths, 40)
assert torch.equal(out, want) and out.isfinite().all() and sq.device_status() == 0
"""
    root = pathlib.Path(__file__).resolve().parents[1]
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_among_the_linear_layers():
    """Attention calls and linear layers one behind the other without a gap, as in a model's step: kernels that
    hold tensor memory and programmatic dependents in both orders."""
    probs = problems_of_all_kinds()
    pages = [pages_of(p.pool) for p in probs]
    first = [attend(p, g)[0] for p, g in zip(probs, pages)]
    rng = np.random.default_rng(53)
    N, K = 512, 1024
    w_q, w_s = cu(rng.integers(0, 256, (N, K // 2)).astype(np.uint8)), cu(rng.random(N).astype(np.float32))
    layers = []
    for M in (1, 16, 300):
        a_q, a_s = cu(rng.integers(0, 256, (M, K // 2)).astype(np.uint8)), cu(rng.random(M).astype(np.float32))
        layers.append((a_q, a_s, sq.w4a4_linear(a_q, a_s, w_q, w_s)))
    torch.cuda.synchronize()
    calls = []
    for p, g in zip(probs, pages):
        q = bf16(p.q)
        args = (cu(p.table()), cu(p.cu), cu(np.array(p.own, np.int32)), max(p.new))
        table = cu(p.prefix_table()) if p.prefix else None
        calls.append((p, g, q, args, table))
    torch.cuda.synchronize()
    got, lin = [], []
    for k in range(60):
        i = int(rng.integers(0, len(calls)))
        p, g, q, args, table = calls[i]
        if p.prefix:
            got.append((i, sq.kv_prefix_attention(q, g, table, p.prefix, *args)))
        else:
            got.append((i, sq.kv_paged_attention(q, g, *args)))
        j = int(rng.integers(0, len(layers)))
        lin.append((j, sq.w4a4_linear(layers[j][0], layers[j][1], w_q, w_s)))
    torch.cuda.synchronize()
    for i, out in got:
        n = sum(probs[i].new)
        assert torch.equal(out[:n], first[i][:n])
    for j, out in lin:
        assert torch.equal(out, layers[j][2])
    assert sq.device_status() == 0


def test_pages_of_several_sequences():
    """Two sequences that begin with the same pages (a copied table): both read them."""
    prob = G.Attention(49, [1, 1], [100, 100], 8, 2, 16, 4)
    prob.pool.table[1, :5] = prob.pool.table[0, :5]
    for key in "kv":
        prob.values[key, 1] = np.concatenate([prob.values[key, 0][:80], prob.values[key, 1][80:]])
    check(prob, *attend(prob))


def test_pool_past_32_bit_offsets():
    """The same rows in a small pool and behind 4 GB of pages give the same bits."""
    hq, hkv, page, bits, n = 8, 8, 4096, 8, 1040                      # 1040 x 4 MB of codes each
    rng = np.random.default_rng(50)
    T = 300
    x = bf16(G.round_bf16(rng.standard_normal((T, hq + 2 * hkv, D))))
    outs = []
    for total, use in ((3, [2, 0]), (n, [n - 1, n - 2])):
        pages = sq.KVPages.empty(total, page, hkv, bits)
        table = cu(np.array([use], np.int32))
        cached = cu(np.array([page - 150], np.int32))
        c = cu(np.array([0, T], np.int32))
        q = sq.kv_paged_append(x[:, :hq], x[:, hq:2 * hq], x[:, 2 * hq:], pages, table, c, cached)
        lengths = cu(np.array([page - 150 + T], np.int32))
        args = dict(window=T)                                         # some rows in front, which hold zeros
        many = sq.kv_paged_attention(q, pages, table, c, lengths, T, **args)
        one = sq.kv_paged_attention(q[-1:], pages, table, cu(np.array([0, 1], np.int32)), lengths, 1, **args)
        back = sq.kv_paged_dequant(pages, table, c, cached, T)
        outs.append((many, one) + back)
    assert sq.device_status() == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert outs[1][0].abs().max() > 0


@pytest.mark.parametrize("new,own", [([1], [300]), ([64], [300])])
def test_rows_that_hold_zeros(new, own):
    """Rows of a fresh pool (scale 0) stand for zeros: keys score 0 and values add nothing, whole tiles of them
    in front of the first others too."""
    prob = G.Attention(51, new, own, 4, 1, 16, 4)
    for key in "kv":
        for pos in range(200):
            at = prob.pool.table[0, pos // 16], slice(None), pos % 16
            for part in ("_codes", "_scale", "_zero"):
                prob.pool.arrays[key + part][at] = 0
        prob.values[key, 0][:200] = 0
    check(prob, *attend(prob))


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e20, 1e30, 1e36])
@pytest.mark.parametrize("new", [1, 64])
def test_value_scales_at_the_ends(new, size):
    prob = G.Attention(52, [new], [300], 4, 1, 16, 4, v_size=size)
    check(prob, *attend(prob))


def test_many_rows_split_and_repeat():
    prob = G.Attention(36, [40, 3], [2500, 9], 8, 2, 64, 4)
    a = attend(prob)
    check(prob, *a)
    b = attend(prob)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(prob, *attend(prob, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")))


def test_waits_that_give_up_are_reported():
    """Every wait of the tile kernel gives up at once: the call ends, reports, and the next one is right."""
    prob = G.Attention(37, [40], [400], 8, 2, 64, 4)
    sq.lib.sq_debug_set_spin_limit(0xFFFFFFFF)
    try:
        attend(prob)
        assert sq.device_status() == 5               # SQ_ERR_TIMEOUT
    finally:
        sq.lib.sq_debug_set_spin_limit(0)
    check(prob, *attend(prob))


def test_many_rows_hidden_infinities_do_not_leak():
    prob = G.Attention(38, [64], [200], 4, 1, 16, 4)
    ref = prob.reference()
    pages = pages_of(prob.pool)
    page, row = prob.table()[0, 199 // 16], 199 % 16
    for bad, keys in ((float("inf"), "kv"), (float("nan"), "kv"), (float("nan"), "v"), (float("inf"), "v")):
        for key in "kv":
            getattr(pages, key + "_scale")[page, :, row] = bad if key in keys else 0.5
        out, lse = attend(prob, pages)
        b_out, b_lse = prob.bounds(ref, TILE_EPS, TILE_STEP)
        o, m = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (np.abs(o[:63] - ref[0][:63]) <= b_out[:63]).all()
        assert (np.abs(m[:63] - ref[1][:63]) <= b_lse[:63]).all()
        if keys == "v":
            assert not np.isfinite(o[63]).any()


def test_long_cache_splits_and_is_repeatable():
    prob = G.Attention(25, [1, 1], [9000, 5], 4, 1, 128, 4)
    a = attend(prob)
    check(prob, *a)
    b = attend(prob)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # unsplit (no workspace worth the name): the same but for the order of sums
    c = attend(prob, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    check(prob, *c)


def test_strided_queries_and_other_stream():
    prob = G.Attention(26, [1, 2], [100, 60], 8, 2, 16, 4)
    wide = torch.zeros((prob.T, 12, D), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = bf16(prob.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = attend(prob, q=wide[:, 2:10])
    side.synchronize()
    check(prob, *got)


def test_hidden_infinities_do_not_leak():
    """A later key's infinite or NaN scale is no business of earlier rows."""
    prob = G.Attention(27, [6], [80], 4, 1, 16, 4)
    ref = prob.reference()
    pages = pages_of(prob.pool)
    page, row = prob.table()[0, 79 // 16], 79 % 16
    for bad, keys in ((float("inf"), "kv"), (float("nan"), "kv"), (float("nan"), "v"), (float("inf"), "v")):
        for key in "kv":
            getattr(pages, key + "_scale")[page, :, row] = bad if key in keys else 0.5
        out, lse = attend(prob, pages)
        b_out, b_lse = prob.bounds(ref, STREAM_EPS)
        o, m = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert (np.abs(o[:5] - ref[0][:5]) <= b_out[:5]).all()
        assert (np.abs(m[:5] - ref[1][:5]) <= b_lse[:5]).all()
        if keys == "v":                                # a visible key's scale, under finite scores
            assert not np.isfinite(o[5]).any()


def test_attention_reports_what_is_out_of_range():
    prob = G.Attention(28, [1, 1, 1], [20, 30, 40], 4, 2, 16, 4)
    pages, q = pages_of(prob.pool), bf16(prob.q)
    good = attend(prob, pages)[0]

    def call(table=None, cu_=None, lengths=None):
        out = torch.full((3, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
        sq.kv_paged_attention(q, pages, cu(prob.table() if table is None else table),
                              cu(prob.cu if cu_ is None else cu_),
                              cu(np.array(prob.own if lengths is None else lengths, np.int32)), 1, out=out)
        assert sq.device_status() == 1
        return out

    for bad in (-1, 16 * prob.table().shape[1] + 1):
        out = call(lengths=[20, bad, 40])
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and (out[1] == 0).all()
    table = prob.table().copy()
    table[1, :] = -1
    out = call(table=table)
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and (out[1] == 0).all()
    out = call(cu_=np.array([0, 1, 2, 9], np.int32))                  # rows behind the batch
    assert torch.equal(out[:2], good[:2]) and (out[2] == 7).all()


def test_two_graphs_replay_side_by_side():
    """Captured calls carry their own workspaces; lengths are read at replay."""
    probs = [G.Attention(29, [1, 1], [3000, 20], 4, 1, 64, 4), G.Attention(30, [1], [2500], 4, 1, 64, 8)]
    eager, graphs, held = [], [], []
    for p in probs:
        pages, q = pages_of(p.pool), bf16(p.q)
        args = (cu(p.table()), cu(p.cu), cu(np.array(p.own, np.int32)), 1)
        eager.append(sq.kv_paged_attention(q, pages, *args).clone())
        out = torch.empty_like(q)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            sq.kv_paged_attention(q, pages, *args, out=out)
        graphs.append((g, out))
        held.append((pages, q, args))
    streams = [torch.cuda.Stream() for _ in probs]
    for _ in range(20):
        for (g, out), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
    torch.cuda.synchronize()
    for (g, out), e in zip(graphs, eager):
        assert torch.equal(out, e)
    # a shorter sequence at the next replay
    held[0][2][2][0] = 1000
    graphs[0][0].replay()
    torch.cuda.synchronize()
    want = sq.kv_paged_attention(held[0][1], held[0][0], *held[0][2])
    assert torch.equal(graphs[0][1], want)


# --------------------------------------------------- the calls one after another


@pytest.mark.parametrize("bits", [4, 8])
def test_prompt_then_steps(bits):
    """A prompt in two chunks, then single tokens: every call's attention equals the oracle's over what the
    cache then holds, and the whole cache reads back."""
    rng = np.random.default_rng(31)
    hq, hkv, page, lens = 8, 2, 16, [37, 20]
    B, longest = 2, 64
    pages = sq.KVPages.empty(12, page, hkv, bits)
    table = rng.permutation(12)[:B * 4].reshape(B, 4).astype(np.int32)
    ang = np.arange(longest)[:, None] * 1e4 ** (-np.arange(0, D, 2) / D)
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    w = (1 + 0.1 * rng.standard_normal(D)).astype(np.float32)
    cached = np.zeros(B, np.int32)
    for new in ([30, 20], [7, 0], [1, 1], [1, 1]):
        T = sum(new)
        x = G.round_bf16(rng.standard_normal((T, hq + 2 * hkv, D)))
        t = bf16(x)
        c = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q = sq.kv_paged_append(t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:], pages, cu(table), cu(c), cu(cached),
                               cu(cos), cu(sin), q_norm=cu(w), k_norm=cu(w))
        cached = (cached + np.array(new)).astype(np.int32)
        out = sq.kv_paged_attention(q, pages, cu(table), cu(c), cu(cached), max(new))
        whole = np.concatenate([[0], np.cumsum(cached)]).astype(np.int32)
        k, v = sq.kv_paged_dequant(pages, cu(table), cu(whole), cu(np.zeros(B, np.int32)), int(cached.sum()))
        k, v, qn = (a.double().cpu().numpy() for a in (k, v, q))
        for b in range(B):
            rows, own = slice(c[b], c[b + 1]), slice(whole[b], whole[b + 1])
            ref, _, spread, size = O.causal_attention(qn[rows], k[own], v[own],
                                                   np.arange(cached[b] - new[b], cached[b]), np.arange(cached[b]))
            # the read-back rounds keys and values to bf16, by 2^-8 of each: a score moves by 2^-8 size at
            # most, a weight by that part of itself, and the output's quotient by twice that and 2^-8
            err = np.abs(out[rows].double().cpu().numpy() - ref)
            assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * (2 * size + 1) * spread).all()
    assert cached.tolist() == [39, 22] and sq.device_status() == 0
