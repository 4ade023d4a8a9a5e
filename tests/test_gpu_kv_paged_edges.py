"""The paged calls where they meet something else: host threads on one stream, values and scales at the
ends of their range, prefixes under a window, and the bounds of the kernel that serves each sequence."""
import threading

import numpy as np
import pytest
import torch

import rotation_ptq_b200 as sq
from tests import paged as G
from tests.test_gpu_kv_paged import STREAM_EPS, TILE_EPS, TILE_STEP, attend, bf16, check, cu, pages_of, problems_of_all_kinds

pytestmark = pytest.mark.gpu


def staged(prob):
    """A call of the problem that copies nothing: everything is on the device before."""
    pages, q = pages_of(prob.pool), bf16(prob.q)
    args = (cu(prob.table()), cu(prob.cu), cu(np.array(prob.own, np.int32)), max(prob.new))
    if not prob.prefix:
        return lambda: sq.kv_paged_attention(q, pages, *args, **prob.rule)
    table = cu(prob.prefix_table())
    return lambda: sq.kv_prefix_attention(q, pages, table, prob.prefix, *args, **prob.rule)


def test_host_threads_share_a_stream():
    """Threads whose calls go to one stream and share its workspace: a call behind a prefix launches two
    kernels, and no other thread's call comes between them."""
    probs = problems_of_all_kinds()
    calls = [staged(p) for p in probs]
    first = [c() for c in calls]
    torch.cuda.synchronize()
    got = [[] for _ in range(4)]
    start = threading.Barrier(len(got))

    def work(k):
        rng = np.random.default_rng(60 + k)
        # every other call is the one with a prefix pass of its own
        order = [len(calls) - 1 if j & 1 else int(rng.integers(0, len(calls))) for j in range(80)]
        start.wait()
        for i in order:
            got[k].append((i, calls[i]()))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(got))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [len(g) for g in got] == [80] * len(got)
    for i, out in (x for g in got for x in g):
        n = sum(probs[i].new)
        assert torch.equal(out[:n], first[i][:n])
    assert sq.device_status() == 0


def scale_key(prob, pos, factor):
    """Multiplies the value scale of sequence 0's key at `pos`; prob.values keeps what it was."""
    at = prob.pool.table[0, pos // prob.pool.page], slice(None), pos % prob.pool.page
    prob.pool.arrays["v_scale"][at] *= np.float32(factor)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("factor", [1e9, 1e20, 1e30, 1e38])
@pytest.mark.parametrize("new,own,window,pos", [
    (6, 80, 0, 79),                                 # streaming kernel: a later token's key
    (6, 80, 10, 65),                                # one that only the first token still sees
    (1, 300, 100, 196),                             # one that the window has left behind, beside visible keys
    (64, 200, 0, 199),                              # tile kernel: the same three
    (64, 200, 10, 130),
    (64, 400, 100, 236),
])
def test_hidden_value_scales_take_no_precision(new, own, window, pos, factor, bits):
    """A key's value scale, however large, is no business of the rows from which it is hidden: their results
    keep the bounds of what they see."""
    prob = G.Attention(61, [new], [own], 4, 1, 16, bits, window=window)
    ref = prob.reference()
    tile = new * 4 > 32
    b_out, b_lse = prob.bounds(ref, *((TILE_EPS, TILE_STEP) if tile else (STREAM_EPS,)))
    scale_key(prob, pos, factor)
    out, lse = attend(prob)
    dist = own - new + np.arange(new) - pos
    blind = (dist < 0) | ((dist >= window) if window else False)
    assert blind.any()
    o, m = out.double().cpu().numpy(), lse.double().cpu().numpy()
    err = np.abs(o - ref[0])[blind] / b_out[blind]
    assert (err <= 1).all(), "out: %.3g times its bound" % err.max()
    assert (np.abs(m - ref[1]) <= b_lse).all()
    assert np.isfinite(o).all() and sq.device_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rule", [{}, dict(softcap=20.0), dict(slopes=True), dict(scale=-0.1), dict(window=20)])
@pytest.mark.parametrize("q_size,k_size", [(3e36, 3e-37), (1e38, 1e-37), (1e-36, 1e30), (1e5, 1e-36)])
@pytest.mark.parametrize("new", [1, 3, 64])
def test_queries_at_the_ends(new, q_size, k_size, rule, bits):
    """Queries up to bf16's end over keys that leave their scores moderate."""
    prob = G.Attention(62, [new], [200], 4, 1, 16, bits, q_size=q_size, k_size=k_size, **rule)
    prob.q = G.round_bf16(np.clip(prob.q, -3.3e38, 3.3e38))      # (the oracle gets what the kernel gets)
    check(prob, *attend(prob))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rule", [{}, dict(slopes=True), dict(scale=-0.1), dict(window=20)])
@pytest.mark.parametrize("q_size,k_size", [(1e4, 1e3), (1e4, 1e5), (1e9, 1e6), (1e20, 1e10), (1.0, 1e28)])
@pytest.mark.parametrize("new", [1, 3, 64])
def test_scores_far_past_the_exponential(new, q_size, k_size, rule, bits):
    """Scores so large that float32 holds them in steps of many: a row is still an average of its visible
    values, and its log sum is its largest score's."""
    prob = G.Attention(63, [new], [200], 4, 1, 16, bits, q_size=q_size, k_size=k_size, **rule)
    out, lse = attend(prob)
    check(prob, out, lse)
    o = out.double().cpu().numpy()
    for i in range(new):
        at = 200 - new + i
        seen = prob.values["v", 0][max(0, at + 1 - (rule.get("window") or 200)):at + 1, 0]
        # weights (11 bits) and their sum's rounding, and bf16's
        slack = (2.0 ** -8 + 2.0 ** -9) * np.abs(seen).max()
        assert (o[i] <= seen.max(0) + slack).all() and (o[i] >= seen.min(0) - slack).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("window,in_a_pass", [(0, True), (100, False), (2500, True)])
def test_prefix_under_a_window(window, in_a_pass, bits):
    """A prefix is read once for the batch by what the window leaves of it: a short window's few keys are
    streamed with each sequence's own, and a pass begins where the first token's window does - here that of a
    sequence with fewer cached tokens than new ones."""
    batch = 150
    count = [1] * batch
    own = [1 + b % 40 for b in range(batch)]
    count[7], own[7] = 8, 2
    prob = G.Attention(64, count, own, 8, 4, 32, bits, prefix=4000, window=window, pad=1)
    need = sq.kv_attention_workspace_bytes(prob.T, 8, pages_of(prob.pool), batch, prob.table().shape[1], 8, 4000)
    workspace = torch.zeros(need, dtype=torch.uint8, device="cuda")
    got = attend(prob, workspace=workspace)
    check(prob, *got)
    # the pass leaves its results behind what streaming alone uses
    alone = sq.kv_attention_workspace_bytes(prob.T, 8, pages_of(prob.pool), batch, prob.table().shape[1], 8)
    assert bool(workspace[alone:].any()) == in_a_pass
    again = attend(prob, workspace=workspace)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def check_as_served(prob, out, lse):
    """check(), with each row's bounds those of the kernel that serves its sequence: up to 32 rows (new tokens x
    query heads per KV head) of a sequence are streamed, more go to the tile kernel, and so do all rows over a
    prefix whose streaming tiles come to 30 an SM while no sequence has more than 128 rows."""
    group, few = prob.hq // prob.hkv, 32
    rows = max(prob.new) * group
    per = 4 if rows <= 4 else 8 if rows <= 8 else 16
    seen = min(prob.prefix, prob.rule["window"] + max(prob.new)) if prob.rule["window"] else prob.prefix
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    in_a_pass = len(prob.new) > 1 and prob.prefix and rows <= 128 and \
        len(prob.new) * -(-rows // per) * prob.hkv * -(-seen // 128) >= 30 * sms
    tile = np.repeat([bool(in_a_pass) or n * group > few for n in prob.new], prob.new)
    ref = prob.reference()
    wide, narrow = prob.bounds(ref, TILE_EPS, TILE_STEP), prob.bounds(ref, STREAM_EPS)
    n = sum(prob.new)
    b_out = np.where(tile[:, None, None], wide[0][:n], narrow[0][:n])
    o, m = out.double().cpu().numpy()[:n], lse.double().cpu().numpy()[:n]
    empty = np.isneginf(ref[1][:n])
    assert np.array_equal(np.isneginf(m), empty) and (o[empty] == 0).all()
    err = np.abs(o - ref[0][:n])
    assert (err <= b_out).all(), "out: %.3g times its bound" % (err / b_out).max()
    err = np.abs(m - np.where(empty, 0, ref[1][:n]))[~empty]
    assert (err <= wide[1][:n][~empty]).all()
    assert sq.device_status() == 0


SERVED = [
    dict(new=[5, 8, 1, 0], own=[300, 200, 90, 5], hq=16, hkv=4, page=16),               # 20 and 32 rows: streamed
    dict(new=[1, 1], own=[333, 90], hq=16, hkv=1, page=16),
    dict(new=[2, 1, 2], own=[700, 31, 40], hq=32, hkv=2, page=64),                      # 32 rows
    dict(new=[1, 64, 2, 5, 0], own=[50, 64, 900, 5, 77], hq=8, hkv=2, page=32),         # both kernels in one call
    dict(new=[1] * 7, own=[2, 4, 6, 16, 18, 64, 66], hq=32, hkv=8, page=32, prefix=130),        # a prefix in line
    dict(new=[2, 5, 1], own=[2, 30, 200], hq=14, hkv=2, page=64, prefix=700),
    dict(new=[1] * 160, own=[2 + 2 * (b % 30) for b in range(160)], hq=8, hkv=4, page=16, prefix=1000),     # in a pass
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kw", SERVED)
def test_bounds_of_the_kernel_that_serves(kw, bits):
    kw = dict(kw)
    prob = G.Attention(65, kw.pop("new"), kw.pop("own"), bits=bits, pad=1, **kw)
    check_as_served(prob, *attend(prob))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kw", SERVED)
def test_weights_keep_their_low_bits(kw, bits):
    """Equal scores over values that all but cancel: + x (1 + 2^-12) and - x in turn.  The streaming kernel's 22
    bits hold the difference, 2^-13 x of a row that sees pairs; 11 bits would lose all of it."""
    kw = dict(kw)
    prob = G.Attention(66, kw.pop("new"), kw.pop("own"), bits=bits, pad=1, **kw)
    prob.q[:] = 0
    x = 2.0 ** bits - 1
    for b, n in enumerate(prob.own + [prob.prefix]):
        pos = np.arange(n)
        at = prob.pool.table[b, pos // prob.pool.page], slice(None), pos % prob.pool.page
        odd = (pos & 1).astype(bool)
        prob.pool.arrays["v_codes"][at] = np.where(odd, 0, 0xFF).astype(np.uint8)[:, None, None]
        prob.pool.arrays["v_zero"][at] = np.where(odd, x, 0).astype(np.uint8)[:, None]
        prob.pool.arrays["v_scale"][at] = np.where(odd, 1.0, 1 + 2.0 ** -12).astype(np.float32)[:, None]
        value = np.where(odd, -x, x * (1 + 2.0 ** -12))
        prob.values["v", b] = np.broadcast_to(value[:, None, None], (n, prob.hkv, 128)).copy()
    check_as_served(prob, *attend(prob))


@pytest.mark.parametrize("rule", [
    dict(softcap=20.0), dict(softcap=0.5), dict(window=1), dict(window=33), dict(slopes=True),
    dict(scale=0.31), dict(scale=-0.1), dict(scale=0.0), dict(softcap=30.0, window=70, slopes=True)])
@pytest.mark.parametrize("prefix", [0, 45])
def test_score_rules_8_bits(rule, prefix):
    prob = G.Attention(67, [1, 4, 20], [150, 81, 20], 8, 2, 16, 8, prefix=prefix, pad=1, **rule)
    check_as_served(prob, *attend(prob))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rule", [{}, dict(softcap=20.0), dict(window=200, slopes=True)])
@pytest.mark.parametrize("new,own,hq,hkv", [
    ([1] * 64, [1 + (97 * b) % 1500 for b in range(64)], 48, 1),              # one 48-row token each
    ([3 + b % 6 for b in range(40)], [9 + (61 * b) % 700 for b in range(40)], 16, 1),         # 48 to 128 rows
    ([9 + 2 * b for b in range(24)], [70 + (131 * b) % 900 for b in range(24)], 8, 2),        # 36 to 220
    ([5, 30], [4000, 900], 7, 1),                                             # few of them: split
])
def test_ragged_batches_of_tile_units(new, own, hq, hkv, rule, bits):
    prob = G.Attention(68, new, own, hq, hkv, 32, bits, pad=1, **rule)
    first = attend(prob)
    check_as_served(prob, *first)
    again = attend(prob)
    n = sum(new)
    assert torch.equal(first[0][:n], again[0][:n]) and torch.equal(first[1][:n], again[1][:n])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new", [1, 20])
@pytest.mark.parametrize("rule", [{}, dict(window=60), dict(slopes=True)])
def test_append_behind_a_prefix(new, rule, bits):
    """Tokens appended behind a shared prefix, with rotary tables that begin at its length, are the tokens of a
    sequence that holds the prefix's keys in pages of its own: the same codes, and the same attention."""
    rng = np.random.default_rng(69)
    hq, hkv, page, P, own = 8, 2, 16, 77, 41
    N = P + own
    x = bf16(G.round_bf16(rng.standard_normal((N, hq + 2 * hkv, 128))))
    ang = np.arange(N)[:, None] * 1e4 ** (-np.arange(0, 128, 2) / 128)
    cos, sin = cu(np.cos(ang).astype(np.float32)), cu(np.sin(ang).astype(np.float32))
    slopes = cu((2.0 ** -np.arange(1, hq + 1)).astype(np.float32)) if rule.get("slopes") else None
    args = dict(window=rule.get("window", 0), slopes=slopes)
    i32 = lambda *a: cu(np.array(a, np.int32))  # noqa: E731
    pages = sq.KVPages.empty(24, page, hkv, bits)
    table = rng.permutation(24).astype(np.int32)
    whole, shared, mine = cu(table[None, :8]), cu(table[8:13]), cu(table[None, 13:16])

    def append(rows, table, tables):
        t = x[rows]
        return sq.kv_paged_append(t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:], pages, table, i32(0, t.shape[0]), i32(0),
                                  *tables)

    q = append(slice(0, N), whole, (cos, sin))[N - new:].contiguous()
    append(slice(0, P), shared[None], (cos, sin))
    q2 = append(slice(P, N), mine, (cos[P:].contiguous(), sin[P:].contiguous()))[own - new:].contiguous()
    assert torch.equal(q, q2)
    k, v = sq.kv_paged_dequant(pages, whole, i32(0, N), i32(0), N)
    for got, want in zip(sq.kv_paged_dequant(pages, mine, i32(0, own), i32(0), own), (k, v)):
        assert torch.equal(got, want[P:])
    lse, lse2 = (torch.zeros((new, hq), device="cuda") for _ in range(2))
    a = sq.kv_paged_attention(q, pages, whole, i32(0, new), i32(N), new, lse=lse, **args)
    b = sq.kv_prefix_attention(q2, pages, shared, P, mine, i32(0, new), i32(own), new, lse=lse2, **args)
    assert sq.device_status() == 0
    # each is off by at most 2^-8 of itself and 2 (e + eps) of the largest value (see bounds() in tests/paged.py)
    size = (q.double().abs().sum(-1).max() * k.double().abs().max() / 128 ** 0.5).item()
    slack = 2 * (2.0 ** -18 * (1 + size) + TILE_EPS) * v.double().abs().max()
    assert ((a.double() - b.double()).abs() <= 2 * (2.0 ** -8 * torch.maximum(a, b).double().abs() + slack)).all()
    assert ((lse - lse2).abs() <= 2 * 2.0 ** -18 * (1 + size)).all()


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e20, 1e30, 1e36])
@pytest.mark.parametrize("kind", ["split", "whole", "pass"])
def test_value_scales_at_the_ends_in_pieces(kind, size):
    """As partial results that are joined, as whole units, and over a prefix that is read once."""
    if kind == "pass":
        prob = G.Attention(71, [1] * 160, [1 + b % 30 for b in range(160)], 8, 4, 16, 4, prefix=1000, v_size=size)
    else:
        prob = G.Attention(71, [64, 40], [1500, 700], 4, 1, 16, 4, v_size=size)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda") if kind == "whole" else None
    check(prob, *attend(prob, workspace=ws))


@pytest.mark.parametrize("factor", [1e9, 1e20, 1e30, 1e38])
@pytest.mark.parametrize("kind", ["split", "whole", "pass"])
def test_hidden_value_scales_in_pieces(kind, factor):
    """The same for keys with large scales that only some rows see, first by the window and then no more."""
    if kind == "pass":
        prob = G.Attention(72, [1] * 160, [1 + b % 40 for b in range(160)], 8, 4, 16, 4, prefix=1200, window=1000)
        pos, b = 215, 160                          # position 215 is visible up to 1214: to own lengths up to 15
    else:
        prob = G.Attention(72, [64], [1500], 4, 1, 16, 4, window=1000)
        pos, b = 470, 0                            # visible up to 1469
    ref = prob.reference()
    b_out, b_lse = prob.bounds(ref, TILE_EPS, TILE_STEP)
    page = prob.pool.table[b, pos // 16]
    prob.pool.arrays["v_scale"][page, :, pos % 16] *= np.float32(factor)
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda") if kind == "whole" else None
    out, lse = attend(prob, workspace=ws)
    at = np.concatenate([prob.prefix + own - n + np.arange(n) for n, own in zip(prob.new, prob.own)])
    blind = at - pos >= 1000
    assert blind.any() and not blind.all()
    o, m = out.double().cpu().numpy(), lse.double().cpu().numpy()
    err = np.abs(o - ref[0])[blind] / b_out[blind]
    assert (err <= 1).all(), "out: %.3g times its bound" % err.max()
    assert (np.abs(m - ref[1]) <= b_lse).all() and np.isfinite(o).all()
    assert sq.device_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kw", [
    dict(new=[1], own=[90]), dict(new=[6], own=[80]), dict(new=[64], own=[300]), dict(new=[64], own=[300], softcap=20.0),
    dict(new=[1] * 160, own=[1 + b % 30 for b in range(160)], hq=8, hkv=4, prefix=1000)])
def test_a_query_that_is_not_finite_keeps_to_its_row(kw, bad):
    kw = dict(dict(hq=4, hkv=1), **kw)
    prob = G.Attention(73, kw.pop("new"), kw.pop("own"), bits=4, **kw)
    ref = prob.reference()
    b_out, b_lse = prob.bounds(ref, TILE_EPS, TILE_STEP)
    q = bf16(prob.q)
    row, head = prob.T // 2, 1
    q[row, head, 5] = bad
    out, lse = attend(prob, q=q)
    o, m = out.double().cpu().numpy(), lse.double().cpu().numpy()
    others = np.ones((prob.T, prob.hq), bool)
    others[row, head] = False
    assert (np.abs(o - ref[0]) <= b_out)[others].all() and (np.abs(m - ref[1]) <= b_lse)[others].all()
    if not prob.rule["softcap"]:                   # (a cap makes an infinite score a finite one)
        assert np.isnan(o[row, head]).any()
    assert sq.device_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("cap", [1e9, 1e25, 1e33, 2.9e38])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("new", [1, 5, 64])
def test_a_large_cap_is_none(new, slopes, cap, bits):
    """Scores a billion times below their cap are the scores to float32's accuracy (x - x^3 / 3 at x = 1e-8)."""
    prob = G.Attention(74, [new], [150], 4, 1, 16, bits, slopes=slopes)
    check(prob, *attend(prob, softcap=cap))


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("cap", [1e-3, 1e-20, 1e-44])
def test_a_small_cap_leaves_equal_weights(new, cap):
    """Scores of at most 1e-3 apart from zero: the weights of a row are equal to that."""
    prob = G.Attention(75, [new], [150], 4, 1, 16, 4)
    out, lse = attend(prob, softcap=cap)
    prob.rule["scale"] = 0.0
    ref = prob.reference()
    b_out, b_lse = prob.bounds(ref, TILE_EPS + 2 * cap, TILE_STEP)
    o, m = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(o - ref[0]) <= b_out).all() and (np.abs(m - ref[1]) <= b_lse + cap).all()
