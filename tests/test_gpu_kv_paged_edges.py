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
@pytest.mark.parametrize("factor", [1e9, 1e20, 1e30])
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
