"""The paged calls where they meet something else: host threads on one stream, values and scales at the
ends of their range, prefixes under a window, and the bounds of the kernel that serves each sequence."""
import threading

import numpy as np
import pytest
import torch

import rotation_ptq_b200 as sq
from tests import paged as G
from tests.test_gpu_kv_paged import attend, bf16, cu, pages_of, problems_of_all_kinds

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
