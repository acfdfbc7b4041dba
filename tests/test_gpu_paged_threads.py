"""Paged attention called by several Python threads at once (the binding gives up the interpreter's lock)."""
import threading

import pytest
import torch

from tests.paged_util import on_dev, paged_case
from tests.test_gpu_paged import F16, mnb, run_attn  # noqa: F401  (mnb: a fixture)

pytestmark = pytest.mark.gpu


def test_threads_with_other_shapes_of_one_kernel(mnb, cuda_dev):  # noqa: F811
    """Three threads, a stream and a workspace each, whose calls need different amounts of shared memory of one kernel
    (heads of 40 in 64-wide tiles): none fails, and each has the bits of the same calls made alone."""
    cases = [paged_case(50 + i, lens, 4, 2, 40, 16, F16) for i, lens in enumerate(([3], [900] * 7, [200] * 40))]
    ready, errors = threading.Barrier(len(cases)), []
    outs = [None] * len(cases)

    def calls(i):
        try:
            q, k, v, table, lens = [on_dev(t, cuda_dev) for t in cases[i]]
            ws = torch.zeros(mnb.mnb_paged_attention_workspace_bytes(q.shape[0], 4, 2, 40), dtype=torch.uint8,
                             device=cuda_dev)
            res = [torch.empty_like(q) for _ in range(60)]
            s = torch.cuda.Stream()
            torch.cuda.synchronize()
            ready.wait(30)
            for o in res:
                mnb.mnb_paged_attention(q, k, v, table, lens, 0.1, o, ws, stream=s)
            s.synchronize()
            outs[i] = [o.cpu() for o in res]
        except Exception as e:  # noqa: BLE001  (told by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors, errors
    for case, got in zip(cases, outs):
        want, _ = run_attn(mnb, cuda_dev, case, 0.1)
        assert all(torch.equal(o, want) for o in got)
