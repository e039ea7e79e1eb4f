"""The serving-step operators called in the ways that their header allows beside the plain ones:
from several host threads at once, at the sizes where a launch's resources change, on inputs that
only the kernels can refuse.  What each operator computes is tested in test_gpu_serving.py."""
import ctypes as C
import os
import subprocess
import sys
import textwrap
import threading

import numpy as np
import pytest

from oracle import serving

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def uw():
    import torch
    assert torch.cuda.is_available()
    from tests.conftest import build_library
    build_library()
    import decode_gemm_b200
    return decode_gemm_b200


def _at_once(*calls, times):
    """Run each call (a library function's status) `times` times, every one in a host thread of its own;
    the statuses that came back."""
    seen, start = set(), threading.Barrier(len(calls))

    def loop(call):
        start.wait(60)
        seen.update({call() for _ in range(times)})
    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return seen


def test_sample_from_several_host_threads(uw):
    """Vocabularies whose launches need different amounts of shared memory, on a stream each."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1)
    cases = []
    for vocab in (100000, 900, 120000, 1100):
        x = torch.randn((75, vocab), generator=gen, device="cuda").to(torch.bfloat16)
        u, t = torch.rand(75, generator=gen, device="cuda"), torch.zeros(75, device="cuda")
        ids, stream = torch.zeros(75, dtype=torch.int64, device="cuda"), torch.cuda.Stream()
        a = uw.uw_sample_args(x.data_ptr(), u.data_ptr(), t.data_ptr(), None, None, None, ids.data_ptr(), None, 75, vocab, vocab, 1)
        cases.append((a, stream, ids, x, u, t))
    torch.cuda.synchronize()
    seen = _at_once(*(lambda a=a, s=s: uw.lib.uw_sample(C.byref(a), s.cuda_stream) for a, s, *_ in cases), times=5000)
    torch.cuda.synchronize()
    assert seen == {uw.UW_OK}
    for _, _, ids, x, *_ in cases:
        at = torch.arange(x.shape[1], device="cuda")
        assert torch.equal(ids, torch.where(x == x.amax(1, keepdim=True), at, x.shape[1]).amin(1))
