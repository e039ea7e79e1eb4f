"""Handles of different sizes used from several host threads at once, a handle by one thread each (as the header
allows): the decoders, whose launches need shared memory by size."""
import numpy as np
import pytest

import synthdata

pytestmark = pytest.mark.gpu

SHAPES = ((2048, 1024), (64, 64), (4096, 512), (192, 128))


@pytest.fixture(scope="module")
def uw():
    import torch
    assert torch.cuda.is_available()
    from tests.conftest import build_library
    build_library()
    import decode_gemm_b200
    return decode_gemm_b200


@pytest.fixture(scope="module")
def handles(uw):
    """(handle, its weights), each on a stream of its own."""
    import torch
    made = []
    for i, (n, k) in enumerate(SHAPES):
        w = synthdata.normal(n, k, 0.02, seed=900 + i)
        h, s = uw.uw_encode(w), torch.cuda.Stream()
        uw.uw_set_stream(h, s)
        made.append((h, w, s))
    yield made
    torch.cuda.synchronize()
    for h, *_ in made:
        h.free()


def test_decoders_from_several_host_threads(uw, handles):
    import torch
    from tests.test_gpu_serving_calls import _at_once
    outs = [torch.zeros(w.size, dtype=torch.int16, device="cuda") for _, w, _ in handles]
    torch.cuda.synchronize()
    seen = _at_once(*(lambda h=h, o=o: uw.lib.uw_decode_full(h.ptr, o.data_ptr()) for (h, *_), o in zip(handles, outs)),
                    times=4000)
    torch.cuda.synchronize()
    assert seen == {uw.UW_OK}
    for (_, w, _), o in zip(handles, outs):
        assert np.array_equal(o.cpu().numpy().view(np.uint16).reshape(w.shape), w)
