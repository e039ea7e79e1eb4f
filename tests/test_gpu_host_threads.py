"""Handles of different sizes used from several host threads at once, a handle by one thread each (as the header
allows): the decoders and the matrix-vector kernel, whose launches need shared memory by size."""
import ctypes as C

import numpy as np
import pytest

import oracle
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


@pytest.mark.parametrize("pipeline", ["palette_direct", "full"])
def test_matrix_vector_products_from_several_host_threads(uw, handles, pipeline):
    import torch
    from tests.test_gpu_serving_calls import _at_once
    pipe = uw.PIPELINES[pipeline]
    calls, cases = [], []
    for i, (h, w, s) in enumerate(handles):
        x = synthdata.activations(1, w.shape[1], seed=950 + i)
        X, Y = torch.from_numpy(x.view(np.int16)).cuda(), torch.zeros((1, w.shape[0]), dtype=torch.float32, device="cuda")
        cfg = uw.gemm_config(pipe, gemv=1)
        ws = torch.empty(max(256, uw.uw_workspace_bytes(h, pipe, 1)), dtype=torch.uint8, device="cuda")
        uw.uw_set_workspace(h, ws)
        uw.uw_gemm_ex(h, X, Y, 1, cfg, True)
        cases.append((x, w, Y, X, ws))
        calls.append(lambda h=h, X=X, Y=Y, cfg=cfg: uw.lib.uw_gemm_ex(h.ptr, X.data_ptr(), Y.data_ptr(), 1, C.byref(cfg), 1))
    torch.cuda.synchronize()
    for *_, Y, _, _ in cases:
        Y.zero_()
    torch.cuda.synchronize()
    seen = _at_once(*calls, times=2000)
    torch.cuda.synchronize()
    assert seen == {uw.UW_OK}
    for x, w, Y, *_ in cases:
        assert oracle.within_tolerance(Y.cpu().numpy().astype(np.float64), oracle.gemm_fp64(x, w), oracle.abs_product_sum(x, w))[0]
