"""Arguments of the serving-step calls that the Python binding itself refuses or has to accept (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def uw():
    from tests.conftest import build_library
    build_library()
    import decode_gemm_b200
    return decode_gemm_b200


def _zeros(*shape, t="float32"):
    import torch
    return torch.zeros(shape, dtype=getattr(torch, t))


def _rope(uw, **over):
    z, bf = _zeros, "bfloat16"
    uw.uw_qk_norm_rope(**dict(q=z(2, 4, 64, t=bf), k=z(2, 2, 64, t=bf), v=z(2, 2, 64, t=bf), positions=z(2, t="int32"),
                              inv_freq=z(32), slots=z(2, t="int64"), k_cache=z(3, 8, 2, 64, t=bf),
                              v_cache=z(3, 8, 2, 64, t=bf), q_out=z(2, 4, 64, t=bf)) | over)


def _attend(uw, **over):
    z, bf = _zeros, "bfloat16"
    uw.uw_paged_attention(**dict(q=z(2, 4, 64, t=bf), k_cache=z(3, 8, 2, 64, t=bf), v_cache=z(3, 8, 2, 64, t=bf),
                                 table=z(1, 3, t="int32"), cu_q=z(2, t="int32"), kv_len=z(1, t="int32"),
                                 out=z(2, 4, 64, t=bf), ws=z(1024, t="uint8")) | over)


def _plan(uw, **over):
    z, i = _zeros, "int32"
    uw.uw_paged_plan(**dict(ctx_len=z(2, t=i), new_len=z(2, t=i), page_size=16, free_pages=z(4, t=i), table=z(2, 3, t=i),
                            cu_q=z(3, t=i), kv_len=z(2, t=i), positions=z(5, t=i), slots=z(5, t="int64"),
                            head_out=z(1, t=i)) | over)


def test_numbers_that_their_fields_cannot_hold(uw):
    """Refused as every other bad argument is, with the call's name."""
    for call, name, over in [(_plan, "uw_paged_plan", dict(page_size=2**40)), (_plan, "uw_paged_plan", dict(page_size=16.0)),
                             (_attend, "uw_paged_attention", dict(window=2**31)), (_attend, "uw_paged_attention", dict(window=None)),
                             (_attend, "uw_paged_attention", dict(scale="1")), (_rope, "uw_qk_norm_rope", dict(eps=None))]:
        with pytest.raises(uw.UwError, match=name) as e:
            call(uw, **over)
        assert e.value.status == uw.UW_ERR_ARG, over
