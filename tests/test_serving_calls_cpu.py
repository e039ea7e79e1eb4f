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


def _cache_that_is_passed_on(uw, monkeypatch, call, fn, args, **over):
    kept = []
    monkeypatch.setattr(uw, fn, lambda packed, stream: kept.append(packed) or 0)
    call(uw, **over)
    return getattr(uw, args).from_buffer_copy(kept[0].ljust(128 * 4, b"\0")).cache


@pytest.mark.parametrize("fn,args", [("_rope_fn", "uw_qk_norm_rope_args"), ("_attention_fn", "uw_paged_attention_args")])
@pytest.mark.parametrize("axis", [0, 1, 2])
def test_caches_with_an_axis_of_one_entry(uw, monkeypatch, fn, args, axis):
    """The stride of such an axis is never stepped along: whatever it is, and whether or not keys and values
    have the same one, the cache is the same."""
    call, shape = (_rope if fn == "_rope_fn" else _attend), [3, 8, 2, 64]
    shape[axis] = 1
    over = dict(k=_zeros(2, shape[2], 64, t="bfloat16"), v=_zeros(2, shape[2], 64, t="bfloat16")) if call is _rope else {}
    plain = _zeros(*shape, t="bfloat16")
    for odd in (0, 1, 3, 10**12):
        strides = list(plain.stride())
        strides[axis] = odd
        other = plain.as_strided(shape, strides)
        for k, v in ((other, plain), (plain, other), (other, other)):
            c = _cache_that_is_passed_on(uw, monkeypatch, call, fn, args, k_cache=k, v_cache=v, **over)
            got = [c.page_stride, c.slot_stride, c.head_stride]
            assert [g for i, g in enumerate(got) if i != axis] == [g for i, g in enumerate(plain.stride()[:3]) if i != axis]
            assert got[axis] > 0 and got[axis] % 8 == 0 and got[axis] < 2**39
            assert [c.n_pages, c.page_size, c.n_kv_heads, c.head_dim] == shape
    # axes that are stepped along have to agree
    wide = _zeros(*[n + (n > 1) for n in shape[:3]], 64, t="bfloat16")[:shape[0], :shape[1], :shape[2]]
    with pytest.raises(uw.UwError) as e:
        call(uw, k_cache=plain, v_cache=wide, **over)
    assert e.value.status == uw.UW_ERR_ARG
