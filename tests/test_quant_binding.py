"""Which caches the Python calls take: the struct of a cache held in 4 bits does not say so, and
where the units of a row happen to be whole heads a call on fp16 numbers would run over codes."""
import pytest

import kv_cache_compression_anchor_amd as cg


def bare(kind, **kw):
    """A cache object without tensors: what it is has to be checked before anything is read."""
    c = kind.__new__(kind)
    c.__dict__.update(kw)
    return c


def test_calls_on_numbers_refuse_a_cache_in_4_bits():
    assert cg.cg_quant_row(32 * 64, 64) == 576  # nine "heads" of 64 units
    c = bare(cg.QuantCache, form=cg.cg_quant_form(32 * 64, 64, 4, 0))
    for call in (lambda: cg.cg_pages_write_async(c, 0, None, None, None),
                 lambda: cg.cg_attention_workspace(c, 1, 9, 64, 1, 0, 1, 0, 1),
                 lambda: cg.cg_attention_prefix_async(c, 0, None, None, 1.0, None, None, None, None, 1, 0, 1, None)):
        with pytest.raises(ValueError, match="not one held in 4 bits"):
            call()


def test_calls_in_4_bits_refuse_a_cache_of_numbers():
    c = bare(cg.PagedCache)
    for call in (lambda: cg.cg_quant_write_async(c, 0, None, None, None),
                 lambda: cg.cg_quant_read_async(c, 0, None, None, None),
                 lambda: cg.cg_quant_attention_workspace(c, 1, 4, 1, 0, 1, 0, 1),
                 lambda: cg.cg_quant_attention_async(c, 0, None, None, 1.0, None, None, None, None, 1, 0, 1, None)):
        with pytest.raises(ValueError, match="takes a QuantCache"):
            call()


@pytest.mark.gpu
def test_refusals_on_the_device_leave_the_outputs():
    """32 heads of 64 channels: q of nine heads of 64 fits the units."""
    from tests import gpu_util as gu
    t = gu.torch()
    row = 2 * cg.cg_quant_row(2048, 64)
    pools = t.zeros((2, 1, 4, 16, row), dtype=t.uint8, device="cuda")
    i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    c = cg.QuantCache(pools[0], pools[1], i32([[0, 1]]), i32([20]), i32([1, 1, 0, 0]), i32([0]), 2048, 64)
    q, out = t.ones((1, 9, 64), dtype=t.float16, device="cuda"), t.full((1, 9, 64), 5.0, dtype=t.float16, device="cuda")
    ws = t.empty(1 << 20, dtype=t.uint8, device="cuda")
    with pytest.raises(ValueError):
        cg.cg_attention_prefix_async(c, 0, q, out, 0.125, None, i32([0, 1]), None, None, 1, 0, 20, ws)
    new = t.ones((1, 1, 576), dtype=t.float16, device="cuda")
    with pytest.raises(ValueError):
        cg.cg_pages_write_async(c, 0, t.zeros(1, dtype=t.int64, device="cuda"), new, new)
    t.cuda.synchronize()
    assert (out == 5.0).all() and (pools == 0).all()
