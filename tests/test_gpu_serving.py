"""The paged-cache operators together, as they are used: a coded context is decoded
into a reserved row, branched, extended, attended to, thinned out and packed, and
every attention agrees with the oracle on the oracle's own decode of the blobs."""
import numpy as np
import pytest

import oracle
import synth
from oracle import paged_cache as pc
from tests import gpu_util as gu
from tests.test_gpu_attention import check, compare, queries, starts_of
from tests.test_gpu_pages import Pair

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P", [8, 64])
def test_context_to_answers(P):
    import kv_cache_compression_anchor_amd as cg
    rng = np.random.default_rng(P)
    w = gu.workload(tokens=1000, chunk_tokens=384, channels=128)
    k, v = synth.gen_kv(w)
    kd, vd = gu.to_dev(k), gu.to_dev(v)
    tab = gu.gpu_tables(w, kd, vd)
    ot = oracle.build_tables(oracle.params_for(w), k, v)
    L, T, C = k.shape
    R = 6
    x = Pair(pc.empty(L, (T + 400) // P + 40, P, C, R, (T + 300) // P + 2))
    # the context's row, and its blobs decoded into the row's pages
    x.reserve([2], [0, T], T)
    dblobs = [gu.gpu_encode(tab, kd, vd, ch, 0)[0] for ch in range(w.n_chunks)]
    infos = [cg.cg_chunk_info_parse(b[:64].cpu()) for b in dblobs]
    cg.cg_decode_paged_async(tab, dblobs, infos, x.k, x.v, P, x.tables[2, :-(-T // P)], x.status)
    for ch in range(w.n_chunks):
        oracle.decode_blob_paged(ot, oracle.encode_chunk(ot, k, v, ch, 0), x.o.k, x.o.v, P, x.o.tables[2])
    x.check(0, "decode")
    x.fork([2, 2, 2], [0, 4, 5])
    rows = [2, 0, 4, 5]
    for counts in ([1, 1, 1, 1], [3, 40, 1, 17], [1, 1, 1, 1]):
        x.new(rng, rows, counts)
        q = queries(rng, sum(counts), 4, 64)
        for layer in (0, L - 1):
            check(x, layer, q, 0.125, rows, starts_of(counts), [0, 4], [T])
    before = check(x, 1, q, 0.125, rows, [0, 1, 2, 3, 4], [0, 4], [T])
    # two answers end; the others are the same after the pool is packed
    x.free([2, 4])
    x.compact()
    after = check(x, 1, q[[1, 3]], 0.125, [0, 5], [0, 1, 2], [0, 2], [T])
    for i, j in enumerate((1, 3)):
        assert np.array_equal(after[1][i], before[1][j]) or np.allclose(
            after[1][i].astype(np.float64), before[1][j].astype(np.float64), rtol=2e-2, atol=2e-2)
    x.fork([0], [1])
    x.new(rng, [1, 0, 5], [5, 1, 2])
    q = queries(rng, 8, 4, 64)
    check(x, 0, q, 0.125, [1, 0, 5], [0, 5, 6, 8], [0, 3], [T])
    x.free([0, 1, 5])
    x.compact()
    assert (x.o.refs == 0).all() and (x.o.lens == 0).all()
