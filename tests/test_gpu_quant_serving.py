"""The operators of a cache held in 4 bits together, as they are used: a coded context is
decoded, held in 4 bits, branched, extended, attended to, thinned out, packed, read back and
coded again, and every step agrees with the oracle's."""
import numpy as np
import pytest

import oracle
import synth
from oracle import paged_cache as pc
from oracle import quant_cache as qc
from tests import gpu_util as gu
from tests.test_gpu_attention import compare, queries, starts_of
from tests.test_gpu_quant import QuantPair, empty
from tests.test_gpu_quant_attention import build, check, gpu_attention
from tests.test_gpu_quant_attention import oracle as attended

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
    x = QuantPair(empty(L, (T + 400) // P + 40, P, C, 64, 6, (T + 300) // P + 2), C, 64)
    # the context, decoded and held in 4 bits
    cg.cg_decode(tab, [gu.gpu_encode(tab, kd, vd, ch, 0)[0] for ch in range(w.n_chunks)], kd, vd)
    dk, dv = np.zeros_like(k), np.zeros_like(v)
    for ch in range(w.n_chunks):
        oracle.decode_blob(ot, oracle.encode_chunk(ot, k, v, ch, 0), dk, dv)
    slots, want = x.reserve([2], [0, T], T)
    cg.cg_quant_write_async(x.cache, 0, slots, kd, vd)
    x.check(qc.write(x.o, C, 64, 0, want, dk, dv)[0], "context")

    def new(rows, counts):
        starts = starts_of(counts)
        at, host = x.reserve(rows, starts, int(starts[-1]))
        fresh = [rng.standard_normal((L, int(starts[-1]), C)).astype(np.float16) for _ in range(2)]
        x.write_numbers(0, at, host, *fresh, held="same")

    x.fork([2, 2, 2], [0, 4, 5])
    rows = [2, 0, 4, 5]
    for counts in ([1, 1, 1, 1], [3, 40, 1, 17], [1, 1, 1, 1]):
        new(rows, counts)
        q = queries(rng, sum(counts), 4, 64)
        for layer in (0, L - 1):
            check(x, layer, q, 0.125, rows, starts_of(counts), [0, 4], [T])
    # two answers end; the others are the same after the pool is packed
    before = gpu_attention(x, 1, q, 0.125, rows, [0, 1, 2, 3, 4], hints=(1, 0, 0))
    x.free([2, 4])
    x.compact()
    after = gpu_attention(x, 1, q, 0.125, [0, 0, 0, 5], [0, 1, 2, 3, 4], hints=(1, 0, 0))
    for i in (1, 3):
        assert gu.same_bits(after[1][i], before[1][i])
    new([0, 5], [2, 5])
    q = queries(rng, 7, 4, 64)
    check(x, 0, q, 0.125, [0, 5], [0, 2, 7], [0, 2], [T])
    # the context as it is held, coded again
    slots, at = x.slots([5], None, [0, T], T)
    ko, vo = (gu.torch().zeros((L, T, C), dtype=gu.torch().float16, device="cuda") for _ in range(2))
    cg.cg_quant_read_async(x.cache, 0, slots, ko, vo)
    hk, hv = np.zeros_like(k), np.zeros_like(v)
    x.check(qc.read(x.o, C, 64, 0, at, hk, hv), "read back")
    again, rebuilt = gu.gpu_tables(w, ko, vo), oracle.build_tables(oracle.params_for(w), hk, hv)
    for ch in range(w.n_chunks):
        blob = gu.gpu_encode(again, ko, vo, ch, 0)[0]
        assert blob.cpu().numpy().tobytes() == oracle.encode_chunk(rebuilt, hk, hv, ch, 0)
    x.free([0, 5])
    x.compact()
    assert (x.o.refs == 0).all() and (x.o.lens == 0).all()


def test_graphs_that_share_a_workspace():
    """A step over shared prefixes, one that cuts up the sequences' tokens and one without a
    join, each in a graph of its own over one workspace, replayed in turn."""
    rng = np.random.default_rng(21)
    C, H, d = 256, 8, 64
    tails = [[300, 1, 700, 64], [90, 2, 33]]
    c, rows = build(rng, 1, C, d, 16, [400, 130], tails)
    x = QuantPair(c, C, d)
    t, cg = x.t, x.cg
    n = len(rows)
    calls = []
    for groups, hints in (([0, 4, 7], (1, 1 << 20, 1 << 21)), (None, (1, 0, 1 << 21)), (None, (1, 0, 0)),
                          (None, (1, 0, 20000))):
        calls.append((groups, hints, cg.cg_quant_attention_workspace(x.cache, n, H, n, 2 if groups else 0, *hints)))
    ws = t.empty(max(need for _, _, need in calls), dtype=t.uint8, device="cuda")
    r, qs, gs, pl = x.i32(rows), x.i32(np.arange(n + 1)), x.i32([0, 4, 7]), x.i32([400, 130])
    qd, out = (t.zeros((n, H, d), dtype=t.float16, device="cuda") for _ in range(2))
    lse = t.zeros((n, H), dtype=t.float32, device="cuda")
    graphs = []
    for groups, hints, _ in calls:
        graphs.append(t.cuda.CUDAGraph())
        with t.cuda.graph(graphs[-1]):
            cg.cg_quant_attention_async(x.cache, 0, qd, out, 0.125, r, qs, gs if groups else None,
                                        pl if groups else None, *hints, ws, lse=lse)
    for step in range(3):
        q = queries(rng, n, H, d)
        qd.copy_(gu.to_dev(q))
        for (groups, _, _), graph in zip(calls, graphs):
            out.fill_(99.0), lse.fill_(99.0)
            graph.replay()
            t.cuda.synchronize()
            got = (int(x.status.item()), out.cpu().numpy(), lse.cpu().numpy())
            compare(got, attended(x, 0, q, 0.125, rows, np.arange(n + 1), groups, [400, 130] if groups else None), q)


@pytest.mark.parametrize("hints", [(1, 0, 0), (1, 0, 1 << 21), (1, 300, 1 << 21)])
def test_more_sequences_than_are_added_up(hints):
    """4,100 sequences of few rows of the cache: more than are cut into parts."""
    rng = np.random.default_rng(22)
    C, H, d, n = 64, 2, 64, 4100
    rows = [7, 4199, 0, 2000]
    c = empty(1, 60, 16, C, d, 4200, 20)
    for row, tokens in zip(rows[:1] + rows, (130, 1, 2, 90, 33)):
        slots = pc.reserve(c, [row], [0, tokens], tokens)[1]
        qc.write(c, C, d, 0, slots, *(rng.standard_normal((1, tokens, C)).astype(np.float16) for _ in range(2)))
        if tokens == 130:
            assert pc.fork(c, rows[:1] * 3, rows[1:]) == 0
    x = QuantPair(c, C, d)
    pick = rng.integers(0, 4, n)
    pick[:4] = range(4)
    four = queries(rng, 4, H, d)
    groups = ([0, n], [130]) if hints[1] else ()
    got = gpu_attention(x, 0, four[pick], 0.125, np.asarray(rows)[pick], np.arange(n + 1), *groups, hints=hints)
    st, recs = attended(x, 0, four, 0.125, rows, np.arange(5))
    compare(got, (st, {j: recs[i] for j, i in enumerate(pick)}), four[pick])
