"""The attention over caches held in 4 bits: calls chosen for the kernel that they take, which the
library's own plan, compiled for the host, confirms.  The bound is test_gpu_attention.py's."""
import numpy as np
import pytest

from oracle import paged_cache as pc
from oracle import quant_cache as qc
from tests import quant_plan as qp
from tests.test_gpu_attention import compare, queries, starts_of
from tests.test_gpu_quant import QuantPair
from tests.test_gpu_quant_attention import build, gpu_attention, oracle, spoil

pytestmark = pytest.mark.gpu


def plan(x, q, q_starts, groups, hints):
    return qp.plans([qp.Call(x.C, x.d, x.o.P, x.o.tables.shape[1], q.shape[1], len(q_starts) - 1, q.shape[0], groups, *hints)])[0]


# Prefixes said to be long, so that they are shared; own tokens in splits, or in parts.
HINTS = {qp.SPLITS: lambda most, kv: (most, 20000, 23000 if kv == 1 else 22000),
         qp.PARTS: lambda most, kv: (most, 1 << 20, 1 << 21)}


# A sequence's rows are 17 to 32, a group's more than 128: prefixes as many rows beside a rest of few.
@pytest.mark.parametrize("kv,G,d,P,most", [(1, 4, 64, 16, 5), (2, 20, 40, 8, 1), (1, 4, 128, 16, 5), (3, 7, 80, 4, 4),
                                           (2, 9, 72, 32, 3)])
@pytest.mark.parametrize("cut", [qp.SPLITS, qp.PARTS])
def test_prefixes_of_many_rows_beside_32_of_a_sequence(kv, G, d, P, most, cut):
    rng = np.random.default_rng(kv + G + d)
    seqs = 44
    tails = [[int(n) for n in rng.integers(most, 400, seqs)]]
    c, rows = build(rng, 1, kv * d, d, P, [777], tails)
    c.tables[rows[0], 300 // P] = -1   # a page of the prefix
    c.tables[rows[3], 777 // P] = c.N  # and one of a sequence's own
    counts = rng.integers(1, most + 1, seqs)
    counts[2], counts[5] = 0, most
    q = queries(rng, int(counts.sum()), kv * G, d)
    x = QuantPair(c, kv * d, d)
    qs = starts_of(counts)
    hints = HINTS[cut](most, kv)
    p = plan(x, q, qs, 1, hints)
    assert (p.pre, p.rest, p.cut) == (qp.MANY32, qp.FEW32, cut) and p.pieces > 1, p
    want = oracle(x, 0, q, d ** -0.5, rows, qs, [0, seqs], [777])
    assert want[0] == pc.BAD_PAGE
    compare(gpu_attention(x, 0, q, d ** -0.5, rows, qs, [0, seqs], [777], hints=hints), want, q)


@pytest.mark.parametrize("kv,G,d", [(1, 4, 64), (2, 4, 128), (1, 4, 96)])
@pytest.mark.parametrize("cut", [qp.SPLITS, qp.PARTS])
def test_values_that_are_no_numbers_beside_a_prefix_of_many_rows(kv, G, d, cut):
    """A NaN group of a value in the shared prefix, and one that the later queries of a sequence see."""
    rng = np.random.default_rng(d)
    seqs, most = 40, 5
    c, rows = build(rng, 1, kv * d, d, 16, [300], [[int(n) for n in rng.integers(most, 90, seqs)]])
    sound = c.copy()
    counts = np.full(seqs, most)
    qs = starts_of(counts)
    q = queries(rng, seqs * most, kv * G, d)
    spoil((kv * d, d), c, rows[0], 70, 3)  # the first group of head 0: everyone sees it
    spoil((kv * d, d), c, rows[7], int(c.lens[rows[7]]) - most + 2, kv * d - 1)  # seen by queries 2 .. of sequence 7
    first, last = slice(0, 32), slice((d - 1) // 32 * 32, d)
    x = QuantPair(c, kv * d, d)
    hints = HINTS[cut](most, kv)
    p = plan(x, q, qs, 1, hints)
    assert (p.pre, p.rest, p.cut) == (qp.MANY32, qp.FEW32, cut) and p.pieces > 1, p
    _, recs = pc.attention(qc.held(sound, kv * d, d), 0, q, 0.125, rows, qs, [0, seqs], [300])
    st, out, lse = gpu_attention(x, 0, q, 0.125, rows, qs, [0, seqs], [300], hints=hints)
    for j in range(seqs * most):
        for h in range(kv * G):
            bad = np.zeros(d, bool)
            if h // G == 0:
                bad[first] = True
            if h // G == kv - 1 and 7 * most + 2 <= j < 8 * most:
                bad[last] = True
            assert not np.isfinite(out[j, h][bad]).any()
            out[j, h][bad] = recs[j][h]["out"][bad]
    compare((st, out, lse), (0, recs), q)
