"""The weights of a sequence of few tokens with up to 32 rows of a kv head, which one workgroup has alone:
the second product takes what their rounding to binary16 lost as well.

Bound of one output, with the names of test_gpu_attention.py.  A weight in two parts of binary16 is off by
u of what u of it left, u^2, and absolutely by the same 2^-25 of the largest weight; the rest as there:
    |out - o| <= u |o| + (u^2 + 4 D + 2 e (n + 64)) A + n 2^-25 max|v| / l + 2^-25
The scores here are small, so that D leaves room for a weight rounded once to pass the bound."""
import numpy as np
import pytest

from oracle import paged_cache as pc
from oracle import quant_cache as qc
from tests import quant_plan as qp
from tests.test_gpu_attention import E, U, compare, queries, starts_of
from tests.test_gpu_quant import QuantPair
from tests.test_gpu_quant_attention import build, gpu_attention, oracle

LENS = [2, 3, 4, 5, 7, 11, 20, 33, 64]


def bound(r, d):
    n, D = r["tokens"], E * (d + 16) * (r["size"] + 1)
    return (U * np.abs(r["out"]) + (U * U + 4 * D + 2 * E * (n + 64)) * r["mean_abs"]
            + n * 2.0 ** -25 * r["vmax"] / r["l"] + 2.0 ** -25)


def case(kv, G, d, most):
    rng = np.random.default_rng(kv * 1000 + G * 10 + d + most)
    counts = [min(most, n) for n in LENS]
    c, rows = build(rng, 1, kv * d, d, 16, LENS, [[0]] * len(LENS))
    return c, rows, queries(rng, sum(counts), kv * G, d), starts_of(counts), 0.2 / d


CASES = [(2, 1, 64, 1), (1, 4, 128, 1), (3, 7, 80, 2), (2, 5, 40, 3), (1, 4, 64, 8), (1, 2, 256, 3), (2, 8, 128, 4)]


@pytest.mark.parametrize("kv,G,d,most", CASES)
def test_the_bound_tells_two_parts_from_one(kv, G, d, most):
    """The formula in binary64 with the weights' rounding put in, on the CPU."""
    c, rows, q, qs, scale = case(kv, G, d, most)
    k, v = (x.astype(np.float64) for x in (qc.numbers(y, kv * d, d) for y in qc.raw(c)))
    _, recs = pc.attention(qc.held(c, kv * d, d), 0, q, scale, rows, qs)
    worst = [0.0, 0.0]
    for s, row in enumerate(rows):
        for j in range(qs[s], qs[s + 1]):
            t = np.arange(recs[j][0]["tokens"])
            K, V = (x[0, c.tables[row, t // 16], t % 16].reshape(len(t), kv, d) for x in (k, v))
            for h, r in enumerate(recs[j]):
                x = scale * (K[:, h // G] @ q[j, h].astype(np.float64)) / np.log(2)
                w = np.exp2(x - x.max() + 6)  # the reference exponent is 6 below the largest
                one = w.astype(np.float16).astype(np.float64)
                two = one + (w - one).astype(np.float16).astype(np.float64)
                for i, p in enumerate((one, two)):
                    out = (p @ V[:, h // G] / w.sum()).astype(np.float16).astype(np.float64)
                    worst[i] = max(worst[i], float((np.abs(out - r["out"]) / bound(r, d)).max()))
    assert worst[0] > 1 >= worst[1], worst


@pytest.mark.gpu
@pytest.mark.parametrize("kv,G,d,most", CASES)
def test_few_tokens_alone_take_the_weights_in_two_parts(kv, G, d, most):
    c, rows, q, qs, scale = case(kv, G, d, most)
    x = QuantPair(c, kv * d, d)
    p = qp.plans([qp.Call(kv * d, d, 16, c.tables.shape[1], kv * G, len(rows), q.shape[0], 0, most, 0, 64)])[0]
    assert p.cut == qp.ALONE and p.rest < qp.MANY16, p
    got = gpu_attention(x, 0, q, scale, rows, qs, hints=(most, 0, 64))
    want = oracle(x, 0, q, scale, rows, qs)
    compare(got, want, q)
    for j, recs in want[1].items():
        for h, r in enumerate(recs):
            off = np.abs(got[1][j, h].astype(np.float64) - r["out"])
            assert (off <= bound(r, d)).all(), (j, h, r["tokens"], float((off / bound(r, d)).max()))
