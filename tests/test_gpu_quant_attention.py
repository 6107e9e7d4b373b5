"""Attention over a cache held in 4 bits against the oracle's binary64 one over the numbers
that the cache stands for.  They are binary16 numbers and meet the same roundings as in a
cache of binary16 (scores and sums in binary32, weights rounded to binary16, one rounding
of the result), so that the bound derived in test_gpu_attention.py holds here too."""
import numpy as np
import pytest

from oracle import paged_cache as pc
from oracle import quant_cache as qc
from tests import gpu_util as gu
from tests.test_gpu_attention import compare, group_starts_of, queries, starts_of
from tests.test_gpu_quant import QuantPair, empty

pytestmark = pytest.mark.gpu


def build(rng, L, C, d, P, prefixes, tails, spare=3, spread=1.0):
    """A cache in which group g's sequences continue a prefix of prefixes[g] tokens by
    tails[g][i] tokens; what no token holds is anything, NaN scales among it."""
    seqs = [(g, n) for g, t in enumerate(tails) for n in t]
    R = len(seqs)
    longest = max(prefixes[g] + n for g, n in seqs)
    pages = sum(-(-(prefixes[g] + n) // P) + 1 for g, n in seqs) + spare
    c = empty(L, pages, P, C, d, R + 2, -(-longest // P) + 2, seed=R)
    order = rng.permutation(R + 2)[:R]
    first, rows = {}, []

    def add(row, n):
        st, slots = pc.reserve(c, [row], [0, n], n)
        assert st == 0
        k, v = ((spread * rng.standard_normal((L, n, C))).astype(np.float16) for _ in range(2))
        qc.write(c, C, d, 0, slots, k, v)

    for (g, _), row in zip(seqs, order):
        if g not in first:
            first[g] = row
            add(row, prefixes[g])
        else:
            assert pc.fork(c, [first[g]], [row]) == 0
        rows.append(row)
    for (g, n), row in zip(seqs, rows):
        if n:
            add(row, n)
    return c, rows


def gpu_attention(x, layer, q, scale, rows, q_starts, group_starts=None, prefix_lens=None, hints=None, lse=True,
                  out=None, stream=None):
    cg, t = x.cg, x.t
    n_q, H, d = q.shape
    hints = hints or (max(1, int(np.max(np.diff(q_starts), initial=0))),
                      int(np.max(prefix_lens, initial=0)) if prefix_lens is not None else 0,
                      int(np.max(x.o.lens)))
    hints = tuple(max(0, h) for h in hints)
    groups = 0 if group_starts is None else len(group_starts) - 1
    ws = t.full((cg.cg_quant_attention_workspace(x.cache, n_q, H, len(q_starts) - 1, groups, *hints),), 0xFF,
                dtype=t.uint8, device="cuda")
    qd = gu.to_dev(q)
    if out is None:
        out = t.full((n_q, H, d), 123.0, dtype=t.float16, device="cuda")
    ld = t.full((n_q, H), 321.0, dtype=t.float32, device="cuda") if lse else None
    opt = lambda v: None if v is None else x.i32(v)  # noqa: E731
    cg.cg_quant_attention_async(x.cache, layer, qd, out, scale, opt(rows), x.i32(q_starts), opt(group_starts),
                                opt(prefix_lens), *hints, ws, lse=ld, stream=stream)
    t.cuda.synchronize()
    st = int(x.status.item())
    x.status.zero_()
    return st, out.cpu().numpy(), None if ld is None else ld.cpu().numpy()


def hints_of(q_starts):
    """The lengths'; a prefix shared, tokens in parts and joined; joined; one kernel; splits."""
    most = max(1, int(np.max(np.diff(q_starts), initial=0)))
    return (None, (most, 1 << 20, 1 << 21), (most, 0, 1 << 21), (most, 0, 0), (most, 1 << 20, (1 << 20) + 200),
            (most, 0, 4000))


def oracle(x, layer, q, scale, rows, q_starts, *groups):
    return pc.attention(qc.held(x.o, x.C, x.d), layer, q, scale, rows, q_starts, *groups)


def check(x, layer, q, scale, rows, q_starts, *groups):
    want = oracle(x, layer, q, scale, rows, q_starts, *groups)
    for hints in hints_of(q_starts):
        got = gpu_attention(x, layer, q, scale, rows, q_starts, *groups, hints=hints)
        compare(got, want, q)
    return got


# heads: kv heads, query heads per kv head, head dimension
@pytest.mark.parametrize("kv,G,d", [(2, 1, 64), (1, 4, 128), (3, 7, 80), (2, 8, 128), (1, 2, 256), (1, 1, 8),
                                    (2, 5, 40), (1, 3, 192), (4, 17, 64), (1, 70, 128), (2, 3, 32), (2, 2, 72),
                                    (1, 40, 160), (3, 2, 136), (8, 4, 128)])
@pytest.mark.parametrize("P", [1, 8, 16, 128])
def test_heads_and_pages(kv, G, d, P):
    rng = np.random.default_rng(kv * 10007 + G * 101 + d + P)
    tails = [[1, 5, 40], [2, 33]]
    c, rows = build(rng, 2, kv * d, d, P, [50, 37], tails)
    x = QuantPair(c, kv * d, d)
    q = queries(rng, 5, kv * G, d)
    check(x, 1, q, d ** -0.5, rows, np.arange(6), group_starts_of(tails), [50, 37])
    check(x, 0, q, d ** -0.5, rows, np.arange(6))


@pytest.mark.parametrize("prefix", [1, 15, 16, 31, 32, 33, 63, 65, 127, 128, 200, 257, 1000])
@pytest.mark.parametrize("tail", [[1], [1, 2, 3], [16, 17, 64, 65, 300]])
def test_lengths(prefix, tail):
    rng = np.random.default_rng(prefix * 31 + len(tail))
    c, rows = build(rng, 1, 128, 64, 16, [prefix], [tail])
    x = QuantPair(c, 128, 64)
    q = queries(rng, len(tail), 4, 64)
    check(x, 0, q, 0.125, rows, np.arange(len(tail) + 1), [0, len(tail)], [prefix])
    check(x, 0, q, 0.125, rows, np.arange(len(tail) + 1))
    check(x, 0, q, 0.125, rows, np.arange(len(tail) + 1), [0, len(tail)], [prefix - prefix // 3])


@pytest.mark.parametrize("counts", [[1, 1, 1], [4, 0, 2], [0, 0, 1], [9, 30, 17], [64, 65, 1], [130, 3, 0]])
@pytest.mark.parametrize("G,d", [(1, 128), (4, 128), (3, 64)])
def test_several_queries(counts, G, d):
    """Drafts and prompts: a sequence's queries see one token more each."""
    rng = np.random.default_rng(sum(counts) * 10 + G)
    tails = [[max(1, counts[0]) + 3, max(1, counts[1])], [max(1, counts[2]) + 70]]
    c, rows = build(rng, 1, 2 * d, d, 8, [45, 20], tails)
    x = QuantPair(c, 2 * d, d)
    q = queries(rng, sum(counts) + 3, 2 * G, d)  # three rows behind the last sequence
    check(x, 0, q, 0.09, rows, starts_of(counts), group_starts_of(tails), [45, 20])
    check(x, 0, q, 0.09, rows, starts_of(counts))


def test_wrong_hints_change_nothing():
    rng = np.random.default_rng(3)
    tails = [[5, 300, 40], [1, 2]]
    c, rows = build(rng, 1, 128, 64, 16, [700, 90], tails)
    x = QuantPair(c, 128, 64)
    counts = [5, 70, 1, 1, 2]
    q = queries(rng, sum(counts), 4, 64)
    args = (0, q, 0.125, rows, starts_of(counts), group_starts_of(tails), [700, 90])
    want = oracle(x, *args)
    for hints in ((0, 0, 0), (1, 1, 1), (1, 100000, 200000), (5000, 700, 1000), (70, 10, 1 << 30),
                  (1 << 20, 1 << 30, 1 << 30)):
        compare(gpu_attention(x, *args, hints=hints), want, q)


def test_many_sequences():
    """Groups of one, an uneven batch, more groups than a wavefront has lanes."""
    rng = np.random.default_rng(4)
    tails = [[int(rng.integers(1, 40)) for _ in range(rng.integers(1, 4))] for _ in range(80)]
    prefixes = [int(rng.integers(1, 50)) for _ in tails]
    c, rows = build(rng, 1, 64, 64, 8, prefixes, tails)
    x = QuantPair(c, 64, 64)
    n = len(rows)
    q = queries(rng, n, 2, 64)
    check(x, 0, q, 0.125, rows, np.arange(n + 1), group_starts_of(tails), prefixes)
    gs = group_starts_of(tails)  # some sequences in no group
    check(x, 0, q, 0.125, rows, np.arange(n + 1), gs[10:41], prefixes[10:40])


@pytest.mark.parametrize("seqs,kv,G,d", [(130, 4, 2, 40), (129, 6, 3, 128), (256, 4, 1, 64), (70, 8, 4, 32),
                                         (131, 4, 2, 200), (64, 8, 4, 128)])
def test_many_sequences_of_several_heads(seqs, kv, G, d):
    """A batch whose workgroups take two or four kv heads each, a page outside the pool."""
    rng = np.random.default_rng(seqs + d)
    tails = [[int(n) for n in rng.integers(2, 20, seqs // 2)], [int(n) for n in rng.integers(2, 150, seqs - seqs // 2)]]
    c, rows = build(rng, 1, kv * d, d, 8, [21, 9], tails)
    c.tables[rows[seqs // 3], 3] = -1
    counts = rng.integers(0, 3, seqs)
    x = QuantPair(c, kv * d, d)
    q = queries(rng, int(counts.sum()), kv * G, d)
    check(x, 0, q, d ** -0.5, rows, starts_of(counts), group_starts_of(tails), [21, 9])
    check(x, 0, q, d ** -0.5, rows, starts_of(counts))


@pytest.mark.parametrize("kv,G,d,P,prefix,seqs", [
    (2, 4, 128, 16, 1500, 40), (1, 8, 128, 8, 1111, 20), (1, 3, 64, 64, 2047, 25), (1, 5, 64, 8, 1300, 50),
    (2, 2, 256, 16, 1200, 40), (1, 6, 80, 16, 1055, 30), (1, 4, 128, 1, 1100, 33), (1, 5, 96, 4, 700, 30),
    (1, 4, 128, 4, 900, 12), (1, 2, 256, 128, 1900, 9), (4, 8, 64, 32, 3200, 16), (1, 33, 32, 16, 800, 5)])
def test_long_shared_prefix(kv, G, d, P, prefix, seqs):
    rng = np.random.default_rng(prefix + d)
    tails = [[int(n) for n in rng.integers(2, 60, seqs)]]
    c, rows = build(rng, 1, kv * d, d, P, [prefix], tails)
    counts = rng.integers(0, 3, seqs)
    q = queries(rng, int(counts.sum()), kv * G, d)
    check(QuantPair(c, kv * d, d), 0, q, d ** -0.5, rows, starts_of(counts), [0, seqs], [prefix])
    # a page of the prefix outside the pool
    c.tables[rows[0], (prefix // 2) // P] = -1
    check(QuantPair(c, kv * d, d), 0, q, d ** -0.5, rows, starts_of(counts), [0, seqs], [prefix])


@pytest.mark.parametrize("d,G,P", [(128, 4, 16), (64, 9, 8), (256, 2, 32), (72, 3, 16)])
def test_long_prompts(d, G, P):
    """Sequences whose queries are a prompt of hundreds of tokens, behind a context."""
    rng = np.random.default_rng(d)
    c, rows = build(rng, 1, d, d, P, [420, 64], [[300, 140], [33]])
    counts = [260, 131, 33]
    q = queries(rng, sum(counts), G, d)
    x = QuantPair(c, d, d)
    check(x, 0, q, d ** -0.5, rows, starts_of(counts), [0, 2, 3], [420, 64])
    check(x, 0, q, d ** -0.5, rows, starts_of(counts))


@pytest.mark.parametrize("seqs,lens,kv,G,d", [(3, 9000, 2, 4, 128), (1, 20000, 1, 8, 64), (2, 5000, 4, 1, 256),
                                              (2, 7000, 5, 7, 80)])
def test_long_rows(seqs, lens, kv, G, d):
    """Rows of their own of thousands of tokens, split and joined."""
    rng = np.random.default_rng(lens)
    c, rows = build(rng, 1, kv * d, d, 16, [1] * seqs, [[lens - 17 * i] for i in range(seqs)])
    q = queries(rng, seqs, kv * G, d)
    x = QuantPair(c, kv * d, d)
    check(x, 0, q, d ** -0.5, rows, np.arange(seqs + 1))


def spoil(x, c, row, t, ch, which="v"):
    """Token t of a row gets a NaN scale in the group of channel ch."""
    groups = qc.sizes(x[0], x[1])[1]
    at = qc.sizes(x[0], x[1])[2] + 2 * (ch // x[1] * groups + ch % x[1] // 32)
    raw = qc.raw(c)[which == "v"]
    raw[0, c.tables[row, t // c.P], t % c.P, at:at + 2] = 0xFF


@pytest.mark.parametrize("kv,G,d", [(1, 4, 128), (2, 2, 64), (1, 20, 128), (1, 40, 64), (2, 1, 256), (2, 3, 80)])
def test_masked_places_have_no_influence(kv, G, d):
    """NaN scales and any codes in free pages, behind the rows' ends (as build leaves them) and in
    tokens that later queries of the same sequence see but earlier ones do not."""
    rng = np.random.default_rng(9)
    counts = [5, 3, 2]
    c, rows = build(rng, 1, kv * d, d, 16, [50], [[7, 20, 33]])
    for raw in qc.raw(c):
        free = c.refs == 0
        raw[:, free] = 0xFF
    q = queries(rng, 10, kv * G, d)
    check(QuantPair(c, kv * d, d), 0, q, 0.09, rows, starts_of(counts), [0, 3], [50])
    want = c.copy()
    for r in rows:  # the last token of each sequence: only its last query sees it
        for which in "kv":
            spoil((kv * d, d), c, r, int(c.lens[r]) - 1, 5, which)
    x = QuantPair(c, kv * d, d)
    for groups in (([0, 3], [50]), (None, None)):
        for hints in hints_of(starts_of(counts)):
            st, out, lse = gpu_attention(x, 0, q, 0.09, rows, starts_of(counts), *groups, hints=hints)
            _, recs = pc.attention(qc.held(want, kv * d, d), 0, q, 0.09, rows, starts_of(counts), *groups)
            for s in range(3):
                j = starts_of(counts)[s + 1] - 1
                assert np.isnan(out[j, :G]).all() and np.isnan(lse[j, :G]).all()
                recs.pop(j)
                out[j], lse[j] = 123.0, 321.0
            compare((st, out, lse), (0, recs), q)


@pytest.mark.parametrize("kv,G,d", [(2, 1, 64), (1, 4, 128), (1, 20, 128), (2, 40, 64), (1, 3, 256), (1, 9, 256)])
def test_values_that_are_no_numbers(kv, G, d):
    """A NaN group of a value: the queries before it are not touched, those that see it get no
    finite number in its channels and the formula in the others, however little it weighs."""
    rng = np.random.default_rng(21)
    c, rows = build(rng, 1, kv * d, d, 16, [300], [[200, 90]])
    want = c.copy()
    counts = [30, 17]
    q = queries(rng, sum(counts), kv * G, d)
    t = int(c.lens[rows[0]]) - 30 + 11
    spoil((kv * d, d), c, rows[0], t, kv * d - 1)  # seen by queries 11 .. of the first sequence
    for r in rows:
        spoil((kv * d, d), c, r, 70, 3)  # in the prefix
    first, last = slice(0, 32), slice((d - 1) // 32 * 32, d)
    x = QuantPair(c, kv * d, d)
    _, recs = pc.attention(qc.held(want, kv * d, d), 0, q, 0.125, rows, starts_of(counts))
    for groups in (([0, 2], [300]), (None, None)):
        for hints in hints_of(starts_of(counts)):
            st, out, lse = gpu_attention(x, 0, q, 0.125, rows, starts_of(counts), *groups, hints=hints)
            for j in range(sum(counts)):
                for h in range(kv * G):
                    bad = np.zeros(d, bool)
                    if h // G == 0:
                        bad[first] = True
                    if h // G == kv - 1 and 11 <= j < 30:
                        bad[last] = True
                    assert not np.isfinite(out[j, h][bad]).any()
                    out[j, h][bad] = recs[j][h]["out"][bad]
            compare((st, out, lse), (0, recs), q)


@pytest.mark.parametrize("kv,G,d", [(2, 1, 64), (1, 4, 128), (1, 20, 128), (1, 40, 64), (1, 3, 256)])
@pytest.mark.parametrize("scale", [2.0 ** 126, -2.0 ** 126, 2.0 ** 127])
def test_scores_past_the_range(kv, G, d, scale):
    """A score past binary32's range is an infinity: NaN for a query with one of +infinity, zeros
    for one that sees -infinity alone; a query of zeros has finite scores."""
    rng = np.random.default_rng(kv * 100 + G + d)
    c, rows = build(rng, 1, kv * d, d, 16, [300], [[5, 40]])
    k, v = qc.raw(c)
    k[:] = qc.rows_of(np.ones((1, kv * d), np.float16), d, np.zeros((1, k.shape[3]), np.uint8))[0]
    x = QuantPair(c, kv * d, d)
    q = np.ones((6, kv * G, d), np.float16)
    q[1], q[4], q[5] = -1, -1, 0
    counts = [3, 3]
    zero = q[5:6]
    want = pc.attention(qc.held(c, kv * d, d), 0, zero, 1.0, [rows[1]], [0, 1])[1][0]
    for groups in (([0, 2], [300]), (None, None)):
        for hints in hints_of(starts_of(counts)):
            st, out, lse = gpu_attention(x, 0, q, scale, rows, starts_of(counts), *groups, hints=hints)
            up, down = ([0, 2, 3], [1, 4]) if scale > 0 else ([1, 4], [0, 2, 3])
            assert st == 0 and np.isnan(out[up]).all() and np.isnan(lse[up]).all(), (groups, hints)
            assert (out[down] == 0).all() and (lse[down] == -np.inf).all(), (groups, hints)
            compare((0, out[5:6], lse[5:6]), (0, {0: want}), zero)


def test_large_scores_and_spread():
    """Peaked weights and scores whose exponentials overflow without the maximum."""
    rng = np.random.default_rng(11)
    c, rows = build(rng, 1, 128, 64, 16, [300], [[9, 40]], spread=3.0)
    x = QuantPair(c, 128, 64)
    q = 8 * queries(rng, 2, 4, 64)
    for scale in (0.125, 4.0, -1.0, 0.0, 1e-6):
        check(x, 0, q, scale, rows, np.arange(3), [0, 2], [300])


@pytest.mark.parametrize("size", [2.0 ** -18, 2.0 ** -8, 2.0 ** 12])
def test_small_and_large_numbers(size):
    """Scales from binary16's subnormal numbers up to its largest."""
    rng = np.random.default_rng(12)
    c, rows = build(rng, 1, 256, 128, 16, [130], [[9, 40]], spread=size)
    x = QuantPair(c, 256, 128)
    q = queries(rng, 2, 4, 128)
    check(x, 0, q, 0.09 / max(size, 2.0 ** -6), rows, np.arange(3), [0, 2], [130])


def test_rows_default_and_empty_rows():
    rng = np.random.default_rng(5)
    c = empty(1, 30, 16, 64, 64, 4, 6)
    x = QuantPair(c, 64, 64)
    slots, want = x.reserve([0, 2], [0, 20, 23], 23)
    x.write_numbers(0, slots, want, *(rng.standard_normal((1, 23, 64)).astype(np.float16) for _ in range(2)))
    q = queries(rng, 8, 1, 64)
    # rows 1 and 3 are empty: their queries see nothing; row 2 has more queries than tokens
    check(x, 0, q, 0.125, None, [0, 1, 2, 7, 8])
    check(x, 0, q, 0.125, [1], [0, 8])


def test_refused_sequences():
    rng = np.random.default_rng(6)
    c, rows = build(rng, 1, 64, 64, 8, [30, 12], [[4, 1, 9], [3]])
    x = QuantPair(c, 64, 64)
    q = queries(rng, 9, 2, 64)
    qs, gs = [0, 2, 4, 7, 9], [0, 3, 4]
    st, out, _ = check(x, 0, q, 0.125, rows, qs, gs, [30, 12])  # the second's queries start before token 31
    assert st == pc.REFUSED and (out[2:4] == 0).all()
    check(x, 0, q, 0.125, rows, qs, gs, [29, 12])
    check(x, 0, q, 0.125, rows, qs, gs, [33, 16])  # longer than the rows
    check(x, 0, q, 0.125, rows, qs, gs, [-1, 1 << 30])
    check(x, 0, q, 0.125, [rows[0], -1, 1 << 20, rows[3]], qs, gs, [29, 12])
    check(x, 0, q, 0.125, rows, qs, [0, 0, 4], [29, 12])  # an empty group


def test_pages_outside_the_pool():
    rng = np.random.default_rng(8)
    for P in (8, 32):
        c, rows = build(rng, 1, 64, 64, P, [90], [[4, 40, 9]])
        c.tables[rows[0], 1], c.tables[rows[1], 2], c.tables[rows[2], 90 // P] = -1, c.N, 1 << 30
        q = queries(rng, 3, 2, 64)
        st, _, _ = check(QuantPair(c, 64, 64), 0, q, 0.125, rows, np.arange(4), [0, 3], [64])
        assert st == pc.BAD_PAGE
        c.tables[rows[1], :] = -1  # a row with no page at all
        check(QuantPair(c, 64, 64), 0, q, 0.125, rows, np.arange(4))


@pytest.mark.parametrize("G,hints", [(2, (2, 30, 40)), (2, (2, 0, 1 << 21)), (2, (2, 1 << 20, 1 << 21)),
                                     (40, (40, 30, 40)), (40, (40, 1 << 20, 1 << 21))])
def test_extreme_numbers_in_lists_stay_in_bounds(G, hints):
    """Starts that descend or leave the batch or whose differences pass 32 bits, lengths, rows and
    prefixes at both ends of the type: nothing outside the outputs is touched, and a sequence
    whose numbers are right is computed."""
    rng = np.random.default_rng(22)
    c, rows = build(rng, 1, 64, 64, 8, [30], [[4, 6, 9]])
    x = QuantPair(c, 64, 64)
    q = queries(rng, 6, G, 64)
    t, lo, hi = x.t, -(1 << 31), (1 << 31) - 1
    for qs in ([0, 4, 2, 6], [-5, 1, 2, 3], [0, 1, 2, 60], [9, 9, 9, 9], [1, lo, 0, 2], [0, 2, lo, hi], [hi, lo, lo, 3],
               [lo, hi, 1, lo], [3, 5, hi, lo + 3]):
        for gs, pl in (([0, 3], [25]), ([0, 3], [hi]), ([lo, hi], [lo]), ([1, lo], [hi]), ([2, 1], [25]), (None, None)):
            big = t.full((8, G, 64), 55.0, dtype=t.float16, device="cuda")
            gpu_attention(x, 0, q, 0.125, rows, qs, gs, pl, hints=hints, out=big[1:7])
            assert (big[0] == 55.0).all() and (big[7] == 55.0).all(), (qs, gs, pl)
            for rr in ([lo, rows[1], hi], None):
                gpu_attention(x, 0, q, 0.125, rr, [0, 2, 4, 6], gs, pl, hints=hints, out=big[1:7])
                assert (big[0] == 55.0).all() and (big[7] == 55.0).all(), (qs, gs, pl)
    # descending starts: the second sequence has no queries, the third's are its own
    _, out, lse = gpu_attention(x, 0, q, 0.125, rows, [1, lo, 2, 5], None, None, hints=hints)
    ost, recs = oracle(x, 0, q, 0.125, [rows[2]], [2, 5])
    out[[0, 1, 5]], lse[[0, 1, 5]] = 123.0, 321.0
    compare((ost, out, lse), (ost, recs), q)
    x.lens.copy_(t.tensor([lo, hi] + [hi] * (len(x.o.lens) - 2), dtype=t.int32))
    st, out, lse = gpu_attention(x, 0, q, 0.125, rows, [0, 2, 4, 6], None, None, hints=hints)
    assert st == pc.REFUSED and (out == 0).all() and (lse == -np.inf).all()


def test_strides_and_no_lse():
    """q as a slice of a wider projection, out inside a wider buffer."""
    rng = np.random.default_rng(12)
    c, rows = build(rng, 1, 128, 64, 16, [70], [[5, 12, 1]])
    x = QuantPair(c, 128, 64)
    t, H, d = x.t, 4, 64
    wide = gu.to_dev(rng.standard_normal((3, 2 * H * d + 24)).astype(np.float16))
    qd = wide[:, 8:8 + H * d].view(3, H, d)
    buf = t.full((3, 2 * H * d), 9.0, dtype=t.float16, device="cuda")
    out = buf[:, H * d:].view(3, H, d)
    ws = t.empty(x.cg.cg_quant_attention_workspace(x.cache, 3, H, 3, 1, 1, 70, 82), dtype=t.uint8, device="cuda")
    args = (0.125, x.i32(rows), x.i32([0, 1, 2, 3]), x.i32([0, 3]), x.i32([70]), 1, 70, 82)
    x.cg.cg_quant_attention_async(x.cache, 0, qd, out, *args, ws)
    t.cuda.synchronize()
    q = qd.cpu().numpy()
    compare((0, out.cpu().numpy(), None), oracle(x, 0, q, 0.125, rows, [0, 1, 2, 3], [0, 3], [70]), q)
    assert (buf[:, :H * d] == 9.0).all()
    with pytest.raises(ValueError):
        x.cg.cg_quant_attention_async(x.cache, 0, qd.float(), out, *args, ws)
    with pytest.raises(x.cg.CgError):
        x.cg.cg_quant_attention_async(x.cache, 0, qd, out, *args, ws[:0])
    with pytest.raises(x.cg.CgError):  # another head dimension than the cache's
        x.cg.cg_quant_attention_async(x.cache, 0, qd.reshape(3, 8, 32), out.reshape(3, 8, 32), *args, ws)


def test_streams_and_repeats():
    """The same bits each time, on the default and another stream."""
    rng = np.random.default_rng(13)
    tails = [[30, 1, 500], [2, 64]]
    c, rows = build(rng, 1, 256, 64, 16, [900, 65], tails)
    x = QuantPair(c, 256, 64)
    q = queries(rng, 5, 8, 64)
    args = (0, q, 0.125, rows, np.arange(6), group_starts_of(tails), [900, 65])
    st, out, lse = gpu_attention(x, *args)
    compare((st, out, lse), oracle(x, *args), q)
    side = x.t.cuda.Stream()
    x.t.cuda.synchronize()
    for s in (None, side, None, side):
        st, o, l = gpu_attention(x, *args, stream=s)
        assert st == 0 and gu.same_bits(o, out) and np.array_equal(l, lse)


def test_two_calls_at_once():
    """On two streams, each with its workspace, over one cache."""
    rng = np.random.default_rng(17)
    tails = [[30, 1, 500], [2, 64]]
    c, rows = build(rng, 2, 256, 64, 16, [900, 65], tails)
    x = QuantPair(c, 256, 64)
    t, cg = x.t, x.cg
    numbers = (5, 8, 5, 2, 1, 900, 1400)
    calls = []
    for layer in (0, 1):
        q = queries(rng, 5, 8, 64)
        calls.append(dict(layer=layer, q=q, qd=gu.to_dev(q), out=gu.to_dev(np.zeros_like(q)),
                          lse=t.zeros((5, 8), dtype=t.float32, device="cuda"), stream=t.cuda.Stream(),
                          ws=t.empty(cg.cg_quant_attention_workspace(x.cache, *numbers), dtype=t.uint8, device="cuda")))
    lists = [x.i32(y) for y in (rows, np.arange(6), group_starts_of(tails), [900, 65])]
    t.cuda.synchronize()
    for _ in range(5):
        for y in calls:
            cg.cg_quant_attention_async(x.cache, y["layer"], y["qd"], y["out"], 0.125, *lists, *numbers[4:], y["ws"],
                                        lse=y["lse"], stream=y["stream"])
    t.cuda.synchronize()
    for y in calls:
        want = oracle(x, y["layer"], y["q"], 0.125, rows, np.arange(6), group_starts_of(tails), [900, 65])
        compare((int(x.status.item()), y["out"].cpu().numpy(), y["lse"].cpu().numpy()), want, y["q"])


def test_most_heads():
    """1,024 query heads of one kv head: more row tiles than one workgroup's."""
    rng = np.random.default_rng(18)
    c, rows = build(rng, 1, 16, 16, 16, [70], [[5, 33]])
    check(QuantPair(c, 16, 16), 0, queries(rng, 3, 1024, 16), 0.25, rows, [0, 1, 3], [0, 2], [70])


@pytest.mark.parametrize("heads", [1, 64])
def test_longest_row(heads):
    """Rows of 2^30 tokens, all of whose table entries name one page.  Keys are 0, so all
    weights are one power of two and their sums exact; values repeat, small whole numbers."""
    import kv_cache_compression_anchor_amd as cg
    t = gu.torch()
    P, B, d = 65536, 16384, 64
    n = P * B
    row = 2 * cg.cg_quant_row(d, d)
    pools = t.zeros((2, 1, 2, P, row), dtype=t.uint8, device="cuda")
    tables = t.zeros((2, B), dtype=t.int32, device="cuda")
    lens = t.tensor([n, n], dtype=t.int32, device="cuda")
    refs = t.tensor([B, 0], dtype=t.int32, device="cuda")
    status = t.zeros(1, dtype=t.int32, device="cuda")
    c = cg.QuantCache(pools[0], pools[1], tables, lens, refs, status, d, d)
    k = t.zeros((1, 2 * P, d), dtype=t.float16, device="cuda")
    v = t.full((1, 2 * P, d), 7.0, dtype=t.float16, device="cuda")
    v[0, ::8, 1::2] = -7.0 * 7  # one token in eight: the mean is 0
    cg.cg_quant_write_async(c, 0, t.arange(2 * P, device="cuda"), k, v)
    i32 = lambda y: t.tensor(y, dtype=t.int32, device="cuda")  # noqa: E731
    q = t.randn((2, heads, d), device="cuda").half()
    for groups, prefix in ((None, None), ([0, 2], [n - P])):
        hint = 0 if prefix is None else prefix[0]
        numbers = (2, heads, 2, 0 if prefix is None else 1, 1, hint, n)
        ws = t.full((cg.cg_quant_attention_workspace(c, *numbers),), 0xFF, dtype=t.uint8, device="cuda")
        out = t.full((2, heads, d), 9.0, dtype=t.float16, device="cuda")
        lse = t.zeros((2, heads), dtype=t.float32, device="cuda")
        opt = lambda y: None if y is None else i32(y)  # noqa: E731
        cg.cg_quant_attention_async(c, 0, q, out, 0.125, None, i32([0, 1, 2]), opt(groups), opt(prefix), 1, hint, n,
                                    ws, lse=lse)
        t.cuda.synchronize()
        assert int(status.item()) == 0
        assert (out[..., ::2] == 7).all() and (out[..., 1::2] == 0).all()
        # log 2^30 with log2f's and one product's roundings
        assert ((lse - 30 * np.log(2)).abs() <= 4 * 2.0 ** -24 * 30).all()


def test_pool_past_four_gib():
    import kv_cache_compression_anchor_amd as cg
    t = gu.torch()
    N, P, C, d = 240000, 32, 1024, 128
    k, v = (t.empty((1, N, P, 576), dtype=t.uint8, device="cuda") for _ in range(2))
    tables = t.arange(N - 6, N, dtype=t.int32, device="cuda").repeat(2, 1).contiguous()
    lens = t.tensor([180, 170], dtype=t.int32, device="cuda")
    refs, status = t.ones(N, dtype=t.int32, device="cuda"), t.zeros(1, dtype=t.int32, device="cuda")
    cache = cg.QuantCache(k, v, tables, lens, refs, status, C, d)
    new = t.randn((2, 1, 6 * P, C), device="cuda").half()
    cg.cg_quant_write_async(cache, 0, t.arange((N - 6) * P, N * P, device="cuda"), new[0], new[1])
    host = pc.Cache(k[:, N - 6:].cpu().numpy().view(np.float16), v[:, N - 6:].cpu().numpy().view(np.float16),
                    np.tile(np.arange(6, dtype=np.int32), (2, 1)), lens.cpu().numpy(), np.ones(6, np.int32))
    q = queries(np.random.default_rng(16), 2, 8, 128)
    ws = t.empty(cg.cg_quant_attention_workspace(cache, 2, 8, 2, 1, 1, 100, 180), dtype=t.uint8, device="cuda")
    out, lse = gu.to_dev(np.zeros_like(q)), t.zeros((2, 8), dtype=t.float32, device="cuda")
    i32 = lambda x: t.tensor(x, dtype=t.int32, device="cuda")  # noqa: E731
    cg.cg_quant_attention_async(cache, 0, gu.to_dev(q), out, 0.088, None, i32([0, 1, 2]), i32([0, 2]), i32([100]),
                                1, 100, 180, ws, lse=lse)
    t.cuda.synchronize()
    want = pc.attention(qc.held(host, C, d), 0, q, 0.088, None, [0, 1, 2], [0, 2], [100])
    compare((int(status.item()), out.cpu().numpy(), lse.cpu().numpy()), want, q)


def test_captured_decode_loop():
    """Reserve, write and attend in one graph: every replay is a decoding step, compared with
    the oracle, with eager work between the replays."""
    rng = np.random.default_rng(15)
    C, H, d = 128, 4, 64
    c, rows = build(rng, 2, C, d, 16, [100], [[3, 14, 30]], spare=10)
    x = QuantPair(c, C, d)
    t, cg = x.t, x.cg
    r, qs, gs, pl = x.i32(rows), x.i32([0, 1, 2, 3]), x.i32([0, 3]), x.i32([100])
    slots = t.empty(3, dtype=t.int64, device="cuda")
    kd, vd = (t.zeros((2, 3, C), dtype=t.float16, device="cuda") for _ in range(2))
    qd, out = (t.zeros((3, H, d), dtype=t.float16, device="cuda") for _ in range(2))
    lse = t.zeros((3, H), dtype=t.float32, device="cuda")
    ws = t.empty(cg.cg_quant_attention_workspace(x.cache, 3, H, 3, 1, 1, 100, 160), dtype=t.uint8, device="cuda")
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        cg.cg_pages_reserve_async(x.cache, r, qs, slots, x.ws)
        cg.cg_quant_write_async(x.cache, 0, slots, kd, vd)
        cg.cg_quant_attention_async(x.cache, 1, qd, out, 0.125, r, qs, gs, pl, 1, 100, 160, ws, lse=lse)
    for step in range(8):
        k, v = (rng.standard_normal((2, 3, C)).astype(np.float16) for _ in range(2))
        q = queries(rng, 3, H, d)
        for dst, src in ((kd, k), (vd, v), (qd, q)):
            dst.copy_(gu.to_dev(src))
        graph.replay()
        t.cuda.synchronize()
        st, want = pc.reserve(c, rows, [0, 1, 2, 3], 3)
        qc.write(c, C, d, 0, want, k, v)
        got = (int(x.status.item()), out.cpu().numpy(), lse.cpu().numpy())
        compare(got, oracle(x, 1, q, 0.125, rows, [0, 1, 2, 3], [0, 3], [100]), q)
        if step % 3 == 1:  # eager, in between
            check(x, 0, q, 0.125, rows, [0, 1, 2, 3], [0, 3], [100])
