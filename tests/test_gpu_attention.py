"""The attention over a paged cache against the oracle's binary64 one.

Bound of one output, in exact arithmetic of the stated roundings (u = 2^-11 is
binary16's half step, e = 2^-24 binary32's): the weights are rounded to binary16
(relative u, and absolutely 2^-25 of the largest weight below binary16's normal
range), scores are binary32 sums of d products of size at most S = max scale
sum |q k|, so that a weight is off by a factor exp(+-D), D = e (d + 16) (S + 1)
with the exponential's own error, binary32 sums over n tokens add e (n + 64), and
the result is rounded once: u |out| + 2^-25.  With A = sum p |v|:
    |out - o| <= u |o| + (u + 4 D + 2 e (n + 64)) A + n 2^-25 max|v| / l + 2^-25
    |lse - x| <= 2 D + e (n + 64) + 4 e |x|
(l = sum exp(s - max) >= 1)."""
import numpy as np
import pytest

from oracle import paged_cache as pc
from tests import gpu_util as gu
from tests.test_gpu_pages import Pair

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -11, 2.0 ** -24


def build(rng, L, C, P, prefixes, tails, spare=3, spread=1.0):
    """A cache in which group g's sequences continue a prefix of prefixes[g] tokens
    by tails[g][i] tokens, made with the page operators of the oracle."""
    seqs = [(g, n) for g, t in enumerate(tails) for n in t]
    R = len(seqs)
    longest = max(prefixes[g] + n for g, n in seqs)
    pages = sum(-(-(prefixes[g] + n) // P) + 1 for g, n in seqs) + spare
    c = pc.empty(L, pages, P, C, R + 2, -(-longest // P) + 2)
    order = rng.permutation(R + 2)[:R]
    first, rows = {}, []

    def add(row, n):
        st, slots = pc.reserve(c, [row], [0, n], n)
        assert st == 0
        k, v = ((spread * rng.standard_normal((L, n, C))).astype(np.float16) for _ in range(2))
        pc.write(c, 0, slots, k, v)

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


def gpu_attention(x, layer, q, scale, rows, q_starts, group_starts, prefix_lens, hints=None, lse=True,
                  out=None, stream=None):
    cg, t = x.cg, x.t
    n_q, H, d = q.shape
    lens = x.o.lens
    hints = hints or (max(1, int(np.max(np.diff(q_starts), initial=0))),
                      int(np.max(prefix_lens, initial=0)) if prefix_lens is not None else 0,
                      int(np.max(lens)))
    hints = tuple(max(0, h) for h in hints)
    groups = 0 if group_starts is None else len(group_starts) - 1
    ws = t.full((cg.cg_attention_workspace(x.cache, n_q, H, d, len(q_starts) - 1, groups, *hints),), 0xFF,
                dtype=t.uint8, device="cuda")
    qd = gu.to_dev(q)
    if out is None:
        out = t.full((n_q, H, d), 123.0, dtype=t.float16, device="cuda")
    ld = t.full((n_q, H), 321.0, dtype=t.float32, device="cuda") if lse else None
    opt = lambda v: None if v is None else x.i32(v)  # noqa: E731
    cg.cg_attention_prefix_async(x.cache, layer, qd, out, scale, opt(rows), x.i32(q_starts),
                                 opt(group_starts), opt(prefix_lens), *hints, ws, lse=ld, stream=stream)
    t.cuda.synchronize()
    st = int(x.status.item())
    x.status.zero_()
    return st, out.cpu().numpy(), None if ld is None else ld.cpu().numpy()


def compare(got, want, q):
    (st, out, lse), (ost, recs) = got, want
    assert st == ost, (st, ost)
    n_q, H, d = q.shape
    for j in range(n_q):
        if j not in recs:  # no sequence's query
            assert (out[j] == 123.0).all() and (lse is None or (lse[j] == 321.0).all()), j
            continue
        for h, r in enumerate(recs[j]):
            if r["lse"] == -np.inf:
                assert (out[j, h] == 0).all(), (j, h)
                assert lse is None or lse[j, h] == -np.inf
                continue
            n = r["tokens"]
            D = E * (d + 16) * (r["size"] + 1)
            tol = (U * np.abs(r["out"]) + (U + 4 * D + 2 * E * (n + 64)) * r["mean_abs"]
                   + n * 2.0 ** -25 * r["vmax"] / r["l"] + 2.0 ** -25)
            off = np.abs(out[j, h].astype(np.float64) - r["out"])
            assert (off <= tol).all(), (j, h, n, float((off / tol).max()))
            if lse is not None:
                assert abs(lse[j, h] - r["lse"]) <= 2 * D + E * (n + 64) + 4 * E * abs(r["lse"]), (j, h)


def check(x, layer, q, scale, rows, q_starts, group_starts=None, prefix_lens=None, **kw):
    got = gpu_attention(x, layer, q, scale, rows, q_starts, group_starts, prefix_lens, **kw)
    want = pc.attention(x.o, layer, q, scale, rows, q_starts, group_starts, prefix_lens)
    compare(got, want, q)
    if not kw:  # and as a long context is computed: prefixes shared, tokens split, sums joined
        most = max(1, int(np.max(np.diff(q_starts), initial=0)))
        for hints in ((most, 1 << 20, 1 << 21), (most, 0, 1 << 21)):
            compare(gpu_attention(x, layer, q, scale, rows, q_starts, group_starts, prefix_lens, hints=hints),
                    want, q)
    return got


def queries(rng, n, H, d):
    return rng.standard_normal((n, H, d)).astype(np.float16)


def starts_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def group_starts_of(tails):
    return starts_of([len(t) for t in tails])


# heads: kv heads, query heads per kv head, head dimension
@pytest.mark.parametrize("kv,G,d", [(2, 1, 64), (1, 4, 128), (3, 7, 80), (2, 8, 128), (1, 2, 256), (1, 1, 8),
                                    (2, 5, 40), (1, 3, 192), (4, 17, 64), (1, 70, 128)])
@pytest.mark.parametrize("P", [1, 16, 128])
def test_heads_and_pages(kv, G, d, P):
    rng = np.random.default_rng(kv * 10007 + G * 101 + d + P)
    tails = [[1, 5, 40], [2, 33]]
    c, rows = build(rng, 2, kv * d, P, [50, 37], tails)
    x = Pair(c)
    q = queries(rng, 5, kv * G, d)
    check(x, 1, q, d ** -0.5, rows, np.arange(6), group_starts_of(tails), [50, 37])
    check(x, 0, q, d ** -0.5, rows, np.arange(6))


@pytest.mark.parametrize("prefix", [1, 15, 16, 63, 64, 65, 127, 128, 200, 257, 1000])
@pytest.mark.parametrize("tail", [[1], [1, 2, 3], [16, 17, 64, 65, 300]])
def test_lengths(prefix, tail):
    rng = np.random.default_rng(prefix * 31 + len(tail))
    c, rows = build(rng, 1, 128, 16, [prefix], [tail])
    x = Pair(c)
    q = queries(rng, len(tail), 4, 64)
    check(x, 0, q, 0.125, rows, np.arange(len(tail) + 1), [0, len(tail)], [prefix])
    # the same by themselves, and with part of the prefix shared
    check(x, 0, q, 0.125, rows, np.arange(len(tail) + 1))
    check(x, 0, q, 0.125, rows, np.arange(len(tail) + 1), [0, len(tail)], [prefix - prefix // 3])


@pytest.mark.parametrize("counts", [[1, 1, 1], [4, 0, 2], [0, 0, 1], [9, 30, 17], [64, 65, 1], [130, 3, 0]])
@pytest.mark.parametrize("G", [1, 4])
def test_several_queries(counts, G):
    """Drafts and prompts: a sequence's queries see one token more each."""
    rng = np.random.default_rng(sum(counts) * 10 + G)
    tails = [[max(1, counts[0]) + 3, max(1, counts[1])], [max(1, counts[2]) + 70]]
    c, rows = build(rng, 1, 256, 8, [45, 20], tails)
    x = Pair(c)
    q = queries(rng, sum(counts) + 3, 2 * G, 128)  # three rows behind the last sequence
    check(x, 0, q, 0.09, rows, starts_of(counts), group_starts_of(tails), [45, 20])
    check(x, 0, q, 0.09, rows, starts_of(counts))


def test_wrong_hints_change_nothing():
    rng = np.random.default_rng(3)
    tails = [[5, 300, 40], [1, 2]]
    c, rows = build(rng, 1, 128, 16, [700, 90], tails)
    x = Pair(c)
    counts = [5, 70, 1, 1, 2]
    q = queries(rng, sum(counts), 4, 64)
    for hints in ((0, 0, 0), (1, 1, 1), (1, 100000, 200000), (5000, 700, 1000), (70, 10, 1 << 30),
                  (1 << 20, 1 << 30, 1 << 30)):
        check(x, 0, q, 0.125, rows, starts_of(counts), group_starts_of(tails), [700, 90], hints=hints)


def test_many_sequences():
    """Groups of one, an uneven batch, more groups than a wavefront has lanes."""
    rng = np.random.default_rng(4)
    tails = [[int(rng.integers(1, 40)) for _ in range(rng.integers(1, 4))] for _ in range(80)]
    prefixes = [int(rng.integers(1, 50)) for _ in tails]
    c, rows = build(rng, 1, 64, 8, prefixes, tails)
    x = Pair(c)
    n = len(rows)
    q = queries(rng, n, 2, 64)
    check(x, 0, q, 0.125, rows, np.arange(n + 1), group_starts_of(tails), prefixes)
    # some sequences in no group
    gs = group_starts_of(tails)
    check(x, 0, q, 0.125, rows, np.arange(n + 1), gs[10:41], prefixes[10:40])


@pytest.mark.parametrize("seqs,kv,G,d", [(130, 4, 2, 40), (129, 6, 3, 128), (256, 4, 1, 64), (70, 8, 4, 32),
                                         (131, 4, 2, 200)])
def test_many_sequences_of_several_heads(seqs, kv, G, d):
    """A batch whose workgroups take two or four kv heads each, with what is no finite
    number behind the rows' ends and, for the last head, in a token of the first row."""
    rng = np.random.default_rng(seqs + d)
    tails = [[int(n) for n in rng.integers(2, 20, seqs // 2)], [int(n) for n in rng.integers(2, 150, seqs - seqs // 2)]]
    c, rows = build(rng, 1, kv * d, 8, [21, 9], tails)
    gone = rows[seqs // 3]
    c.tables[gone, 3] = -1
    counts = rng.integers(0, 3, seqs)
    n = int(counts.sum())
    x = Pair(c)
    q = queries(rng, n, kv * G, d)
    starts = starts_of(counts)
    check(x, 0, q, d ** -0.5, rows, starts, group_starts_of(tails), [21, 9])
    check(x, 0, q, d ** -0.5, rows, starts)
    counts[0], counts[1:] = 2, 1
    n = int(counts.sum())
    q, starts = queries(rng, n, kv * G, d), starts_of(counts)
    ost, recs = pc.attention(c, 0, q, d ** -0.5, rows, starts)
    last = int(c.lens[rows[0]]) - 1  # only the second query of the first sequence sees it
    c.v[0, c.tables[rows[0], last // 8], last % 8, (kv - 1) * d + 3] = np.inf
    for row in range(len(c.tables)):
        for t in range(int(c.lens[row]), 8 * c.tables.shape[1]):
            page = c.tables[row, t // 8]
            if page >= 0 and c.refs[page] == 1:
                c.k[0, page, t % 8] = c.v[0, page, t % 8] = np.nan
    for hints in (None, (2, 0, 1 << 21)):
        st, out, lse = gpu_attention(Pair(c), 0, q, d ** -0.5, rows, starts, None, None, hints=hints)
        hit = out[1, (kv - 1) * G:, 3]
        assert (hit == np.inf).all()
        for h in range((kv - 1) * G, kv * G):
            out[1, h, 3] = recs[1][h]["out"][3]
        compare((st, out, lse), (ost, recs), q)


def test_group_of_many():
    """More rows than one tile of the shared part: 70 sequences of 4 heads, ragged queries."""
    rng = np.random.default_rng(14)
    tails = [[int(n) for n in rng.integers(3, 30, 70)]]
    c, rows = build(rng, 1, 128, 16, [333], tails)
    x = Pair(c)
    counts = rng.integers(0, 4, 70)
    q = queries(rng, int(counts.sum()), 8, 64)
    check(x, 0, q, 0.125, rows, starts_of(counts), [0, 70], [333])


@pytest.mark.parametrize("kv,G,d,P,prefix,seqs", [
    (2, 4, 128, 16, 1500, 40), (1, 8, 128, 8, 1111, 20), (1, 3, 64, 64, 2047, 25), (1, 5, 64, 8, 1300, 50),
    (2, 2, 256, 16, 1200, 40), (1, 6, 80, 16, 1055, 30), (1, 4, 128, 1, 1100, 33), (1, 5, 96, 4, 700, 30),
    (1, 4, 128, 4, 900, 12), (1, 2, 256, 128, 1900, 9), (4, 8, 64, 32, 3200, 16)])
def test_long_shared_prefix(kv, G, d, P, prefix, seqs):
    """The rounds of a ring of tiles over several splits, for each width of head and
    number of rows, pages that they take and that they do not."""
    rng = np.random.default_rng(prefix + d)
    tails = [[int(n) for n in rng.integers(2, 60, seqs)]]
    c, rows = build(rng, 1, kv * d, P, [prefix], tails)
    x = Pair(c)
    counts = rng.integers(0, 3, seqs)
    q = queries(rng, int(counts.sum()), kv * G, d)
    check(x, 0, q, d ** -0.5, rows, starts_of(counts), [0, seqs], [prefix])
    # a page of the prefix outside the pool, in the middle of a round
    c.tables[rows[0], (prefix // 2) // P] = -1
    check(Pair(c), 0, q, d ** -0.5, rows, starts_of(counts), [0, seqs], [prefix])


@pytest.mark.parametrize("d,G,P", [(128, 4, 16), (64, 9, 8), (256, 2, 32), (72, 3, 16)])
def test_long_prompts(d, G, P):
    """Sequences whose queries are a prompt of hundreds of tokens, behind a context."""
    rng = np.random.default_rng(d)
    tails = [[300, 140], [33]]
    c, rows = build(rng, 1, d, P, [420, 64], tails)
    counts = [260, 131, 33]
    q = queries(rng, sum(counts), G, d)
    check(Pair(c), 0, q, d ** -0.5, rows, starts_of(counts), [0, 2, 3], [420, 64])
    check(Pair(c), 0, q, d ** -0.5, rows, starts_of(counts))


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_masked_places_in_many_rows(bad):
    """Values that are no finite number in a prompt's own tokens: the queries before
    them are not touched, those behind them get what the formula says."""
    rng = np.random.default_rng(21)
    c, rows = build(rng, 1, 128, 16, [300], [[200, 90]])
    want = c.copy()
    counts = [150, 70]
    hit = {0: [100, 120], 1: [40]}  # queries of a sequence whose own token is bad
    for s, js in hit.items():
        for j in js:
            t = int(c.lens[rows[s]]) - counts[s] + j
            c.v[0, c.tables[rows[s], t // 16], t % 16, ::5] = bad
    x = Pair(c)
    q = queries(rng, sum(counts), 4, 64)
    base = [0, counts[0]]
    _, recs = pc.attention(want, 0, q, 0.125, rows, starts_of(counts), [0, 2], [300])
    spoilt = np.zeros(128, bool)
    spoilt[::5] = True
    for hints in (None, (150, 1 << 20, 1 << 21), (150, 0, 1 << 21)):
        st, out, lse = gpu_attention(x, 0, q, 0.125, rows, starts_of(counts), [0, 2], [300], hints=hints)
        assert st == 0
        for s in (0, 1):
            first = base[s] + min(hit[s])
            for j in range(base[s], base[s] + counts[s]):
                for h in range(4):
                    ch = spoilt[64 * (h // 2):64 * (h // 2) + 64]
                    if j >= first:  # those channels, and no other
                        assert not np.isfinite(out[j, h][ch]).any()
                        out[j, h][ch] = recs[j][h]["out"][ch]
                    assert np.isfinite(out[j, h]).all()
        compare((st, out, lse), (0, recs), q)


def test_rows_default_and_empty_rows():
    rng = np.random.default_rng(5)
    x = Pair(pc.empty(1, 30, 16, 64, 4, 6))
    x.new(rng, [0, 2], [20, 3])
    q = queries(rng, 8, 1, 64)
    # rows 1 and 3 are empty: their queries see nothing; row 2 has more queries than tokens
    check(x, 0, q, 0.125, None, [0, 1, 2, 7, 8])
    check(x, 0, q, 0.125, [1], [0, 8])


def test_refused_sequences():
    rng = np.random.default_rng(6)
    tails = [[4, 1, 9], [3]]
    c, rows = build(rng, 1, 64, 8, [30, 12], tails)
    x = Pair(c)
    q = queries(rng, 9, 2, 64)
    qs, gs = [0, 2, 4, 7, 9], [0, 3, 4]
    # the second sequence's two queries start before token 30 + 1
    st, out, _ = check(x, 0, q, 0.125, rows, qs, gs, [30, 12])
    assert st == pc.REFUSED and (out[2:4] == 0).all()
    check(x, 0, q, 0.125, rows, qs, gs, [29, 12])
    check(x, 0, q, 0.125, rows, qs, gs, [33, 16])     # longer than the rows
    check(x, 0, q, 0.125, rows, qs, gs, [-1, 1 << 30])
    check(x, 0, q, 0.125, [rows[0], -1, 1 << 20, rows[3]], qs, gs, [29, 12])
    check(x, 0, q, 0.125, rows, qs, [0, 0, 4], [29, 12])  # an empty group


def test_malformed_lists_stay_in_bounds():
    """Starts that descend or leave the batch: no value is promised, but nothing
    outside the outputs is touched and the call comes back."""
    rng = np.random.default_rng(7)
    c, rows = build(rng, 1, 64, 8, [30], [[4, 6, 9]])
    x = Pair(c)
    q = queries(rng, 6, 2, 64)
    t = x.t
    for qs in ([0, 4, 2, 6], [-5, 1, 2, 3], [0, 1, 2, 60], [3, 3, 3, 3], [9, 9, 9, 9], [5, 4, 3, 2]):
        for gs, pl in (([0, 3], [25]), ([-4, 3], [25]), ([2, 1], [25]), ([0, 50], [25]), ([1, 9], [1 << 30])):
            big = t.full((8, 2, 64), 55.0, dtype=t.float16, device="cuda")
            gpu_attention(x, 0, q, 0.125, rows, qs, gs, pl, hints=(2, 30, 40), out=big[1:7])
            assert (big[0] == 55.0).all() and (big[7] == 55.0).all()


@pytest.mark.parametrize("G,hints", [(2, (2, 30, 40)), (2, (2, 0, 1 << 21)), (2, (2, 1 << 20, 1 << 21)),
                                     (20, (40, 30, 40)), (20, (40, 1 << 20, 1 << 21))])
def test_extreme_numbers_in_lists_stay_in_bounds(G, hints):
    """Starts whose differences pass 32 bits, lengths, rows and prefixes at both ends of
    the type: nothing outside the outputs is touched, and a sequence whose numbers are
    right is computed."""
    rng = np.random.default_rng(22)
    c, rows = build(rng, 1, 64, 8, [30], [[4, 6, 9]])
    x = Pair(c)
    q = queries(rng, 6, G, 64)
    t, lo, hi = x.t, -(1 << 31), (1 << 31) - 1
    for qs in ([1, lo, 0, 2], [0, 2, lo, hi], [hi, lo, lo, 3], [2, lo + 1, hi, 6], [lo, hi, 1, lo], [3, 5, hi, lo + 3]):
        for gs, pl in (([0, 3], [25]), ([0, 3], [hi]), ([lo, hi], [lo]), ([1, lo], [hi]), (None, None)):
            big = t.full((8, G, 64), 55.0, dtype=t.float16, device="cuda")
            gpu_attention(x, 0, q, 0.125, rows, qs, gs, pl, hints=hints, out=big[1:7])
            assert (big[0] == 55.0).all() and (big[7] == 55.0).all(), (qs, gs, pl)
            for rr in ([lo, rows[1], hi], None):
                gpu_attention(x, 0, q, 0.125, rr, [0, 2, 4, 6], gs, pl, hints=hints, out=big[1:7])
                assert (big[0] == 55.0).all() and (big[7] == 55.0).all(), (qs, gs, pl)
    # descending starts: the second sequence has no queries, the third's are its own
    _, out, lse = gpu_attention(x, 0, q, 0.125, rows, [1, lo, 2, 5], None, None, hints=hints)
    ost, recs = pc.attention(c, 0, q, 0.125, [rows[2]], [2, 5])
    out[[0, 1, 5]], lse[[0, 1, 5]] = 123.0, 321.0
    compare((ost, out, lse), (ost, recs), q)
    x.lens.copy_(t.tensor([lo, hi] + [hi] * (len(x.o.lens) - 2), dtype=t.int32))
    st, out, lse = gpu_attention(x, 0, q, 0.125, rows, [0, 2, 4, 6], None, None, hints=hints)
    assert st == pc.REFUSED and (out == 0).all() and (lse == -np.inf).all()


def test_pages_outside_the_pool():
    rng = np.random.default_rng(8)
    tails = [[4, 40, 9]]
    c, rows = build(rng, 1, 64, 8, [30], tails)
    c.tables[rows[0], 1], c.tables[rows[1], 5], c.tables[rows[2], 4] = -1, c.N, 1 << 30
    x = Pair(c)
    q = queries(rng, 3, 2, 64)
    st, _, _ = check(x, 0, q, 0.125, rows, np.arange(4), [0, 3], [24])
    assert st == pc.BAD_PAGE
    # a row with no page at all
    c.tables[rows[1], :] = -1
    check(Pair(c), 0, q, 0.125, rows, np.arange(4))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_masked_places_have_no_influence(bad):
    """NaN and infinities behind the rows' ends, in free pages, and in tokens that
    later queries of the same sequence see but earlier ones do not."""
    rng = np.random.default_rng(9)
    tails = [[7, 20, 33]]
    counts = [5, 3, 2]
    c, rows = build(rng, 1, 128, 16, [50], tails)
    want = c.copy()
    used = np.zeros((c.N, c.P), bool)
    for r in rows:
        tt = np.arange(c.lens[r])
        used[c.tables[r, tt // c.P], tt % c.P] = True
    for x in (c.k, c.v):
        x[0][~used] = bad
    q = queries(rng, 10, 2, 128)
    check(Pair(c), 0, q, 0.09, rows, starts_of(counts), [0, 3], [50])
    # the last token of each sequence: only its last query sees it
    for r in rows:
        n = int(c.lens[r]) - 1
        c.v[0, c.tables[r, n // c.P], n % c.P, ::3] = bad
        c.k[0, c.tables[r, n // c.P], n % c.P, 5] = bad
    for groups in (([0, 3], [50]), (None, None)):
        st, out, lse = gpu_attention(Pair(c), 0, q, 0.09, rows, starts_of(counts), *groups)
        _, recs = pc.attention(want, 0, q, 0.09, rows, starts_of(counts), *groups)
        early = [j for s in range(3) for j in range(sum(counts[:s]), sum(counts[:s + 1]) - 1)]
        for j in range(10):
            if j not in early:
                recs.pop(j)
                out[j], lse[j] = 123.0, 321.0
        compare((st, out, lse), (0, recs), q)


def test_infinite_scores():
    """Scores of -infinity weigh nothing; a row of nothing else gives zeros; NaN in a
    visible token is an output of NaN."""
    rng = np.random.default_rng(10)
    c, rows = build(rng, 1, 64, 16, [40], [[3, 5, 6]])
    q = np.abs(queries(rng, 3, 1, 64))
    for t in range(0, 40, 2):  # every other token of the prefix
        c.k[0, c.tables[rows[0], t // 16], t % 16, :] = -np.inf
    x = Pair(c)
    st, out, lse = gpu_attention(x, 0, q, 0.125, rows, np.arange(4), [0, 3], [40])
    _, recs = pc.attention(c, 0, q, 0.125, rows, np.arange(4), [0, 3], [40])
    for j in range(3):
        for r in recs[j]:
            r["size"] = 30.0  # the finite scores' size
    compare((st, out, lse), (0, recs), q)
    c.k[:] = -np.inf
    st, out, lse = gpu_attention(Pair(c), 0, q, 0.125, rows, np.arange(4), [0, 3], [40])
    assert (out == 0).all() and (lse == -np.inf).all()
    c, rows = build(rng, 1, 64, 16, [40], [[3, 5, 6]])
    c.k[0, c.tables[rows[1], 44 // 16], 44 % 16, 3] = np.nan  # the second sequence's last token
    st, out, lse = gpu_attention(Pair(c), 0, q, 0.125, rows, np.arange(4), [0, 3], [40])
    assert np.isnan(out[1]).all() and np.isnan(lse[1]).all()
    assert np.isfinite(out[[0, 2]]).all()


# the lengths'; one kernel; prefixes shared and sums joined; joined
ALL_HINTS = (None, (5, 0, 0), (5, 1 << 20, 1 << 21), (5, 0, 1 << 21))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("kv,G,d", [(2, 1, 64), (1, 4, 128), (4, 2, 40), (1, 9, 128), (1, 20, 128), (1, 40, 64),
                                    (2, 1, 256), (1, 7, 256)])
def test_nothing_but_infinite_scores(kv, G, d, bad):
    """Queries that see only scores of -infinity get zeros whatever the values hold, in
    tiles that all queries see and in those that some do."""
    rng = np.random.default_rng(kv * 100 + G + d)
    c, rows = build(rng, 1, kv * d, 16, [100], [[5, 40]])
    c.k[..., ::d] = -np.inf  # the first channel of each head
    c.v[:, :, ::3, 1::7] = bad
    counts = [3, 5]
    q = queries(rng, sum(counts), kv * G, d)
    q[..., 0] = np.abs(q[..., 0]) + 0.5
    for groups in (([0, 2], [100]), (None, None)):
        for hints in ALL_HINTS:
            st, out, lse = gpu_attention(Pair(c), 0, q, d ** -0.5, rows, starts_of(counts), *groups, hints=hints)
            assert st == 0 and (out == 0).all() and (lse == -np.inf).all(), (groups, hints)


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("kv,G,d", [(2, 1, 64), (1, 4, 128), (1, 20, 128), (1, 40, 64), (1, 3, 256)])
def test_weights_of_zero_and_odd_values(kv, G, d, bad):
    """Zero times what is no finite number is none either: values of tokens whose scores
    are -infinity, which are whole splits of the tokens when they are joined, and those
    channels alone."""
    rng = np.random.default_rng(kv * 100 + G + d)
    c, rows = build(rng, 1, kv * d, 16, [400], [[5, 40]])
    want = c.copy()
    tt = np.arange(200)
    pages, at = c.tables[rows[0], tt // 16], tt % 16
    for x in (c, want):
        x.k[0, pages, at, ::d] = -np.inf
    odd = np.zeros(kv * d, bool)
    odd[2::7] = True
    c.v[0, pages[70], at[70], odd] = bad
    counts = [3, 5]
    q = queries(rng, sum(counts), kv * G, d)
    q[..., 0] = np.abs(q[..., 0]) + 0.5
    _, recs = pc.attention(want, 0, q, d ** -0.5, rows, starts_of(counts))
    finite = want.copy()  # for the size of the scores that are
    finite.k[0, pages, at, ::d] = 0
    _, sizes = pc.attention(finite, 0, q, d ** -0.5, rows, starts_of(counts))
    for j in recs:
        for r, x in zip(recs[j], sizes[j]):
            r["size"] = x["size"]
    for groups in (([0, 2], [400]), (None, None)):
        for hints in ALL_HINTS:
            st, out, lse = gpu_attention(Pair(c), 0, q, d ** -0.5, rows, starts_of(counts), *groups, hints=hints)
            for h in range(kv * G):
                ch = odd[h // G * d:h // G * d + d]
                assert not np.isfinite(out[:, h, ch]).any(), (groups, hints, h)
                for j in recs:
                    out[j, h, ch] = recs[j][h]["out"][ch]
            compare((st, out, lse), (0, recs), q)


@pytest.mark.parametrize("kv,G,d", [(2, 1, 64), (1, 4, 128), (1, 20, 128), (1, 40, 64), (1, 3, 256)])
@pytest.mark.parametrize("scale", [2.0 ** 126, -2.0 ** 126, 2.0 ** 127])
def test_scores_past_the_range(kv, G, d, scale):
    """A score past binary32's range is an infinity: exp(inf - inf) is no number, and a
    query of scores of -infinity alone gets zeros.  Products are +-d, so that every score
    passes the range by far; one query's products with the shared tokens have the other
    sign, and one's are all 0, whose scores are finite."""
    rng = np.random.default_rng(kv * 100 + G + d)
    c, rows = build(rng, 1, kv * d, 16, [300], [[5, 40]])
    c.k[:] = 1
    q = np.ones((6, kv * G, d), np.float16)
    q[1], q[4], q[5] = -1, -1, 0
    counts = [3, 3]
    for groups in (([0, 2], [300]), (None, None)):
        for hints in ALL_HINTS:
            st, out, lse = gpu_attention(Pair(c), 0, q, scale, rows, starts_of(counts), *groups, hints=hints)
            up = [0, 2, 3] if scale > 0 else [1, 4]
            down = [1, 4] if scale > 0 else [0, 2, 3]
            assert st == 0 and np.isnan(out[up]).all() and np.isnan(lse[up]).all(), (groups, hints)
            assert (out[down] == 0).all() and (lse[down] == -np.inf).all(), (groups, hints)
            mean = np.stack([c.v[0, c.tables[rows[1], t // 16], t % 16] for t in range(340)]).astype(np.float64)
            want = mean.mean(0).reshape(kv, 1, d)
            # equal weights of a power of two: the values' sum in binary32, n e A, and one rounding
            tol = U * np.abs(want) + 340 * E * np.abs(mean).mean(0).reshape(kv, 1, d) + 2.0 ** -25
            assert (np.abs(out[5].reshape(kv, G, d) - want) <= tol).all()
            assert np.abs(lse[5] - np.log(340)).max() <= 8 * E * np.log(340)


def test_large_scores_and_spread():
    """Peaked weights (one token takes all) and scores whose exponentials overflow
    without the maximum."""
    rng = np.random.default_rng(11)
    c, rows = build(rng, 1, 128, 16, [300], [[9, 40]], spread=3.0)
    x = Pair(c)
    q = 8 * queries(rng, 2, 4, 64)
    for scale in (0.125, 4.0, -1.0, 0.0, 1e-6):
        check(x, 0, q, scale, rows, np.arange(3), [0, 2], [300])


def test_strides_and_no_lse():
    """q as a slice of a wider projection, out inside a wider buffer."""
    rng = np.random.default_rng(12)
    c, rows = build(rng, 1, 128, 16, [70], [[5, 12, 1]])
    x = Pair(c)
    t, H, d = x.t, 4, 64
    wide = gu.to_dev(rng.standard_normal((3, 2 * H * d + 24)).astype(np.float16))
    qd = wide[:, 8:8 + H * d].view(3, H, d)
    buf = t.full((3, 2 * H * d), 9.0, dtype=t.float16, device="cuda")
    out = buf[:, H * d:].view(3, H, d)
    ws = t.empty(x.cg.cg_attention_workspace(x.cache, 3, H, d, 3, 1, 1, 70, 82), dtype=t.uint8, device="cuda")
    x.cg.cg_attention_prefix_async(x.cache, 0, qd, out, 0.125, x.i32(rows), x.i32([0, 1, 2, 3]), x.i32([0, 3]),
                                   x.i32([70]), 1, 70, 82, ws)
    t.cuda.synchronize()
    q = qd.cpu().numpy()
    want = pc.attention(c, 0, q, 0.125, rows, [0, 1, 2, 3], [0, 3], [70])
    compare((0, out.cpu().numpy(), None), want, q)
    assert (buf[:, :H * d] == 9.0).all()
    with pytest.raises(ValueError):
        x.cg.cg_attention_prefix_async(x.cache, 0, qd.float(), out, 0.125, None, x.i32([0, 1]), None, None, 1, 0,
                                       82, ws)
    with pytest.raises(x.cg.CgError):
        x.cg.cg_attention_prefix_async(x.cache, 0, qd, out, 0.125, x.i32(rows), x.i32([0, 1, 2, 3]), x.i32([0, 3]),
                                       x.i32([70]), 1, 70, 82, ws[:16 * ((ws.numel() - 1) // 16)])


def test_streams_and_repeats():
    """The same bits each time, on the default and another stream."""
    rng = np.random.default_rng(13)
    tails = [[30, 1, 500], [2, 64]]
    c, rows = build(rng, 1, 256, 16, [900, 65], tails)
    x = Pair(c)
    q = queries(rng, 5, 8, 64)
    args = (0, q, 0.125, rows, np.arange(6), group_starts_of(tails), [900, 65])
    st, out, lse = check(x, *args)
    side = x.t.cuda.Stream()
    x.t.cuda.synchronize()
    for s in (None, side, None, side):
        st, o, l = gpu_attention(x, *args, stream=s)
        assert st == 0 and gu.same_bits(o, out) and np.array_equal(l, lse)


def test_two_calls_at_once():
    """On two streams, each with its workspace, over one cache."""
    rng = np.random.default_rng(17)
    tails = [[30, 1, 500], [2, 64]]
    c, rows = build(rng, 2, 256, 16, [900, 65], tails)
    x = Pair(c)
    t, cg = x.t, x.cg
    numbers = (5, 8, 64, 5, 2, 1, 900, 1400)
    calls = []
    for layer in (0, 1):
        q = queries(rng, 5, 8, 64)
        calls.append(dict(layer=layer, q=q, qd=gu.to_dev(q), out=gu.to_dev(np.zeros_like(q)),
                          lse=t.zeros((5, 8), dtype=t.float32, device="cuda"), stream=t.cuda.Stream(),
                          ws=t.empty(cg.cg_attention_workspace(x.cache, *numbers), dtype=t.uint8, device="cuda")))
    lists = [x.i32(y) for y in (rows, np.arange(6), group_starts_of(tails), [900, 65])]
    t.cuda.synchronize()
    for _ in range(5):
        for y in calls:
            cg.cg_attention_prefix_async(x.cache, y["layer"], y["qd"], y["out"], 0.125, *lists, *numbers[5:], y["ws"],
                                         lse=y["lse"], stream=y["stream"])
    t.cuda.synchronize()
    for y in calls:
        want = pc.attention(c, y["layer"], y["q"], 0.125, rows, np.arange(6), group_starts_of(tails), [900, 65])
        compare((int(x.status.item()), y["out"].cpu().numpy(), y["lse"].cpu().numpy()), want, y["q"])


def test_most_heads():
    """1,024 query heads of one kv head: more row tiles than one workgroup's."""
    rng = np.random.default_rng(18)
    c, rows = build(rng, 1, 16, 16, [70], [[5, 33]])
    q = queries(rng, 3, 1024, 16)
    check(Pair(c), 0, q, 0.25, rows, [0, 1, 3], [0, 2], [70])


@pytest.mark.parametrize("heads", [1, 64])
def test_longest_row(heads):
    """Rows of 2^30 tokens, all of whose table entries name one page.  Keys are 0, so
    all weights are one power of two and their sums, 2^30 of them in halves of
    halves, are exact; values repeat every 65,536 tokens, small integers whose sums
    are exact too.  A row is full then: a token more is refused."""
    import kv_cache_compression_anchor_amd as cg
    t = gu.torch()
    P, B, d = 65536, 16384, 64
    n = P * B
    k = t.zeros((1, 2, P, d), dtype=t.float16, device="cuda")
    v = t.ones((1, 2, P, d), dtype=t.float16, device="cuda")
    v[0, :, ::4, 1::2] = -3.0  # one token in four: the mean is 0
    tables = t.zeros((2, B), dtype=t.int32, device="cuda")
    lens = t.tensor([n, n], dtype=t.int32, device="cuda")
    refs = t.tensor([B, 0], dtype=t.int32, device="cuda")
    status = t.zeros(1, dtype=t.int32, device="cuda")
    c = cg.PagedCache(k, v, tables, lens, refs, status)
    i32 = lambda y: t.tensor(y, dtype=t.int32, device="cuda")  # noqa: E731
    q = t.randn((2, heads, d), device="cuda").half()
    for groups, prefix in ((None, None), ([0, 2], [n - P])):
        hint = 0 if prefix is None else prefix[0]
        numbers = (2, heads, d, 2, 0 if prefix is None else 1, 1, hint, n)
        ws = t.full((cg.cg_attention_workspace(c, *numbers),), 0xFF, dtype=t.uint8, device="cuda")
        out = t.full((2, heads, d), 9.0, dtype=t.float16, device="cuda")
        lse = t.zeros((2, heads), dtype=t.float32, device="cuda")
        opt = lambda y: None if y is None else i32(y)  # noqa: E731
        cg.cg_attention_prefix_async(c, 0, q, out, 0.125, None, i32([0, 1, 2]), opt(groups), opt(prefix), 1, hint, n,
                                     ws, lse=lse)
        t.cuda.synchronize()
        assert int(status.item()) == 0
        assert (out[..., ::2] == 1).all() and (out[..., 1::2] == 0).all()
        # log 2^30 with log2f's and one product's roundings
        assert ((lse - 30 * np.log(2)).abs() <= 4 * E * 30).all()
    pages = t.empty(cg.cg_pages_workspace(c), dtype=t.uint8, device="cuda")
    slots = t.empty(2, dtype=t.int64, device="cuda")
    lens[1] = n - 1
    cg.cg_pages_reserve_async(c, i32([0, 1]), i32([0, 1, 2]), slots, pages)
    assert slots.tolist() == [-1, P - 1] and lens.tolist() == [n, n] and int(status.item()) == pc.REFUSED


def test_captured_decode_loop():
    """Reserve, write and attend in one graph: every replay is a decoding step,
    compared with the oracle, with eager work between the replays."""
    rng = np.random.default_rng(15)
    tails = [[3, 14, 30]]
    c, rows = build(rng, 2, 128, 16, [100], tails, spare=10)
    x = Pair(c)
    t, cg = x.t, x.cg
    H, d = 4, 64
    r, qs, gs, pl = x.i32(rows), x.i32([0, 1, 2, 3]), x.i32([0, 3]), x.i32([100])
    slots = t.empty(3, dtype=t.int64, device="cuda")
    kd, vd = (t.zeros((2, 3, 128), dtype=t.float16, device="cuda") for _ in range(2))
    qd, out = (t.zeros((3, H, d), dtype=t.float16, device="cuda") for _ in range(2))
    lse = t.zeros((3, H), dtype=t.float32, device="cuda")
    ws = t.empty(cg.cg_attention_workspace(x.cache, 3, H, d, 3, 1, 1, 100, 160), dtype=t.uint8, device="cuda")
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        cg.cg_pages_reserve_async(x.cache, r, qs, slots, x.ws)
        cg.cg_pages_write_async(x.cache, 0, slots, kd, vd)
        cg.cg_attention_prefix_async(x.cache, 1, qd, out, 0.125, r, qs, gs, pl, 1, 100, 160, ws, lse=lse)
    for step in range(8):
        k, v = (rng.standard_normal((2, 3, 128)).astype(np.float16) for _ in range(2))
        q = queries(rng, 3, H, d)
        for dst, src in ((kd, k), (vd, v), (qd, q)):
            dst.copy_(gu.to_dev(src))
        graph.replay()
        t.cuda.synchronize()
        st, want = pc.reserve(c, rows, [0, 1, 2, 3], 3)
        pc.write(c, 0, want, k, v)
        got = (int(x.status.item()), out.cpu().numpy(), lse.cpu().numpy())
        compare(got, pc.attention(c, 1, q, 0.125, rows, [0, 1, 2, 3], [0, 3], [100]), q)
        if step % 3 == 1:  # eager, in between
            check(x, 0, q, 0.125, rows, [0, 1, 2, 3], [0, 3], [100])


def test_pool_past_four_gib():
    import kv_cache_compression_anchor_amd as cg
    t = gu.torch()
    N, P, C = 70000, 32, 1024
    k, v = (t.empty((1, N, P, C), dtype=t.float16, device="cuda") for _ in range(2))
    k[0, N - 6:], v[0, N - 6:] = t.randn((6, P, C), device="cuda").half(), t.randn((6, P, C), device="cuda").half()
    tables = t.full((2, 6), -1, dtype=t.int32, device="cuda")
    tables[0], tables[1] = t.arange(N - 6, N), t.arange(N - 6, N)
    lens = t.tensor([180, 170], dtype=t.int32, device="cuda")
    refs, status = t.ones(N, dtype=t.int32, device="cuda"), t.zeros(1, dtype=t.int32, device="cuda")
    cache = cg.PagedCache(k, v, tables, lens, refs, status)
    host = pc.Cache(k[:, N - 6:].cpu().numpy(), v[:, N - 6:].cpu().numpy(),
                    np.tile(np.arange(6, dtype=np.int32), (2, 1)), lens.cpu().numpy(), np.ones(6, np.int32))
    q = queries(np.random.default_rng(16), 2, 8, 128)
    ws = t.empty(cg.cg_attention_workspace(cache, 2, 8, 128, 2, 1, 1, 100, 180), dtype=t.uint8, device="cuda")
    out, lse = gu.to_dev(np.zeros_like(q)), t.zeros((2, 8), dtype=t.float32, device="cuda")
    i32 = lambda x: t.tensor(x, dtype=t.int32, device="cuda")  # noqa: E731
    cg.cg_attention_prefix_async(cache, 0, gu.to_dev(q), out, 0.088, None, i32([0, 1, 2]), i32([0, 2]), i32([100]),
                                 1, 100, 180, ws, lse=lse)
    t.cuda.synchronize()
    want = pc.attention(host, 0, q, 0.088, None, [0, 1, 2], [0, 2], [100])
    compare((int(status.item()), out.cpu().numpy(), lse.cpu().numpy()), want, q)
