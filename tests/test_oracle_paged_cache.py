"""What pins the paged-cache oracle: closed forms of the attention, and a model
of a cache as plain token lists that every sequence of page operations must
agree with."""
import numpy as np
import pytest

from oracle import paged_cache as pc


def new(c, rng, rows, counts, layers):
    """Reserve and write random tokens; returns (status, slots, k, v)."""
    starts = np.concatenate([[0], np.cumsum(counts)])
    st, slots = pc.reserve(c, rows, starts, int(starts[-1]))
    k = rng.standard_normal((layers, int(starts[-1]), c.k.shape[3])).astype(np.float16)
    v = rng.standard_normal(k.shape).astype(np.float16)
    return st | pc.write(c, 0, slots, k, v), starts, slots, k, v


def seen(c, pool, r):
    """Row r's tokens as [layers, n, C], through its table."""
    n = int(c.lens[r])
    t = np.arange(n)
    return pool[:, c.tables[r, t // c.P], t % c.P]


def check_invariants(c):
    count = np.zeros(c.N, int)
    for r, n in enumerate(c.lens):
        nb = pc.blocks(c, n)
        assert (c.tables[r, nb:] == -1).all()
        assert ((c.tables[r, :nb] >= 0) & (c.tables[r, :nb] < c.N)).all()
        np.add.at(count, c.tables[r, :nb], 1)
        if n % c.P:
            assert c.refs[c.tables[r, nb - 1]] == 1
    assert (count == c.refs).all()


@pytest.mark.parametrize("P,seed", [(1, 0), (4, 1), (8, 2), (64, 3)])
def test_random_sequences_agree_with_token_lists(P, seed):
    rng = np.random.default_rng(seed)
    R, L = 9, 2
    c = pc.empty(L, 400 // P + 12, P, 3, R, 200 // P + 2)
    model = {r: np.zeros((2, L, 0, 3), np.float16) for r in range(R)}
    for _ in range(120):
        kind = rng.integers(4)
        if kind == 0:
            rows = rng.permutation(R)[:rng.integers(1, 4)]
            counts = rng.integers(0, 20, len(rows))
            before = c.lens.copy()
            st, starts, slots, k, v = new(c, rng, rows, counts, L)
            for i, r in enumerate(rows):
                mine = slice(starts[i], starts[i + 1])
                if c.lens[r] != before[r] + counts[i]:
                    assert st & (pc.NO_PAGES | pc.REFUSED) and (slots[mine] == -1).all()
                    continue
                model[r] = np.concatenate([model[r], np.stack([k[:, mine], v[:, mine]])], 2)
        elif kind == 1:
            a, b = rng.integers(R), rng.permutation(R)[:2]
            before = c.lens.copy()
            pc.fork(c, [a] * 2, b)
            for x in b:
                if before[x] == 0 and x != a and c.lens[x]:  # not refused, not left out
                    model[x] = model[a].copy()
        elif kind == 2:
            for r in (rows := rng.permutation(R)[:2]):
                model[r] = model[r][:, :, :0]
            pc.free(c, rows)
        else:
            st, live = pc.compact(c)
            assert st == 0 and (c.refs[:live] > 0).all() and (c.refs[live:] == 0).all()
        check_invariants(c)
        for r in range(R):
            assert c.lens[r] == model[r].shape[2]
            assert np.array_equal(seen(c, c.k, r), model[r][0]) and np.array_equal(seen(c, c.v, r), model[r][1])


def test_refusals_leave_the_cache_alone():
    c = pc.empty(1, 6, 4, 2, 4, 3)
    rng = np.random.default_rng(0)
    assert new(c, rng, [0], [9], 1)[0] == 0
    before = c.copy()
    assert pc.reserve(c, [1, 1], [0, 2, 4], 4)[0] == pc.REFUSED          # the same row twice
    assert pc.reserve(c, [7], [0, 2], 2)[0] == pc.REFUSED
    assert pc.reserve(c, [0], [0, 4], 4)[0] == pc.REFUSED                # 13 tokens need four blocks
    assert pc.reserve(c, [1, 2], [0, 0, 12], 11)[0] == pc.REFUSED
    assert pc.fork(c, [0, 0], [1, 1]) == pc.REFUSED
    assert pc.fork(c, [0], [0]) == pc.REFUSED
    assert pc.copy(c, [0, 1], [4, 4]) == pc.REFUSED
    assert pc.copy(c, [0, 4], [4, 4]) == pc.REFUSED
    assert pc.copy(c, [0], [6]) == pc.BAD_PAGE
    for a, b in zip(dataclass_arrays(before), dataclass_arrays(c)):
        assert a.tobytes() == b.tobytes()
    # four of the pages: the first request fits, the second does not, the third needs none
    st, slots = pc.reserve(c, [1, 2, 3], [0, 8, 16, 16], 16)
    assert st == pc.NO_PAGES and c.lens.tolist() == [9, 8, 0, 0] and (slots[8:] == -1).all()


def dataclass_arrays(c):
    return [c.k, c.v, c.tables, c.lens, c.refs]


def one(c, q, scale=1.0, **kw):
    n = kw.pop("n", 1)
    st, got = pc.attention(c, 0, q, scale, kw.pop("rows", None), kw.pop("q_starts", [0, n]), **kw)
    return st, got


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    c = pc.empty(1, 20, 4, 16, 3, 8)
    new(c, rng, [0], [1], 1)
    q = rng.standard_normal((1, 4, 8)).astype(np.float16)  # 4 heads on 2 kv heads
    st, got = one(c, q)
    v0 = seen(c, c.v, 0)[0, 0].astype(np.float64).reshape(2, 8)
    for h in range(4):  # one token: its value, whatever the score
        assert st == 0 and np.allclose(got[0][h]["out"], v0[h // 2], atol=0, rtol=1e-15)
    # equal scores: the mean; lse = log n
    new(c, rng, [1], [13], 1)
    st, got = one(c, np.zeros((1, 4, 8), np.float16), rows=[1])
    mean = seen(c, c.v, 1)[0].astype(np.float64).mean(0).reshape(2, 8)
    for h in range(4):
        assert np.allclose(got[0][h]["out"], mean[h // 2], rtol=1e-12)
        assert np.isclose(got[0][h]["lse"], np.log(13))
    # several queries: the j-th sees one token more; more queries than tokens: the first see none
    st, got = one(c, np.zeros((14, 4, 8), np.float16), rows=[1], n=14)
    assert got[0][0]["lse"] == -np.inf and (got[0][0]["out"] == 0).all()
    assert all(np.isclose(got[j][0]["lse"], np.log(j)) for j in range(1, 14))


def test_prefix_groups_change_nothing_for_forks():
    rng = np.random.default_rng(2)
    c = pc.empty(1, 40, 4, 16, 4, 12)
    new(c, rng, [0], [10], 1)
    assert pc.fork(c, [0, 0], [1, 2]) == 0
    new(c, rng, [0, 1, 2], [3, 1, 7], 1)
    q = rng.standard_normal((4, 2, 8)).astype(np.float16)
    kw = dict(rows=[0, 1, 2], q_starts=[0, 2, 3, 4])
    _, a = one(c, q, **kw)
    st, b = one(c, q, group_starts=[0, 3], prefix_lens=[10], **kw)
    assert st == 0
    for j in a:
        for h in range(2):
            assert np.array_equal(a[j][h]["out"], b[j][h]["out"]) and a[j][h]["lse"] == b[j][h]["lse"]
    # a prefix that reaches into a sequence's queries is refused for that sequence alone
    st, b = one(c, q, group_starts=[0, 3], prefix_lens=[11], **kw)
    assert st == pc.REFUSED and b[2][0]["lse"] == -np.inf and np.isfinite(b[0][0]["lse"])
