"""GPU parity of the page operators with the oracle: the whole state (tables,
lengths, counts, slots, every pool byte) equal after each call, for page and
channel sizes that take each copy width, repeated and bad requests, empty and
full caches, exhausted pools, strided new tokens, another stream and a captured
graph."""
import numpy as np
import pytest

from oracle import paged_cache as pc
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


class Pair:
    """The same cache on the device and in the oracle."""

    def __init__(self, host):
        import kv_cache_compression_anchor_amd as cg
        t = gu.torch()
        self.cg, self.t, self.o = cg, t, host
        self.k, self.v = gu.to_dev(host.k), gu.to_dev(host.v)
        self.tables, self.lens, self.refs = (gu.to_dev(x) for x in (host.tables, host.lens, host.refs))
        self.status = t.zeros(1, dtype=t.int32, device="cuda")
        self.cache = cg.PagedCache(self.k, self.v, self.tables, self.lens, self.refs, self.status)
        self.ws = t.full((cg.cg_pages_workspace(self.cache),), 0xA5, dtype=t.uint8, device="cuda")

    def i32(self, x):
        return gu.to_dev(np.asarray(x, np.int32))

    def check(self, status, what):
        self.t.cuda.synchronize()
        assert int(self.status.item()) == status, (what, int(self.status.item()), status)
        self.status.zero_()
        for name in ("tables", "lens", "refs"):
            assert np.array_equal(getattr(self, name).cpu().numpy(), getattr(self.o, name)), (what, name)
        assert gu.same_bits(self.k.cpu().numpy(), self.o.k), (what, "k")
        assert gu.same_bits(self.v.cpu().numpy(), self.o.v), (what, "v")

    def reserve(self, rows, starts, n_tokens, what="reserve"):
        slots = self.t.full((n_tokens,), 77, dtype=self.t.int64, device="cuda")
        self.cg.cg_pages_reserve_async(self.cache, self.i32(rows), self.i32(starts), slots, self.ws)
        st, want = pc.reserve(self.o, rows, starts, n_tokens)
        self.check(st, what)
        assert np.array_equal(slots.cpu().numpy(), want), what
        return slots, want

    def write(self, layer0, slots, want, k, v, what="write"):
        self.cg.cg_pages_write_async(self.cache, layer0, slots, gu.to_dev(k), gu.to_dev(v))
        self.check(pc.write(self.o, layer0, want, k, v), what)

    def new(self, rng, rows, counts):
        starts = np.concatenate([[0], np.cumsum(counts)])
        slots, want = self.reserve(rows, starts, int(starts[-1]))
        L, n, C = self.o.k.shape[0], int(starts[-1]), self.o.k.shape[3]
        k, v = (rng.standard_normal((L, n, C)).astype(np.float16) for _ in range(2))
        self.write(0, slots, want, k, v)

    def fork(self, parents, children, what="fork"):
        self.cg.cg_pages_fork_async(self.cache, self.i32(parents), self.i32(children), self.ws)
        self.check(pc.fork(self.o, parents, children), what)

    def free(self, rows, what="free"):
        self.cg.cg_pages_free_async(self.cache, self.i32(rows))
        self.check(pc.free(self.o, rows), what)

    def copy(self, src, dst, what="copy"):
        self.cg.cg_pages_copy_async(self.cache, self.i32(src), self.i32(dst))
        self.check(pc.copy(self.o, src, dst), what)

    def compact(self, what="compact"):
        live = self.t.full((1,), -5, dtype=self.t.int32, device="cuda")
        self.cg.cg_pages_compact_async(self.cache, self.ws, live)
        st, want = pc.compact(self.o)
        self.check(st, what)
        assert int(live.item()) == want


def randomised(c, rng):
    """Pool contents that no two pages share."""
    for x in (c.k, c.v):
        x[:] = rng.integers(0, 1 << 16, x.shape, dtype=np.uint16).view(np.float16)
    return c


# channels 128 and 1000: 16-byte units; 138: 4-byte rows; 65: 2-byte rows
@pytest.mark.parametrize("P,C", [(1, 128), (1, 65), (4, 138), (16, 128), (16, 65), (64, 1000)])
def test_random_sequences(P, C):
    rng = np.random.default_rng(P * 1000 + C)
    R, L = 11, 3
    c = randomised(pc.empty(L, 500 // P + 14, P, C, R, 250 // P + 2), rng)
    x = Pair(c)
    for step in range(60):
        kind = rng.integers(5)
        if kind == 0 or step < 3:
            rows = rng.permutation(R)[:rng.integers(1, 6)]
            x.new(rng, rows, rng.integers(0, 24, len(rows)))
        elif kind == 1:
            n = rng.integers(1, 5)
            x.fork(rng.integers(0, R, n), rng.permutation(R)[:n])
        elif kind == 2:
            x.free(rng.permutation(R)[:rng.integers(1, 4)])
        elif kind == 3:
            x.compact()
        else:  # contents only, free pages or not
            n = rng.integers(1, c.N // 2)
            pages = rng.permutation(c.N)
            x.copy(pages[:n], pages[n:2 * n])


def test_repeated_and_bad_requests():
    rng = np.random.default_rng(5)
    x = Pair(randomised(pc.empty(2, 40, 4, 64, 8, 6), rng))
    x.new(rng, [0, 1, 2], [5, 8, 24])
    x.reserve([3, 3, 0], [0, 2, 4, 7], 7, "a row twice")
    x.reserve([-1, 8, 1 << 30, 4], [0, 1, 2, 3, 4], 4, "rows out of range")
    x.reserve([2, 3], [0, 1, 2], 2, "a full row")
    x.reserve([3, 4], [0, 3, 2], 3, "starts that descend")
    x.reserve([3, 4], [0, 3, 9], 8, "starts past the tokens")
    x.reserve([5, 6], [2, 4, 4], 6, "tokens of no request")
    x.fork([0, 1, 0], [3, 3, 6], "a child twice, and one that holds tokens")
    x.fork([0, 3], [7, 0], "a child that is a parent")
    x.fork([-1, 0, 9], [7, 8, 7], "rows out of range")
    x.free([1, 1, -3, 8, 7], "twice, out of range, empty")
    x.copy([0, 1, 2, 3], [30, 30, 31, 2], "a dst twice, a src that is a dst")
    x.copy([0, -1, 40, 5], [32, 33, 34, 40], "pages out of range")
    x.copy([5], [5], "a page onto itself")
    x.compact()


def test_exhausted_pool():
    rng = np.random.default_rng(6)
    x = Pair(randomised(pc.empty(1, 10, 4, 64, 9, 6), rng))
    x.new(rng, [0, 1, 2, 3], [10, 9, 17, 0])   # 3 + 3 pages; 5 do not fit; none needed
    x.fork([0, 1, 0, 1, 0], [4, 5, 6, 7, 8])   # four partly filled pages, then none
    x.reserve([0, 1], [0, 1, 2], 2, "room in the last pages")
    x.free([0])
    x.free([4, 5])
    x.compact()
    x.new(rng, [0], [9])


def test_garbage_state_is_bounded():
    """Entries, lengths and counts that no call leaves behind: flagged, in bounds."""
    rng = np.random.default_rng(7)
    x = Pair(randomised(pc.empty(1, 30, 4, 64, 6, 5), rng))
    x.new(rng, [0, 1, 2, 3], [10, 9, 17, 6])
    x.o.tables[0, 1], x.o.tables[1, 2], x.o.tables[2, 0] = 30, -7, 1 << 30
    x.o.lens[3], x.o.lens[4] = 21, -1
    x.tables.copy_(gu.to_dev(x.o.tables))
    x.lens.copy_(gu.to_dev(x.o.lens))
    x.reserve([1, 3, 4], [0, 2, 3, 4], 4, "reserve")
    x.fork([0, 1, 3, 4], [5, 5, 5, 5], "children repeated")
    x.fork([1], [5], "a last page outside the pool")
    x.fork([2], [5], "a full page outside the pool")
    x.compact()
    x.free([0, 1, 2, 3, 4, 5], "free")
    x.o.refs[5], x.o.refs[29] = -3, 4
    x.refs.copy_(gu.to_dev(x.o.refs))
    # a negative count is neither free nor in use: fewer free pages than moves
    x.o.refs[:5] = -1
    x.refs.copy_(gu.to_dev(x.o.refs))
    x.t.cuda.synchronize()
    live = x.t.zeros(1, dtype=x.t.int32, device="cuda")
    x.cg.cg_pages_compact_async(x.cache, x.ws, live)
    x.t.cuda.synchronize()
    assert int(x.status.item()) == pc.REFUSED and int(live.item()) == (x.o.refs > 0).sum()


def test_nothing_to_do():
    x = Pair(pc.empty(1, 4, 4, 64, 3, 4))
    for call in (lambda: x.reserve([], [0], 0), lambda: x.fork([], []), lambda: x.free([]),
                 lambda: x.copy([], []), x.compact):
        call()
    # tokens but no request: every slot is -1
    x.reserve([], [0], 5)
    # no slots wanted
    x.cg.cg_pages_reserve_async(x.cache, x.i32([1]), x.i32([0, 6]), None, x.ws, n_tokens=6)
    x.check(pc.reserve(x.o, [1], [0, 6], 6)[0], "no slots")


def test_many_rows_and_pages():
    """More requests than a workgroup has threads, more pages than one scan step."""
    rng = np.random.default_rng(8)
    R = 2500
    x = Pair(randomised(pc.empty(1, 40000, 2, 8, 2 * R, 40), rng))
    x.new(rng, rng.permutation(R), rng.integers(0, 21, R))
    x.fork(rng.integers(0, R, R), R + rng.permutation(R))
    x.free(rng.permutation(2 * R)[:R + 77])
    x.compact()
    x.copy(*np.split(rng.permutation(40000)[:6000], 2))
    # the highest pages in use: moves from past the first scan steps
    x.o.refs[39990:] = 1
    x.refs.copy_(gu.to_dev(x.o.refs))
    x.compact()


def test_more_bad_requests_than_threads():
    """Repeated, invalid and refused requests, and a pool that ends, among 1,500."""
    rng = np.random.default_rng(13)
    R, n = 3000, 1500
    x = Pair(randomised(pc.empty(1, 3700, 2, 8, R, 6), rng))
    odd = [-1, R, 1 << 30, -(1 << 31), (1 << 31) - 1]

    def rows_of(count, least=0):
        rows = least + rng.permutation(R - least)[:count].astype(np.int64)
        rows[rng.random(count) < 0.02] = rng.choice(odd)
        again = rng.random(count) < 0.02
        rows[again] = rows[rng.integers(0, count, int(again.sum()))]
        return rows

    for step in range(3):
        counts = rng.integers(0, 5, n)
        starts = np.concatenate([[0], np.cumsum(counts)])
        x.reserve(rows_of(n), starts, int(starts[-1]) + step, ("reserve", step))
        x.fork(rng.choice(np.concatenate([np.arange(R // 2), odd]), n), rows_of(n, R // 2), ("fork", step))
        full = (x.o.refs > 0).all()
        x.free(rows_of(400), ("free", step))
        x.compact(("compact", step))
    assert full


@pytest.mark.parametrize("n", [7, 1100])
def test_extreme_numbers_stay_in_bounds(n):
    """Rows, lengths, entries, counts and starts at both ends of the type: flagged, and
    pools whose pages no valid number names keep their contents."""
    rng = np.random.default_rng(n)
    lo, hi = -(1 << 31), (1 << 31) - 1
    ends = np.array([lo, lo + 1, -1, hi, hi - 1, 1 << 30, -(1 << 30)])
    x = Pair(randomised(pc.empty(1, 40, 4, 64, 1200, 5), rng))
    cg, c, t = x.cg, x.cache, x.t
    slots = t.zeros(50, dtype=t.int64, device="cuda")
    mixed = lambda size, top: np.where(rng.random(size) < 0.7, rng.choice(ends, size),  # noqa: E731
                                       rng.integers(0, top, size))
    for _ in range(20):
        x.tables.copy_(x.i32(mixed(x.tables.shape, 44)))
        x.lens.copy_(x.i32(mixed(1200, 22)))
        x.refs.copy_(x.i32(mixed(40, 3)))
        cg.cg_pages_reserve_async(c, x.i32(mixed(n, 1200)), x.i32(mixed(n + 1, 52)), slots, x.ws)
        cg.cg_pages_fork_async(c, x.i32(mixed(n, 1200)), x.i32(mixed(n, 1200)), x.ws)
        cg.cg_pages_free_async(c, x.i32(mixed(n, 1200)))
        cg.cg_pages_compact_async(c, x.ws)
        m = min(n, 40)
        cg.cg_pages_copy_async(c, x.i32(mixed(m, 44)), x.i32(mixed(m, 44)))
        t.cuda.synchronize()
        assert int(x.status.item()) & ~14 == 0 and int(x.status.item())
    far = t.tensor([lo, hi, -(1 << 63), (1 << 63) - 1, 160, -2], dtype=t.int64, device="cuda")
    k, v = x.k.clone(), x.v.clone()
    new = t.ones((1, 6, 64), dtype=t.float16, device="cuda")
    x.status.zero_()
    cg.cg_pages_write_async(c, 0, far, new, new)
    assert int(x.status.item()) == pc.BAD_PAGE
    assert t.equal(k.view(t.int16), x.k.view(t.int16)) and t.equal(v.view(t.int16), x.v.view(t.int16))


def test_write_layers_and_strides():
    """Layer ranges, K and V as slices of a wider projection, slots outside the pool."""
    rng = np.random.default_rng(9)
    t = gu.torch()
    for C in (64, 65):
        x = Pair(randomised(pc.empty(4, 20, 8, C, 2, 10), rng))
        slots, want = x.reserve([1, 0], [0, 33, 40], 40)
        both = rng.standard_normal((2, 40, 3 * C + 5)).astype(np.float16)
        dev = gu.to_dev(both)
        k, v = both[:, :, C:2 * C], both[:, :, 2 * C:3 * C]
        x.cg.cg_pages_write_async(x.cache, 1, slots, dev[:, :, C:2 * C], dev[:, :, 2 * C:3 * C])
        x.check(pc.write(x.o, 1, want, k, v), "slices")
        one = rng.standard_normal((1, 40, C)).astype(np.float16)
        x.write(3, slots, want, one, -one)
        bad = want.copy()
        bad[3], bad[9], bad[17], bad[20] = -1, -2, 160, 1 << 40
        x.write(0, t.from_numpy(bad).cuda(), bad, one, -one)
        # a single token
        x.write(2, slots[5:6], want[5:6], one[:, :1], -one[:, :1])


def test_reserve_without_slots():
    rng = np.random.default_rng(12)
    x = Pair(randomised(pc.empty(1, 30, 4, 64, 5, 6), rng))
    for rows, starts in (([3, 1], [0, 9, 14]), ([0], [2, 5]), ([3, 4], [0, 15, 16])):
        x.cg.cg_pages_reserve_async(x.cache, x.i32(rows), x.i32(starts), None, x.ws, n_tokens=16)
        x.check(pc.reserve(x.o, rows, starts, 16)[0], rows)


# channels 64 and 8: 16-byte units; 138: 4; 65: 2.  4,096 pairs are the most of the simpler kernel
@pytest.mark.parametrize("n,N,P,C,L", [(4096, 9000, 4, 64, 2), (4097, 9000, 4, 64, 2), (5000, 12000, 1, 65, 3),
                                       (12295, 30000, 8, 138, 1), (6000, 12100, 16, 1024, 3),
                                       (1 << 20, 1 << 21, 1, 8, 1), (1 << 23, 1 << 24, 1, 8, 1)])
def test_copies_of_many_pairs(n, N, P, C, L):
    """Among them pairs with one dst, with the dst of another as src, onto themselves and
    out of range; in a time that does not grow with the square of their number."""
    import kv_cache_compression_anchor_amd as cg
    t = gu.torch()
    g = t.Generator(device="cuda").manual_seed(n + C)
    pools = [t.randint(-(1 << 15), 1 << 15, (L, N, P, C), generator=g, device="cuda", dtype=t.int16).view(t.float16)
             for _ in range(2)]
    before = [p.clone() for p in pools]
    status = t.zeros(1, dtype=t.int32, device="cuda")
    meta = t.full((1, 1), -1, dtype=t.int32, device="cuda")
    cache = cg.PagedCache(*pools, meta, t.zeros(1, dtype=t.int32, device="cuda"),
                          t.ones(N, dtype=t.int32, device="cuda"), status)
    order = t.randperm(N, generator=g, device="cuda").int()
    some = lambda share: t.nonzero(t.rand(n, generator=g, device="cuda") < share).flatten()  # noqa: E731
    for kinds in ((), ("dst twice",), ("a dst as src",), ("itself",), ("out of range",),
                  ("dst twice", "a dst as src", "itself", "out of range")):
        src, dst = order[:n].clone(), order[N - n:].clone()  # they overlap where N < 2 n
        for kind in kinds:
            at = some(0.02)
            other = t.randint(0, n, at.shape, generator=g, device="cuda")
            if kind == "dst twice":
                dst[at] = dst[other]
            elif kind == "a dst as src":
                src[at] = dst[other]
            elif kind == "itself":
                src[at] = dst[at]
            else:
                bad = t.tensor([-1, N, 1 << 30, -(1 << 31), (1 << 31) - 1], dtype=t.int32, device="cuda")
                src[at[::2]] = bad[other[::2] % 5]
                dst[at[1::3]] = bad[other[1::3] % 5]
        inside = (src >= 0) & (src < N) & (dst >= 0) & (dst < N)
        named = t.bincount(dst[(dst >= 0) & (dst < N)].long(), minlength=N)
        clash = (named[src.clamp(0, N - 1).long()] > 0) | (named[dst.clamp(0, N - 1).long()] > 1)
        want = (pc.BAD_PAGE if not bool(inside.all()) else 0) | (pc.REFUSED if bool((inside & clash).any()) else 0)
        for p, q in zip(pools, before):
            p.copy_(q)
        ev = [t.cuda.Event(enable_timing=True) for _ in range(2)]
        ev[0].record()
        cg.cg_pages_copy_async(cache, src, dst)
        ev[1].record()
        t.cuda.synchronize()
        assert ev[0].elapsed_time(ev[1]) < 1000, (n, kinds)
        assert int(status.item()) == want, kinds
        status.zero_()
        go = inside & ~clash
        assert kinds or bool(go.any())
        for p, q in zip(pools, before):
            q = q.view(t.int16).clone()
            q[:, dst[go].long()] = q[:, src[go].long()]
            assert t.equal(p.view(t.int16), q), kinds


def test_another_stream():
    rng = np.random.default_rng(10)
    x = Pair(randomised(pc.empty(2, 64, 4, 64, 6, 12), rng))
    side = x.t.cuda.Stream()
    k, v = (rng.standard_normal((2, 20, 64)).astype(np.float16) for _ in range(2))
    kd, vd, slots = gu.to_dev(k), gu.to_dev(v), x.t.empty(20, dtype=x.t.int64, device="cuda")
    lists = [x.i32(y) for y in ([0, 1], [0, 13, 20], [0, 1], [2, 3], [0, 1])]
    x.t.cuda.synchronize()
    cg, c = x.cg, x.cache
    cg.cg_pages_reserve_async(c, lists[0], lists[1], slots, x.ws, stream=side)
    cg.cg_pages_write_async(c, 0, slots, kd, vd, stream=side)
    cg.cg_pages_fork_async(c, lists[2], lists[3], x.ws, stream=side)
    cg.cg_pages_free_async(c, lists[4], stream=side)
    cg.cg_pages_compact_async(c, x.ws, stream=side)
    side.synchronize()
    st, want = pc.reserve(x.o, [0, 1], [0, 13, 20], 20)
    st |= pc.write(x.o, 0, want, k, v) | pc.fork(x.o, [0, 1], [2, 3]) | pc.free(x.o, [0, 1])
    st |= pc.compact(x.o)[0]
    x.check(st, "side stream")


def test_captured_step():
    """A decoding step in a graph: each replay adds a token to every row, with eager
    calls and synchronisations between the replays."""
    rng = np.random.default_rng(11)
    x = Pair(randomised(pc.empty(2, 64, 4, 64, 5, 12), rng))
    x.new(rng, [0, 2, 4], [3, 4, 9])
    t, cg, c = x.t, x.cg, x.cache
    rows, starts = x.i32([4, 0, 2]), x.i32([0, 1, 2, 3])
    slots = t.empty(3, dtype=t.int64, device="cuda")
    kd, vd = t.zeros((2, 3, 64), dtype=t.float16, device="cuda"), t.zeros((2, 3, 64), dtype=t.float16, device="cuda")
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        cg.cg_pages_reserve_async(c, rows, starts, slots, x.ws)
        cg.cg_pages_write_async(c, 0, slots, kd, vd)
    for step in range(6):
        k, v = (rng.standard_normal((2, 3, 64)).astype(np.float16) for _ in range(2))
        kd.copy_(gu.to_dev(k))
        vd.copy_(gu.to_dev(v))
        graph.replay()
        st, want = pc.reserve(x.o, [4, 0, 2], [0, 1, 2, 3], 3)
        st |= pc.write(x.o, 0, want, k, v)
        x.check(st, ("replay", step))
        assert np.array_equal(slots.cpu().numpy(), want)
        if step == 2:
            x.fork([0], [1])
        if step == 3:
            x.free([2])
            x.compact()


def test_pool_past_four_gib():
    """Offsets past 32 bits inside one layer's pool."""
    import kv_cache_compression_anchor_amd as cg
    t = gu.torch()
    N, P, C = 70000, 32, 1024
    k, v = (t.empty((1, N, P, C), dtype=t.float16, device="cuda") for _ in range(2))
    tables, lens = (t.full((3, 8), -1, dtype=t.int32, device="cuda"),
                    t.zeros(3, dtype=t.int32, device="cuda"))
    refs = t.ones(N, dtype=t.int32, device="cuda")
    refs[N - 6:] = 0
    status = t.zeros(1, dtype=t.int32, device="cuda")
    c = cg.PagedCache(k, v, tables, lens, refs, status)
    ws = t.empty(cg.cg_pages_workspace(c), dtype=t.uint8, device="cuda")
    new = t.randn((1, 100, C), device="cuda").half()
    slots = t.empty(100, dtype=t.int64, device="cuda")
    i32 = lambda x: t.tensor(x, dtype=t.int32, device="cuda")  # noqa: E731
    cg.cg_pages_reserve_async(c, i32([0]), i32([0, 100]), slots, ws)
    cg.cg_pages_write_async(c, 0, slots, new, -new)
    assert tables[0, :4].tolist() == [N - 6, N - 5, N - 4, N - 3]
    assert slots.tolist() == [(N - 6) * P + i for i in range(100)]
    assert t.equal(k[0, N - 6:N - 2].reshape(-1, C)[:100], new[0])
    cg.cg_pages_fork_async(c, i32([0]), i32([1]), ws)
    assert tables[1, :4].tolist() == [N - 6, N - 5, N - 4, N - 2]
    assert t.equal(v[0, N - 2, :4], -new[0, 96:])
    cg.cg_pages_copy_async(c, i32([N - 6]), i32([3]))
    assert t.equal(k[0, 3], new[0, :32])
    refs[7] = 0
    cg.cg_pages_compact_async(c, ws)
    assert tables[0, :4].tolist() == [N - 6, N - 5, N - 4, N - 3] and tables[1, 3].item() == 7
    assert t.equal(v[0, 7, :4], -new[0, 96:]) and int(refs[7]) == 1 and int(refs[N - 2]) == 0
    assert int(status.item()) == 0


def test_binding_refuses_wrong_tensors():
    x = Pair(pc.empty(1, 8, 4, 64, 3, 4))
    cg, t, c = x.cg, x.t, x.cache
    i64 = t.zeros(2, dtype=t.int64, device="cuda")
    ok = x.i32([0, 1])
    for call in (lambda: cg.PagedCache(x.k, x.v[:, :4], x.tables, x.lens, x.refs, x.status),
                 lambda: cg.PagedCache(x.k, x.v, x.tables, x.lens[:2], x.refs, x.status),
                 lambda: cg.PagedCache(x.k, x.v, x.tables, x.lens, x.refs[:4], x.status),
                 lambda: cg.PagedCache(x.k.cpu(), x.v, x.tables, x.lens, x.refs, x.status),
                 lambda: cg.PagedCache(x.k.float(), x.v.float(), x.tables, x.lens, x.refs, x.status),
                 lambda: cg.cg_pages_copy_async(c, i64, i64),
                 lambda: cg.cg_pages_copy_async(c, ok, ok[:1]),
                 lambda: cg.cg_pages_copy_async(c, ok.cpu(), ok.cpu()),
                 lambda: cg.cg_pages_reserve_async(c, ok, ok, i64, x.ws),
                 lambda: cg.cg_pages_fork_async(c, ok, ok[:1], x.ws),
                 lambda: cg.cg_pages_write_async(c, 0, i64, x.k[0, 0, :2], x.k[0, 0, :2])):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(cg.CgError):
        cg.cg_pages_fork_async(c, ok, ok, x.ws[:64])
