"""Measured cases of the operators of a paged cache held in 4 bits: the plain forms
in elementary torch operations (32 bits, rounded once) and the framework's own calls.

A row of the cache is a token's K (or V) of one layer.  A head of `dim` channels
takes 16 ceil(dim / 32) bytes of codes, 8 channels a little-endian word (channel e of
the 8 at bit 16 (e % 2) + 4 (e // 2)), padded to whole groups of 32 channels; behind
all heads' codes stand their binary16 scales, one a group; the row is padded to 16
bytes.  With a the group's largest magnitude, its scale s is the smallest binary16 of
at most 8 significant bits that is not below a / 7 (at most 9344), the code of x is
floor(x / s + 1/2) + 8, and a code n stands for s (n - 8), which binary16 holds
exactly.  The operators: writing tokens (with the values that they are held as),
reading them back, and attention over such a cache.
"""
import random

import torch

own = False

# Shapes named here come from the repository's workloads: tiny (2 layers, 128
# channels), Llama-7B (32 layers, 4096 channels, 32 heads), Mistral-7B (32
# layers, 1024 channels = 8 heads of 128, 9216 tokens), Llama-34B (1024
# channels, 81920 tokens).


def listed():
    return [
        # one decoding step of four answers, a small model: the latency of a call
        dict(name="write_tiny_4", op="write", layers=2, kv_heads=2, dim=64, page=16, rows=4, most=1, longest=90,
             wide=0, shape=1),
        # one decoding step of 64 requests, every layer
        dict(name="write_step_64", op="write", layers=32, kv_heads=8, dim=128, page=16, rows=64, most=1,
             longest=2000, wide=0, shape=2),
        # K and V as slices of one projection, heads that are no whole number of groups
        dict(name="write_odd_333", op="write", layers=3, kv_heads=5, dim=80, page=8, rows=7, most=90, longest=50,
             wide=6, shape=3),
        # ragged prompts of 16 requests
        dict(name="write_prompts_16", op="write", layers=32, kv_heads=8, dim=128, page=16, rows=16, most=700,
             longest=300, wide=0, shape=4),
        # parts of a few short rows, heads of 80
        dict(name="read_odd_3", op="read", layers=3, kv_heads=5, dim=80, page=8, rows=3, longest=130, shape=5),
        # a context on its way back to the codec
        dict(name="read_mistral_9k", op="read", layers=32, kv_heads=8, dim=128, page=16, rows=1, longest=9216,
             shape=6),
        # two answers on a short context: the latency of a call
        dict(name="attn_tiny_2", op="attn", kv_heads=2, group=1, dim=64, page=16, groups=0, per_group=2, prefix=0,
             least=1, longest=64, most_q=1, pad=0, shape=7),
        # odd heads, pages smaller than a tile, drafts, a padded batch
        dict(name="attn_odd_9", op="attn", kv_heads=5, group=7, dim=80, page=4, groups=0, per_group=9, prefix=0,
             least=1, longest=700, most_q=4, pad=3, shape=8),
        # 64 requests, one new token each, each with a context of its own of up to 9K
        dict(name="attn_mistral_64", op="attn", kv_heads=8, group=4, dim=128, page=16, groups=0, per_group=64,
             prefix=0, least=1000, longest=9216, most_q=1, pad=0, shape=9),
        # 64 requests on one shared 9K context and up to 600 tokens of their own
        dict(name="attn_shared_64", op="attn", kv_heads=8, group=4, dim=128, page=16, groups=1, per_group=64,
             prefix=9216, least=1, longest=600, most_q=1, pad=0, shape=10),
        # three system prompts, ragged drafts of 0 to 5 tokens, Llama-7B heads, a padded batch
        dict(name="attn_llama7b_drafts", op="attn", kv_heads=32, group=1, dim=128, page=64, groups=3, per_group=7,
             prefix=1536, least=5, longest=333, most_q=5, pad=3, shape=11),
        # four requests, each with an 80K context of its own
        dict(name="attn_long_4", op="attn", kv_heads=8, group=8, dim=128, page=16, groups=0, per_group=4, prefix=0,
             least=81920, longest=81920, most_q=1, pad=0, shape=12),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["write", "write", "read", "attn", "attn", "attn"])
    c = dict(op=op, shape=rng.randrange(1 << 30), page=rng.choice([1, 4, 8, 16, 16, 32, 64, 128]))
    dim = rng.choice([8, 40, 64, 64, 80, 96, 128, 128, 128, 256])
    kv = rng.choice([1, 2, 5, 8, 8, 32]) if dim <= 128 else rng.choice([1, 2, 4])
    c |= dict(kv_heads=kv, dim=dim)
    if op == "attn":
        group = rng.choice([1, 2, 4, 4, 7, 8]) if kv <= 8 else rng.choice([1, 2])
        groups, longest = rng.choice([0, 0, 1, 2, 3]), _log(rng, 1, 12000)
        c |= dict(group=group, groups=groups, per_group=_log(rng, 1, 64 // max(1, groups)),
                  prefix=_log(rng, 1, 20000) if groups else 0, least=rng.randint(1, longest), longest=longest,
                  most_q=rng.choice([1, 1, 1, 2, 4, 9]), pad=rng.choice([0, 0, 5]))
        # no dearer than the largest listed case
        while max(1, groups) * c["per_group"] * (c["prefix"] + c["longest"]) * kv * dim * c["most_q"] > 300_000_000:
            c["prefix"] = max(1, c["prefix"] // 2) if groups else 0
            c["longest"] = max(1, c["longest"] * 3 // 4)
            c["least"] = min(c["least"], c["longest"])
            c["per_group"] = max(1, c["per_group"] * 3 // 4)
        return c
    layers = rng.randint(1, 32)
    room = max(64, 300_000_000 // (layers * kv * dim))  # tokens: at most 0.6 GB of K as binary16
    if op == "write":
        most, longest = _log(rng, 1, 900), _log(rng, 1, 600)
        c |= dict(layers=layers, rows=max(1, min(_log(rng, 1, 128), room // (2 * (most + longest)))), most=most,
                  longest=longest, wide=rng.choice([0, 0, 6, 64]))
    else:
        longest = _log(rng, 1, min(9216, room))
        c |= dict(layers=layers, rows=max(1, min(_log(rng, 1, 40), room // longest)), longest=longest)
    return c


def _cdiv(a, b):
    return -(-a // b)


def _row_bytes(kv, dim):
    groups = kv * _cdiv(dim, 32)
    return _cdiv(groups * 16 + groups * 2, 16) * 16


def _layout(c):
    """The whole numbers of a case: lengths and counts, from the case alone."""
    r = random.Random(c["shape"])
    if c["op"] == "write":
        return dict(lens=[r.randint(0, c["longest"]) for _ in range(c["rows"])],
                    counts=[r.randint(1, c["most"]) for _ in range(c["rows"])])
    if c["op"] == "read":
        if c["rows"] == 1:
            return dict(lens=[c["longest"]], first=[0], counts=[c["longest"]])
        lens = [r.randint(1, c["longest"]) for _ in range(c["rows"])]
        first = [r.randint(0, n - 1) for n in lens]
        return dict(lens=lens, first=first, counts=[r.randint(1, n - f) for n, f in zip(lens, first)])
    n = max(1, c["groups"]) * c["per_group"]
    ql = [c["most_q"] if c["most_q"] == 1 else r.randint(0, c["most_q"]) for _ in range(n)]
    tail = [max(q, r.randint(c["least"], c["longest"])) for q in ql]
    ql[-1] = max(1, ql[-1])
    tail[-1] = max(ql[-1], tail[-1])
    # the first group's prompt is the longest
    pre = [c["prefix"]] + [r.randint(_cdiv(c["prefix"], 2), c["prefix"]) for _ in range(c["groups"] - 1)]
    return dict(ql=ql, tail=tail, pre=pre, lens=[pre[i // c["per_group"]] + t for i, t in enumerate(tail)])


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _values(shape, g):
    """K or V as the codec's workloads have them: lognormal channel scales, a few outlier channels."""
    scale = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    scale = torch.where(torch.rand(shape[-1], generator=g, device="cuda") < 0.02, scale * 8, scale).half()
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float16) * scale


# --- the plain forms of a row ---------------------------------------------------


def _shifts():
    return torch.tensor([16 * (e % 2) + 4 * (e // 2) for e in range(8)], device="cuda")


def _quantise(x, kv, dim):
    """fp16 [..., kv * dim] -> codes int32 and scales fp32 [..., kv, groups, 32 and 1]."""
    x = x.float().unflatten(-1, (kv, dim))
    x = torch.nn.functional.pad(x, (0, -dim % 32)).unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(x).all(-1, keepdim=True)
    # A quotient that is no multiple of its unit, or no half, is off from one by 2^-13 of itself
    # at least (11 and 8 bits): a little less before rounding up, a little more before rounding
    # down, and a division's last bit decides nothing.
    v = x.abs().amax(-1, keepdim=True) * ((1 - 2.0 ** -20) / 7)
    m, e = torch.frexp(v)
    s = torch.where(v < 2.0 ** -16, torch.ceil(v * 2.0 ** 24) * 2.0 ** -24, torch.ldexp(torch.ceil(m * 256), e - 8))
    s = s.clamp(max=9344.0)
    n = torch.where(bad | (s == 0), 8.0, torch.floor(x / s + (8.5 + 2.0 ** -14))).int()
    return n, torch.where(bad, float("nan"), s)


def _store(n, s, pool):
    """Codes and scales of rows into bytes [..., row]."""
    kv, groups = n.shape[-3:-1]
    w = (n.unflatten(-1, (4, 8)).long() << _shifts()).sum(-1).flatten(-3)
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).int().view(torch.uint8)
    sc = s.flatten(-3).half().view(torch.uint8)
    pool[..., : kv * groups * 16] = w
    pool[..., kv * groups * 16: kv * groups * 18] = sc


def _held(n, s, dim):
    return ((n - 8) * s).flatten(-2)[..., :dim].flatten(-2)


def _load(rows, kv, dim):
    """Bytes [..., row] -> the values that they stand for, fp32 [..., kv, dim]."""
    groups = _cdiv(dim, 32)
    w = rows[..., : kv * groups * 16].contiguous().view(torch.int32)
    n = (w.unsqueeze(-1) >> _shifts().int()) & 15
    s = rows[..., kv * groups * 16: kv * groups * 18].contiguous().view(torch.float16).float()
    x = (n.unflatten(-2, (kv * groups, 4)).flatten(-2) - 8) * s.unsqueeze(-1)
    return x.unflatten(-2, (kv, groups)).flatten(-2)[..., :dim]


# --- state -----------------------------------------------------------------------


def _cache(s, c, tables, lens, refs, k, v):
    s["tables"], s["lens"], s["refs"] = _ints(tables), _ints(lens), _ints(refs)
    s["k_pool"], s["v_pool"] = k, v
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:  # the handle that a serving program keeps beside its cache
        import kv_cache_compression_anchor_amd as cg
        s["cache"] = cg.QuantCache(k, v, s["tables"], s["lens"], s["refs"], s["status"], c["kv_heads"] * c["dim"],
                                   c["dim"])


def _pool(layers, pages, c, g, filled):
    """[layers][pages][page][row] bytes: rows of values, or what the memory held before."""
    kv, dim = c["kv_heads"], c["dim"]
    shape = (layers, pages, c["page"], _row_bytes(kv, dim))
    if not filled:
        return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    pool = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (c["page"] * kv * dim))
    for layer in range(layers):
        for a in range(0, pages, step):
            part = pool[layer, a: a + step]
            _store(*_quantise(_values(part.shape[:2] + (kv * dim,), g), kv, dim), part)
    return pool


def prepare(case, seed):
    c, lay = case, _layout(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    h = torch.Generator().manual_seed(int(seed))
    P, kv, dim = c["page"], c["kv_heads"], c["dim"]
    s = dict(op=c["op"], P=P, kv=kv, dim=dim)
    if c["op"] == "write":
        n = sum(lay["counts"])
        blocks = [_cdiv(a + b, P) for a, b in zip(lay["lens"], lay["counts"])]
        pages = sum(blocks) + 3
        order, at, tables, slots = torch.randperm(pages, generator=h).tolist(), 0, [], []
        for a, b, m in zip(lay["lens"], lay["counts"], blocks):
            row = order[at:at + m]
            at += m
            tables.append(row + [-1] * (max(blocks) - m))
            slots += [row[t // P] * P + t % P for t in range(a, a + b)]
        refs = [0] * pages
        for p in order[:at]:
            refs[p] = 1
        s["slots"] = torch.tensor(slots, dtype=torch.int64, device="cuda")
        # K and V in one buffer, as a projection leaves them
        both = _values((c["layers"], n, 2 * kv * dim + c["wide"]), g)
        s["k_new"], s["v_new"] = both[..., : kv * dim], both[..., kv * dim: 2 * kv * dim]
        s["k_held"], s["v_held"] = (torch.zeros((c["layers"], n, kv * dim), dtype=torch.float16, device="cuda")
                                    for _ in range(2))
        _cache(s, c, tables, [a + b for a, b in zip(lay["lens"], lay["counts"])], refs,
               _pool(c["layers"], pages, c, g, False), _pool(c["layers"], pages, c, g, False))
        return s
    if c["op"] == "read":
        blocks = [_cdiv(n, P) for n in lay["lens"]]
        pages = sum(blocks) + 3
        order, at, tables = torch.randperm(pages, generator=h).tolist(), 0, []
        for m in blocks:
            tables.append(order[at:at + m] + [-1] * (max(blocks) - m))
            at += m
        refs = [0] * pages
        for p in order[:at]:
            refs[p] = 1
        s["n"] = sum(lay["counts"])
        s["rows"], s["first"], s["starts"] = (_ints(x) for x in (range(c["rows"]), lay["first"],
                                                                 _starts(lay["counts"])))
        s["slots"] = torch.zeros(s["n"], dtype=torch.int64, device="cuda")
        s["k_out"], s["v_out"] = (torch.zeros((c["layers"], s["n"], kv * dim), dtype=torch.float16, device="cuda")
                                  for _ in range(2))
        _cache(s, c, tables, lay["lens"], refs, _pool(c["layers"], pages, c, g, True),
               _pool(c["layers"], pages, c, g, True))
        return s
    n, per = len(lay["ql"]), c["per_group"]
    shared = [p // P for p in lay["pre"]]  # full pages of a prefix are shared, as forks leave them
    blocks = [_cdiv(m, P) for m in lay["lens"]]
    pages = sum(shared) + sum(b - shared[i // per] for i, b in enumerate(blocks)) + 3
    order, at, tables, refs = torch.randperm(pages, generator=h).tolist(), 0, [], [0] * pages
    for i, b in enumerate(blocks):
        sh = shared[i // per]
        if i % per == 0:
            pre = order[at:at + sh]
            at += sh
        row = pre + order[at:at + b - sh]
        at += b - sh
        for p in row:
            refs[p] += 1
        tables.append(row + [-1] * (max(blocks) - b))
    layers = 2 if pages * P * kv * dim < 100_000_000 else 1
    _cache(s, c, tables, lay["lens"], refs, _pool(layers, pages, c, g, True), _pool(layers, pages, c, g, True))
    for i in range(n):  # the rows of a prefix that end inside a page: a copy in each sequence
        p, f = lay["pre"][i // per], i - i % per
        if p % P and i != f:
            for x in (s["k_pool"], s["v_pool"]):
                x[:, tables[i][p // P], : p % P] = x[:, tables[f][p // P], : p % P]
    H, starts = kv * c["group"], _starts(lay["ql"])
    s |= dict(total=starts[-1], heads=H, layer=layers - 1, scale=dim ** -0.5, max_q=max(lay["ql"]),
              max_prefix=max(lay["pre"]), max_len=max(lay["lens"]), groups=c["groups"], n=n)
    s["q_starts"] = _ints(starts)
    s["group_starts"] = _ints([i * per for i in range(c["groups"] + 1)]) if c["groups"] else None
    s["prefix_lens"] = _ints(lay["pre"]) if c["groups"] else None
    n_q = starts[-1] + c["pad"]
    s["q"] = torch.randn((n_q, H, dim), generator=g, device="cuda", dtype=torch.float16)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((n_q, H), dtype=torch.float32, device="cuda")
    if own:  # the workspace that a serving program keeps
        import kv_cache_compression_anchor_amd as cg
        s["ws"] = torch.empty(cg.cg_quant_attention_workspace(s["cache"], n_q, H, n, s["groups"], s["max_q"],
                                                              s["max_prefix"], s["max_len"]),
                              dtype=torch.uint8, device="cuda")
    return s


# --- the framework's calls -------------------------------------------------------


def _own(s):
    import kv_cache_compression_anchor_amd as cg
    cache = s["cache"]
    if s["op"] == "write":
        cg.cg_quant_write_async(cache, 0, s["slots"], s["k_new"], s["v_new"], s["k_held"], s["v_held"])
        return dict(k=s["k_held"], v=s["v_held"], k_pool=s["k_pool"], v_pool=s["v_pool"])
    if s["op"] == "read":
        cg.cg_pages_slots_async(cache, s["rows"], s["first"], s["starts"], s["slots"])
        cg.cg_quant_read_async(cache, 0, s["slots"], s["k_out"], s["v_out"])
        return dict(slots=s["slots"], k=s["k_out"], v=s["v_out"])
    cg.cg_quant_attention_async(cache, s["layer"], s["q"], s["out"], s["scale"], None, s["q_starts"],
                                s["group_starts"], s["prefix_lens"], s["max_q"], s["max_prefix"], s["max_len"],
                                s["ws"], lse=s["lse"])
    return dict(out=s["out"], lse=s["lse"])


# --- the plain forms ---------------------------------------------------------------


def _plain_write(s):
    for new, pool, held in ((s["k_new"], s["k_pool"], s["k_held"]), (s["v_new"], s["v_pool"], s["v_held"])):
        n, sc = _quantise(new, s["kv"], s["dim"])
        held.copy_(_held(n, sc, s["dim"]))
        flat = pool.view(pool.shape[0], -1, pool.shape[3])
        rows = flat[:, s["slots"]]
        _store(n, sc, rows)
        flat[:, s["slots"]] = rows
    return dict(k=s["k_held"], v=s["v_held"], k_pool=s["k_pool"], v_pool=s["v_pool"])


def _plain_read(s):
    P, starts = s["P"], s["starts"].long()
    cnt = starts[1:] - starts[:-1]
    seq = torch.repeat_interleave(torch.arange(cnt.numel(), device=cnt.device), cnt, output_size=s["n"])
    pos = s["first"].long()[seq] + torch.arange(s["n"], device=cnt.device) - starts[seq]
    s["slots"].copy_(s["tables"][s["rows"].long()[seq], pos // P].long() * P + pos % P)
    for pool, out in ((s["k_pool"], s["k_out"]), (s["v_pool"], s["v_out"])):
        for layer in range(pool.shape[0]):
            rows = pool[layer].view(-1, pool.shape[3])[s["slots"]]
            out[layer] = _load(rows, s["kv"], s["dim"]).flatten(-2)
    return dict(slots=s["slots"], k=s["k_out"], v=s["v_out"])


def _plain_attn(s):
    P, d, H, n, kv = s["P"], s["dim"], s["heads"], s["n"], s["kv"]
    lens, starts = s["lens"].long(), s["q_starts"].long()
    ql = starts[1:] - starts[:-1]
    T, G = s["max_len"], H // kv
    t = torch.arange(T, device=lens.device)
    slot = s["tables"].long().clamp(min=0)[:, t // P] * P + t % P
    row = s["k_pool"].shape[3]
    # [sequence, kv head, token, d]
    k, v = (_load(x[s["layer"]].view(-1, row)[slot], kv, d).transpose(1, 2) for x in (s["k_pool"], s["v_pool"]))
    j = torch.arange(s["max_q"], device=lens.device)
    at = (starts[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().view(n, s["max_q"], kv, G, d).permute(0, 2, 1, 3, 4).reshape(n, kv, -1, d)
    x = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    lim = lens[:, None] - ql[:, None] + j + 1  # [sequence, query]: tokens that it sees
    x = x.view(n, kv, s["max_q"], G, T).masked_fill_((t >= lim[:, :, None])[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul((p / l).view(n, kv, -1, T), v.contiguous()).view(n, kv, s["max_q"], G, d)
    seq = torch.repeat_interleave(torch.arange(n, device=lens.device), ql, output_size=s["total"])
    own_j = torch.arange(s["total"], device=lens.device) - starts[seq]
    s["out"][: s["total"]] = o[seq, :, own_j].reshape(-1, H, d).half()
    s["lse"][: s["total"]] = (m + torch.log(l))[seq, :, own_j].reshape(-1, H)
    return dict(out=s["out"], lse=s["lse"])


def run(state):
    if own:
        return _own(state)
    return {"write": _plain_write, "read": _plain_read, "attn": _plain_attn}[state["op"]](state)


def work(case):
    c, lay = case, _layout(case)
    kv, dim = c["kv_heads"], c["dim"]
    row, values = _row_bytes(kv, dim), 2 * kv * dim  # of a token, K or V
    if c["op"] == "write":
        n = sum(lay["counts"])
        return dict(bytes=n * (2 * c["layers"] * (row + 2 * values) + 8), flops=0)
    if c["op"] == "read":
        n = sum(lay["counts"])
        return dict(bytes=n * (2 * c["layers"] * (row + values) + 8), flops=0)
    H, nq = kv * c["group"], sum(lay["ql"])
    tokens = sum(lay["lens"])
    if c["groups"]:
        tokens = sum(lay["pre"]) + sum(lay["tail"])
    seen = sum(n * m - m * (m - 1) // 2 for n, m in zip(lay["lens"], lay["ql"]))
    return dict(bytes=2 * row * tokens + nq * H * (4 * dim + 4), flops=4 * dim * H * seen)


# --- the definitions, in 64 bits and whole numbers -----------------------------------


def _exact_scale(a):
    """float64 magnitudes -> float64 scales."""
    q = a / torch.full_like(a, 7.0)
    unit = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -40))) - 7).clamp(min=2.0 ** -24)
    return (torch.ceil(q / unit - 1e-9) * unit).clamp(max=9344)


def _exact_values(rows, kv, dim):
    """Bytes [n, row] -> float64 [n, kv, dim], channel by channel of a word."""
    groups = _cdiv(dim, 32)
    b = rows[:, : kv * groups * 16].reshape(-1, kv, groups * 4, 4).long()
    x = torch.empty(b.shape[:3] + (8,), dtype=torch.float64, device=rows.device)
    for e in range(8):
        byte = b[..., 2 * (e % 2) + e // 4]
        x[..., e] = (byte // 16 if e // 2 % 2 else byte % 16) - 8
    s = rows[:, kv * groups * 16: kv * groups * 18].contiguous().view(torch.float16).double()
    return (x.flatten(-2).unflatten(-1, (groups, 32)) * s.view(-1, kv, groups, 1)).flatten(-2)[..., :dim]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    P, kv, d = s["P"], s["kv"], s["dim"]
    row = s["k_pool"].shape[3]
    if c["op"] == "write":
        got = {}
        for name in "kv":
            new, pool, out = s[name + "_new"], s[name + "_pool"], torch.empty_like(s[name + "_held"]).double()
            for layer in range(new.shape[0]):
                x = new[layer].double().view(-1, kv, d)
                rows = pool[layer].view(-1, row)[s["slots"]]
                for j in range(_cdiv(d, 32)):
                    y = x[..., 32 * j: 32 * j + 32]
                    sc = _exact_scale(y.abs().amax(-1))
                    n = torch.floor(y / torch.where(sc > 0, sc, 1.0)[..., None] + (0.5 + 1e-9))
                    out[layer].view(-1, kv, d)[..., 32 * j: 32 * j + 32] = n * sc[..., None]
                    n = torch.nn.functional.pad(n, (0, 32 - y.shape[-1])).long() + 8
                    head = torch.arange(kv, device="cuda")[:, None] * _cdiv(d, 32) + j
                    for e in range(0, 32, 8):  # bytes of a word: channels 0 and 2, 4 and 6, 1 and 3, 5 and 7
                        for i, (lo, hi) in enumerate(((0, 2), (4, 6), (1, 3), (5, 7))):
                            rows[:, (head * 16 + e // 2 + i).flatten()] = (n[..., e + lo] + 16 * n[..., e + hi]).byte()
                    half = sc.half().unsqueeze(-1).view(torch.uint8)
                    for i in range(2):
                        rows[:, (kv * _cdiv(d, 32) * 16 + 2 * head + i).flatten()] = half[..., i]
                pool[layer].view(-1, row).index_copy_(0, s["slots"], rows)
            got[name], got[name + "_pool"] = out, pool
        return dict(k=got["k"], v=got["v"], k_pool=got["k_pool"], v_pool=got["v_pool"])
    T = s["tables"].tolist()
    if c["op"] == "read":
        starts, slots = s["starts"].tolist(), []
        for i, (r, f) in enumerate(zip(s["rows"].tolist(), s["first"].tolist())):
            slots += [T[r][t // P] * P + t % P for t in range(f, f + starts[i + 1] - starts[i])]
        at = torch.tensor(slots, device="cuda")
        k, v = (torch.stack([_exact_values(layer.view(-1, row)[at], kv, d).flatten(-2) for layer in x])
                for x in (s["k_pool"], s["v_pool"]))
        return dict(slots=at, k=k, v=v)
    n, H = s["lens"].tolist(), s["heads"]
    out, lse = torch.zeros(s["q"].shape, dtype=torch.float64), torch.zeros(s["lse"].shape, dtype=torch.float64)
    starts = s["q_starts"].tolist()
    for i, pages in enumerate(T):
        a, b = starts[i], starts[i + 1]
        if a == b:
            continue
        at = torch.tensor(pages[: _cdiv(n[i], P)], device="cuda")
        K, V = (_exact_values(x[s["layer"], at].reshape(-1, row)[: n[i]], kv, d) for x in (s["k_pool"], s["v_pool"]))
        for h in range(kv):
            g = H // kv
            Q = s["q"][a:b, h * g:(h + 1) * g].double()  # [query, head of the group, d]
            x = (Q.reshape(-1, d) @ K[:, h].T.contiguous() * s["scale"]).view(b - a, g, n[i])
            for j in range(b - a):
                seen = n[i] - (b - a) + j + 1
                y = x[j, :, :seen]
                z = torch.logsumexp(y, -1)
                out[a + j, h * g:(h + 1) * g] = (torch.exp(y - z[:, None]) @ V[:seen, h].contiguous()).cpu()
                lse[a + j, h * g:(h + 1) * g] = z.cpu()
    return dict(out=out, lse=lse)
