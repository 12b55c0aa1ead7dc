"""Cases that measure the operators of many continuations of shared prompts on 8-bit key/value caches.

Four operators: attention for rows that share the places of a long prefix, which is read once for all
rows of a group ("attend"); one token per row drawn from its logits with the row's own temperature,
top-k, top-p and min-p ("sample"); rows of a page table that fork, shrink, grow and are freed, with the
copies of the pages they would both write ("fork"); and the pages in use moved to the front of the pool
("compact").

run() computes a case in elementary torch operations, or with `own` through the package's entry
points; exact() from the definitions, in 64 bits.  Shapes are those of the repository's workloads (an 8B
decoder: 8 key/value heads of 128, groups of 4, 32 layers; a 1.7B decoder: 32 heads of 64; a 135M one: 3
heads of 64, 30 layers; vocabularies of 49152 and 128256) and generic ones.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16   # positions that share a scale
PAGE = 64    # positions of a page
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GREEDY = 0.0


# ---- cases ----------------------------------------------------------------------------------

def listed():
    return [
        # four samples of one short prompt, 8B shape, one decode step
        dict(name="attend_b4", op="attend", rows=4, groups=1, tokens=1, kv=8, group=4, head=128, prefix=1000, suffix=45, type="f32", paged=True),
        # 32 requests behind one long system prompt, each with a conversation of its own
        dict(name="attend_b32", op="attend", rows=32, groups=1, tokens=1, kv=8, group=4, head=128, prefix=8192, suffix=511, type="bf16", paged=True),
        # several prompts with several samples each (uneven groups), 1.7B shape, rows in place
        dict(name="attend_groups", op="attend", rows=48, groups=6, tokens=1, kv=32, group=1, head=64, prefix=2047, suffix=130, type="f32", paged=False),
        # drafted tokens of 16 rows behind one prompt
        dict(name="attend_drafts", op="attend", rows=16, groups=1, tokens=5, kv=8, group=4, head=128, prefix=4099, suffix=300, type="f32", paged=True),
        # a document of 131072 positions that 64 questions are asked about
        dict(name="attend_document", op="attend", rows=64, groups=1, tokens=1, kv=8, group=4, head=128, prefix=131072, suffix=200, type="bf16", paged=True),
        # one sequence, and batches whose rows bring their own settings
        dict(name="sample_b1", op="sample", rows=1, vocab=49152),
        dict(name="sample_b32", op="sample", rows=32, vocab=128256),
        dict(name="sample_b256_odd", op="sample", rows=256, vocab=50257),
        # one prompt of a small model forked into four rows
        dict(name="fork_b4", op="fork", rows=4, fan=4, length=333, kv=3, head=64, layers=30),
        # eight prompts forked into 64 rows, 8B shape
        dict(name="fork_b64", op="fork", rows=64, fan=8, length=1000, kv=8, head=128, layers=32),
        # a small pool, and a large one from which requests of all lengths have gone
        dict(name="compact_small", op="compact", rows=6, pages=96, fill=0.5, kv=3, head=64, layers=30),
        dict(name="compact_8b", op="compact", rows=24, pages=1088, fill=0.6, kv=8, head=128, layers=16),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "sample", "fork", "compact"])
    if op == "sample":
        return dict(op=op, rows=_spread(rng, 1, 256), vocab=_spread(rng, 1000, 128256))
    kv, head = rng.choice([1, 2, 3, 4, 8, 8, 16, 32]), rng.choice([64, 128])
    if op == "attend":
        out = dict(op=op, rows=_spread(rng, 1, 64), tokens=rng.choice([1, 1, 1, 2, 5, 8]), kv=kv, head=head,
                   group=rng.choice([1, 2, 3, 4, 5, 7, 8]), type=rng.choice(["f32", "bf16"]), paged=rng.random() < 0.6)
        out["groups"] = rng.randint(1, min(8, out["rows"]))
        heads = out["rows"] * out["tokens"] * kv * out["group"]
        # no more work than the largest listed case, and no more cache than about 1 GB
        held = kv * head * 2 * (out["groups"] if out["paged"] else out["rows"])
        most = min(131072, int(1.3e11 / (4 * heads * head)), int(1e9 / held))
        out["prefix"] = _spread(rng, 1, max(64, most))
        out["suffix"] = out["tokens"] + _spread(rng, 1, max(16, min(2048, int(4e8 / (kv * head * 2 * out["rows"])))))
        return out
    layers = _spread(rng, 1, 32)
    if op == "fork":
        fan = rng.choice([2, 3, 4, 8])
        return dict(op=op, rows=fan * _spread(rng, 1, 64 // fan), fan=fan, length=_spread(rng, 70, 1000), kv=min(kv, 8), head=head, layers=layers)
    return dict(op=op, rows=_spread(rng, 1, 32), pages=_spread(rng, 64, 1000), fill=round(0.3 + 0.5 * rng.random(), 3), kv=min(kv, 8), head=head,
                layers=_spread(rng, 1, 16))


def work(case):
    c = case
    if c["op"] == "sample":
        return {"bytes": c["rows"] * (c["vocab"] * 4 + 24), "flops": 2 * c["rows"] * c["vocab"]}
    if c["op"] == "attend":
        bound, prefix, length = _shared(c)
        own_ = int((length - np.repeat(prefix, np.diff(bound))).sum())
        heads, size = c["kv"] * c["group"], 4 if c["type"] == "f32" else 2
        values = (int(prefix[np.diff(bound) > 0].sum()) + own_) * c["kv"] * c["head"] * 2
        ends = c["rows"] * c["tokens"] * heads * c["head"] * size * 2
        return {"bytes": values + values // (BLOCK * c["head"]) * 4 + ends, "flops": 4 * int(length.sum()) * c["tokens"] * heads * c["head"]}
    page = c["kv"] * (PAGE * c["head"] + PAGE // BLOCK * 4) * 2
    if c["op"] == "fork":
        moves, table = c["rows"] - c["rows"] // c["fan"], c["rows"] * (c["length"] // PAGE + 2)
    else:
        moves, table = _high(c), _used(c)
    return {"bytes": moves * c["layers"] * page * 2 + table * 8, "flops": moves + table}


def _shared(c):
    """Row bounds of the groups, positions that each shares, and the rows' lengths; all uneven."""
    G, B = c["groups"], c["rows"]
    bound = np.array([int(B * (i / G) ** 1.2) for i in range(G)] + [B])
    prefix = np.maximum(1, c["prefix"] - np.arange(G) * 97 % max(1, c["prefix"] // 3))
    suffix = np.maximum(c["tokens"], c["suffix"] - np.arange(B) * 37 % max(1, c["suffix"] // 2))
    return bound, prefix, np.repeat(prefix, np.diff(bound)) + suffix


def _used(c):
    return max(c["rows"], int(c["pages"] * c["fill"]))


def _high(c):
    """How many of the pages in use lie behind as many pages as are in use."""
    return min(c["pages"] - _used(c), int(_used(c) * (1 - c["fill"])))


# ---- inputs ---------------------------------------------------------------------------------

def _pow2_scale(amax):
    """The least power of two s >= 2^-126 with amax / s <= 448 (the largest e4m3 value)."""
    m, e = torch.frexp(amax)
    e = torch.where(amax == 0, -126, e - 9 + (m > 0.875).int()).clamp(min=-126)
    return (e.int() + 127 << 23).view(torch.float32)


def _filled(rows, kv, cap, head, g, wide):
    """Codes and scales of a cache whose every position holds a value: keys and values are normal,
    with a head-wise spread and a few large key channels, as decoders have them."""
    codes = torch.empty((rows, kv, cap // BLOCK, BLOCK, head), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, kv, cap // BLOCK), device="cuda")
    spread = torch.exp(torch.randn(kv, 1, 1, head, device="cuda", generator=g) * (0.5 if wide else 0.2))
    for r in range(rows):
        x = torch.randn((kv, cap // BLOCK, BLOCK, head), device="cuda", generator=g) * spread
        scales[r] = _pow2_scale(x.abs().amax((-1, -2)))
        codes[r] = (x / scales[r][..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(rows, kv, cap, head), scales


def _int32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def _layers(c, rows, cap, g):
    """The caches of all layers, every code and scale a value."""
    out = {}
    for name in ("k", "v"):
        bits = torch.randint(-1 << 31, 1 << 31, (c["layers"], rows, c["kv"], cap, c["head"] // 4), device="cuda", generator=g, dtype=torch.int32)
        out[name] = (bits & -0x40404041).view(torch.uint8)                               # (any sign, no code of a NaN)
        out[name + "_scale"] = torch.exp2(torch.randint(-6, 3, (c["layers"], rows, c["kv"], cap // BLOCK), device="cuda", generator=g).float())
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = dict(case=c)
    if c["op"] == "sample":
        B, V = c["rows"], c["vocab"]
        s["logits"] = torch.randn(B, V, device="cuda", generator=g) * 2.5
        s["temp"] = torch.from_numpy(rng.choice([GREEDY, 0.6, 0.8, 1.0, 1.0, 1.5], B).astype(np.float32)).cuda()
        s["k"] = _int32(rng.choice([V, V, 20, 50, 1000, V // 3], B))
        s["p"] = torch.from_numpy(rng.choice([1.0, 0.9, 0.95, 0.99], B).astype(np.float32)).cuda()
        s["min_p"] = torch.from_numpy(rng.choice([0.0, 0.0, 0.02, 0.1], B).astype(np.float32)).cuda()
        if B == 1:  # a sequence is drawn from with top-p
            s["temp"].fill_(0.8)
            s["k"].fill_(V)
            s["p"].fill_(0.95)
        s["u"] = torch.randint(0, 1 << 24, (B,), device="cuda", generator=g).float() / (1 << 24)
        s["ids"] = torch.empty(B, dtype=torch.int32, device="cuda")
        return s
    if c["op"] == "attend":
        bound, prefix, length = _shared(c)
        B, G = c["rows"], c["groups"]
        leader = np.repeat(bound[:-1], np.diff(bound))
        shared = np.repeat(prefix, np.diff(bound))
        held = -(-length // PAGE)
        per_row = int(held.max())
        s["table"] = None
        if c["paged"]:
            # a row has the leader's pages where all of a page is shared, else its own, scattered over the pool
            table = np.full((B, per_row), -1, np.int64)
            first = np.where(np.arange(B) == leader, 0, shared // PAGE)
            pool_rows = 4
            cap = -(-int((held - first).sum()) // pool_rows) * PAGE
            free, at = rng.permutation(pool_rows * cap // PAGE), 0
            for b in range(B):
                table[b, : first[b]] = table[leader[b], : first[b]]
                table[b, first[b] : held[b]] = free[at : at + held[b] - first[b]]
                at += held[b] - first[b]
            s["table"] = _int32(table)
        else:
            pool_rows, cap = B, per_row * PAGE
        s["k"], s["k_scale"] = _filled(pool_rows, c["kv"], cap, c["head"], g, True)
        s["v"], s["v_scale"] = _filled(pool_rows, c["kv"], cap, c["head"], g, False)
        shape = (B, c["tokens"], c["kv"] * c["group"], c["head"])
        s["q"] = (torch.randn(shape, device="cuda", generator=g) * 1.5).to(TYPES[c["type"]])
        s["out"] = torch.zeros_like(s["q"])
        s["length"], s["groups"], s["shared"] = _int32(length), _int32(bound), _int32(prefix)
        s["most"] = (int(prefix.max()), int((length - shared).max()), int(np.diff(bound).max()))
        return s
    if c["op"] == "fork":
        # every fan-th row holds a prompt that ends inside a page; the others' tables are empty
        R = c["rows"]
        per_row = -(-(c["length"] + 1) // PAGE)
        pages = 2 * R * per_row
        old = np.maximum(1, c["length"] - rng.integers(0, 64, R) - 1)
        old += old % PAGE == 0
        old[np.arange(R) % c["fan"] != 0] = 0
        held = -(-old // PAGE)
        table, free, at = np.full((R, per_row), -1, np.int64), rng.permutation(pages), 0
        for r in range(R):
            table[r, : held[r]] = free[at : at + held[r]]
            at += held[r]
        parent = np.arange(R) // c["fan"] * c["fan"]
        s["parent"], s["new"] = _int32(parent), _int32(old[parent] + 1)
        moves = R
    else:
        R, pages, used, high = c["rows"], c["pages"], _used(c), _high(c)
        at = np.concatenate([rng.permutation(used)[: used - high], used + rng.permutation(pages - used)[:high]])
        at = rng.permutation(at)
        bound = np.array([int(used * (r / R) ** 1.5) for r in range(R)] + [used])
        held = np.diff(bound)
        per_row = int(held.max())
        table = np.full((R, per_row), -1, np.int64)
        for r, n in enumerate(held):
            table[r, :n] = at[bound[r] : bound[r + 1]]
        old = np.maximum(0, held * PAGE - rng.integers(0, PAGE, R))
        moves = max(1, pages // 2)
    pool_rows = 4 if pages % 4 == 0 else 1
    s.update(_layers(c, pool_rows, pages // pool_rows * PAGE, g), table=_int32(table), length=_int32(old), pages=pages)
    s["table_out"], s["length_out"] = torch.empty_like(s["table"]), torch.empty_like(s["length"])
    s["moves"] = torch.empty(moves, 2, dtype=torch.int32, device="cuda")
    s["counts"] = torch.empty(2, dtype=torch.int32, device="cuda")
    return s


# ---- the plain forms ------------------------------------------------------------------------

def _places(s, row, block):
    """Cache row and block in it of blocks `block` of the call's rows `row`."""
    if s["table"] is None:
        return row.expand_as(block), block
    per_page, per_row = PAGE // BLOCK, s["k"].shape[2] // PAGE
    page = s["table"].long()[row, (block // per_page).clamp(max=s["table"].shape[1] - 1)].clamp(min=0)
    return page // per_row, page % per_row * per_page + block % per_page


def _values(codes, scales, r, b):
    """The values that blocks stand for: [n][kv][blocks * 16][head] from places [n][blocks]."""
    rows, kv, cap, head = codes.shape
    at = (r[:, None], torch.arange(kv, device="cuda")[:, None], b[:, None])
    x = codes.view(rows, kv, cap // BLOCK, BLOCK, head)[at].view(torch.float8_e4m3fn).float()
    return (x * scales[at][..., None, None]).flatten(2, 3)


def _attend_plain(s):
    c, L = s["case"], s["length"].long()
    B, S, G, kv, g, head = c["rows"], c["tokens"], c["groups"], c["kv"], c["group"], c["head"]
    bound, shared = s["groups"].long(), s["shared"].long()
    most_shared, most_own, most_rows = s["most"]
    row = torch.arange(B, device="cuda")
    of = torch.searchsorted(bound, row, right=True) - 1                                 # the row's group
    x = s["q"].float().view(B, S, kv, g, head).permute(0, 2, 1, 3, 4).flatten(2, 3)     # [B][kv][S * g][head]
    x = x * head ** -0.5
    see = (L[:, None] - S + 1 + torch.arange(S, device="cuda")).repeat_interleave(g, 1)  # [B][S * g] positions seen
    # the shared positions: the rows of a group as one batch of queries
    n = -(-most_shared // BLOCK)
    block = torch.arange(n, device="cuda").expand(G, n)
    r, b = _places(s, bound[:-1, None].clamp(max=B - 1), block.clamp(max=s["k"].shape[2] // BLOCK - 1) if s["table"] is None else block)
    member = (bound[:-1, None] + torch.arange(most_rows, device="cuda")).clamp(max=B - 1)  # [G][rows]
    queries = x[member].transpose(1, 2).flatten(2, 3)                                   # [G][kv][rows * S * g][head]
    place = torch.arange(n * BLOCK, device="cuda")
    seen = place < torch.minimum(see[member].flatten(1, 2), shared[:, None])[:, :, None]
    score = torch.matmul(queries, _values(s["k"], s["k_scale"], r, b).transpose(-1, -2))
    score = torch.where(seen[:, None], score, -torch.inf)
    # their own
    m = -(-(most_own + BLOCK) // BLOCK)
    mine = (shared[of] // BLOCK)[:, None] + torch.arange(m, device="cuda")              # [B][blocks]
    limit = s["k"].shape[2] if s["table"] is None else s["table"].shape[1] * PAGE
    r2, b2 = _places(s, row[:, None], mine.clamp(max=limit // BLOCK - 1))
    place2 = (mine[:, :, None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(1)
    seen2 = (place2[:, None] >= shared[of][:, None, None]) & (place2[:, None] < see[:, :, None])
    score2 = torch.where(seen2[:, None], torch.matmul(x, _values(s["k"], s["k_scale"], r2, b2).transpose(-1, -2)), -torch.inf)
    # one softmax over both
    slot = row - bound[of]
    top1 = score.amax(-1).view(G, kv, most_rows, S * g)[of, :, slot]
    top = torch.maximum(top1, score2.amax(-1))                                          # [B][kv][S * g]
    spread = top[member].transpose(1, 2).flatten(2, 3)[..., None]
    score.sub_(spread).exp_()
    total = score.sum(-1).view(G, kv, most_rows, S * g)[of, :, slot]
    o = torch.matmul(score, _values(s["v"], s["v_scale"], r, b)).view(G, kv, most_rows, S * g, head)[of, :, slot]
    w = torch.exp(score2 - top[..., None])
    o = (o + torch.matmul(w, _values(s["v"], s["v_scale"], r2, b2))) / (total + w.sum(-1))[..., None]
    return o.view(B, kv, S, g, head).permute(0, 2, 1, 3, 4).reshape(s["q"].shape).to(s["q"].dtype)


def _share(total, part24):
    """floor(part24 * total / 2^24) in 64 bits."""
    return part24 * (total >> 24) + (part24 * (total & 0xFFFFFF) >> 24)


def _sample_plain(s):
    v, V = s["logits"], s["logits"].shape[1]
    top = v.amax(-1, keepdim=True)
    index = torch.arange(V, device="cuda")
    best = torch.where(v == top, index, V).amin(-1)
    inverse = (1.0 / s["temp"]).clamp(max=torch.finfo(torch.float32).max)[:, None]
    q = ((top - v) * inverse).clamp(max=30.0).double().mul(1 << 27).floor()             # distance from the top, in 2^-27
    q, order = torch.sort(q, dim=-1, stable=True)
    w = torch.exp(-q / (1 << 27)).mul(2.0 ** 31).round().long()
    kept = index < s["k"].long()[:, None]
    before = w.cumsum(-1) - w
    total = (w * kept).sum(-1)
    limit = _share(total, s["p"].double().mul(1 << 24).floor().long())
    kept &= (before < limit[:, None]) | (index == 0)
    kept &= w >= s["min_p"].double().mul(2.0 ** 31).floor().long()[:, None]
    total = (w * kept).sum(-1)
    goal = _share(total, s["u"].double().mul(1 << 24).floor().long())
    at = ((before + w <= goal[:, None]) & kept).sum(-1)
    drawn = order.gather(1, at[:, None])[:, 0]
    return torch.where(s["temp"] == 0, best, drawn).int()


def _first(mask):
    """The indices at which mask holds, ascending, before the others."""
    return torch.sort((~mask).int(), stable=True)[1]


def _fork_plain(s):
    old, length, parent, new = s["table"].long(), s["length"].long(), s["parent"].long(), s["new"].long()
    R, per_row = old.shape
    row, j = torch.arange(R, device="cuda"), torch.arange(per_row, device="cuda")
    alive = parent >= 0
    keep = torch.where(alive, torch.minimum(length[parent.clamp(min=0)], new), 0)
    kept, total = (keep + PAGE - 1) // PAGE, torch.where(alive, (new + PAGE - 1) // PAGE, 0)
    base = old[parent.clamp(min=0)]
    is_kept, open_ = j < kept[:, None], keep % PAGE != 0
    last = base.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0]
    is_open = open_[:, None] & (j == kept[:, None] - 1)
    page = torch.where(is_kept, base, s["pages"])                                       # (one page more takes what counts not)
    whole = torch.zeros(s["pages"] + 1, dtype=torch.long, device="cuda")
    whole.scatter_add_(0, page.flatten(), (is_kept & ~is_open).long().flatten())
    lowest = torch.full((s["pages"] + 1,), R, device="cuda")
    lowest.scatter_reduce_(0, torch.where(open_, last, s["pages"]), row, "amin")
    copied = open_ & ((whole[last.clamp(min=0)] > 0) | (lowest[last.clamp(min=0)] != row))
    taken = ((whole > 0) | (lowest < R))[:-1]
    free = torch.nn.functional.pad(_first(~taken), (0, per_row + 2))
    need = copied.long() + total - kept
    at = need.cumsum(0) - need
    fresh = free[(at[:, None] + copied.long()[:, None] + j - kept[:, None]).clamp(0, s["pages"])]
    table = torch.where(is_kept, base, torch.where(j < total[:, None], fresh, -1))
    table = torch.where(is_open & copied[:, None], free[at.clamp(max=s["pages"])][:, None], table)
    moves = torch.full((R + 1, 2), -1, device="cuda")
    moves[torch.where(copied, copied.long().cumsum(0) - 1, R)] = torch.stack([last, free[at.clamp(max=s["pages"])]], 1)
    s["table_out"].copy_(table)
    s["length_out"].copy_(torch.where(alive, new, 0))
    s["moves"].copy_(moves[:R])
    s["moves"][copied.sum() <= row] = -1
    s["counts"].copy_(torch.stack([copied.sum(), taken.sum() + need.sum()]))


def _compact_plain(s):
    table, pages = s["table"].long(), s["pages"]
    held = torch.arange(table.shape[1], device="cuda") < ((s["length"] + PAGE - 1) // PAGE)[:, None]
    used = torch.zeros(pages + 1, dtype=torch.bool, device="cuda")
    used[torch.where(held, table, pages)] = True
    used = used[:-1]
    index, total = torch.arange(pages, device="cuda"), used.sum()
    src, dst = _first(used & (index >= total)), _first(~used & (index < total))
    n = (used & (index >= total)).sum()
    to = index.clone()
    to[src] = torch.where(index < n, dst, src)
    s["table_out"].copy_(torch.where(held, to[table.clamp(min=0)], -1))
    s["length_out"].copy_(s["length"])
    m = s["moves"].shape[0]
    s["moves"].copy_(torch.where(index[:m, None] < n, torch.stack([src[:m], dst[:m]], 1), -1))
    s["counts"].copy_(torch.stack([n, total]))


def _copy_plain(s):
    """The pages of every layer; moves behind the last repeat the first."""
    moves = torch.where(s["moves"][:, :1] >= 0, s["moves"], s["moves"][:1].clamp(min=0)).long()
    per_row = s["k"].shape[3] // PAGE
    at = lambda page: (slice(None), page // per_row, slice(None), page % per_row)  # noqa: E731
    for name in ("k", "v", "k_scale", "v_scale"):
        x = s[name]
        x = x.view(*x.shape[:3], per_row, -1)
        x[at(moves[:, 1])] = x[at(moves[:, 0])]


def _caches(s, package):
    """The package's views of the layers' caches, which a program makes once."""
    if "caches" not in s:
        layer = lambda i: package.QCache(*(s[n][i] for n in ("k", "v", "k_scale", "v_scale")))  # noqa: E731
        s["caches"] = package.QCacheLayers([layer(i) for i in range(s["case"]["layers"])])
        s["book"] = package.Pages(s["table"], s["length"], s["pages"])
        s["book_out"] = package.Pages(s["table_out"], s["length_out"], s["pages"])
        s["workspace"] = s["book"].workspace()
    return s["caches"]


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import llama_architecture_kv_gb300 as package
        stream = torch.cuda.current_stream().cuda_stream
        if op == "sample":
            package.llm_sample_rows(s["logits"], s["temp"], s["u"], s["ids"], k=s["k"], p=s["p"], min_p=s["min_p"], stream=stream)
            return s["ids"]
        if op == "attend":
            if "cache" not in s:  # a program keeps these beside its cache
                s["cache"] = package.QCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
                s["workspace"] = s["cache"].workspace_shared(s["case"]["group"], s["case"]["rows"], s["case"]["tokens"], s["case"]["groups"])
            s["cache"].attend_shared(s["q"], s["length"], s["groups"], s["shared"], s["out"], s["workspace"], table=s["table"], stream=stream)
            return s["out"]
        caches = _caches(s, package)
        if op == "fork":
            s["book"].update(s["book_out"], s["moves"], s["counts"], s["workspace"], parent=s["parent"], length=s["new"], stream=stream)
        else:
            s["book"].compact(s["book_out"], s["moves"], s["counts"], s["workspace"], stream=stream)
        caches.copy(s["moves"], counts=s["counts"], stream=stream)
    elif op == "sample":
        return _sample_plain(s)
    elif op == "attend":
        return _attend_plain(s)
    else:
        _fork_plain(s) if op == "fork" else _compact_plain(s)
        _copy_plain(s)
    return (s["table_out"], s["length_out"], s["moves"], s["counts"], s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn),
            s["k_scale"], s["v_scale"])


# ---- the definitions in 64 bits -------------------------------------------------------------

def _e4m3_values():
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v[(code & 127) == 127] = np.nan
    return np.where(code & 128, -v, v)


def _exact_attend(s):
    c = s["case"]
    lut = torch.from_numpy(_e4m3_values()).cuda()
    table = None if s["table"] is None else s["table"].cpu().numpy()
    bound, shared, length = (s[n].tolist() for n in ("groups", "shared", "length"))
    cap = s["k"].shape[2]

    def values(codes, scales, head, row, lo, hi):
        """Positions lo .. hi - 1 of a row, in 64 bits."""
        got = []
        for p in range(lo // PAGE, -(-hi // PAGE)):
            a, b = max(lo, p * PAGE), min(hi, (p + 1) * PAGE)
            r, at = row, a
            if table is not None:
                page = int(table[row, p])
                r, at = page // (cap // PAGE), page % (cap // PAGE) * PAGE + a % PAGE
            got.append((r, at, b - a))
        if not got:
            return torch.zeros(0, c["head"], dtype=torch.float64, device="cuda")
        r = np.concatenate([np.full(n, r) for r, _, n in got])
        at = np.concatenate([np.arange(a, a + n) for _, a, n in got])
        r, at = torch.from_numpy(r).cuda(), torch.from_numpy(at).cuda()
        return lut[codes[r, head, at].long()] * scales[r, head, at // BLOCK].double()[:, None]

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    S, g = c["tokens"], c["group"]
    for i in range(c["groups"]):
        lo, hi, n = bound[i], bound[i + 1], shared[i]
        for h in range(c["kv"] if hi > lo else 0):
            k1, v1 = values(s["k"], s["k_scale"], h, lo, 0, n), values(s["v"], s["v_scale"], h, lo, 0, n)
            for b in range(lo, hi):
                k = torch.cat([k1, values(s["k"], s["k_scale"], h, b, n, length[b])])
                v = torch.cat([v1, values(s["v"], s["v_scale"], h, b, n, length[b])])
                for t in range(S):
                    m = length[b] - S + t + 1
                    w = torch.softmax(s["q"][b, t, h * g : (h + 1) * g].double() @ k[:m].T / math.sqrt(c["head"]), -1)
                    out[b, t, h * g : (h + 1) * g] = w @ v[:m]
    return out


def _exact_sample(s):
    ids = []
    for b in range(s["case"]["rows"]):
        v = s["logits"][b].cpu().numpy()
        temp, k, p, min_p, u = (s[n][b].item() for n in ("temp", "k", "p", "min_p", "u"))
        if temp == 0:
            ids.append(int(np.argmax(v)))
            continue
        far = (v.max() - v) * (np.float32(1) / np.float32(temp))
        far = np.floor(np.minimum(far, np.float32(30)).astype(np.float64) * 2.0 ** 27)
        order = np.argsort(far, kind="stable")[:k]
        w = [int(x) for x in np.rint(np.exp(-far[order] * 2.0 ** -27) * 2.0 ** 31)]
        limit, cut, before = math.floor(p * 2 ** 24) * sum(w) >> 24, 0, 0
        while cut < len(w) and (cut == 0 or before < limit) and w[cut] >= math.floor(min_p * 2 ** 31):
            before += w[cut]
            cut += 1
        goal, at, run_ = math.floor(u * 2 ** 24) * before >> 24, 0, w[0]
        while run_ <= goal:
            at += 1
            run_ += w[at]
        ids.append(int(order[at]))
    return np.array(ids, np.int32)


def _exact_pages(s):
    c, table, length = s["case"], s["table"].tolist(), s["length"].tolist()
    rows, per_row, pages = len(table), len(table[0]), s["pages"]
    moves, out = [], [[-1] * per_row for _ in range(rows)]
    if c["op"] == "fork":
        parent, new = s["parent"].tolist(), s["new"].tolist()
        keep = [min(length[p], n) if p >= 0 else 0 for p, n in zip(parent, new)]
        mine = [table[max(p, 0)][: -(-n // PAGE)] for p, n in zip(parent, keep)]
        whole = {x for m, n in zip(mine, keep) for x in m[: n // PAGE]}
        opened = {}
        for r in range(rows):
            if keep[r] % PAGE:
                opened.setdefault(mine[r][-1], r)
        free = (x for x in range(pages) if x not in whole and x not in opened)
        for r in range(rows):
            if keep[r] % PAGE and (mine[r][-1] in whole or opened[mine[r][-1]] != r):
                moves.append((mine[r][-1], next(free)))
                mine[r] = mine[r][:-1] + [moves[-1][1]]
            total = -(-new[r] // PAGE) if parent[r] >= 0 else 0
            mine[r] = mine[r] + [next(free) for _ in range(total - len(mine[r]))]
            out[r][:total] = mine[r]
        length = [n if p >= 0 else 0 for p, n in zip(parent, new)]
        used = len({x for m in mine for x in m})
    else:
        mine = [t[: -(-n // PAGE)] for t, n in zip(table, length)]
        held = {x for m in mine for x in m}
        used = len(held)
        moves = list(zip(sorted(x for x in held if x >= used), (x for x in range(used) if x not in held)))
        to = dict(moves)
        for r in range(rows):
            out[r][: len(mine[r])] = [to.get(x, x) for x in mine[r]]
    per = s["k"].shape[3] // PAGE
    for name in ("k", "v", "k_scale", "v_scale"):
        n = PAGE if name in "kv" else PAGE // BLOCK
        for a, b in moves:
            s[name][:, b // per, :, b % per * n : (b % per + 1) * n] = s[name][:, a // per, :, a % per * n : (a % per + 1) * n]
    n = len(moves)
    moves = (moves + [(-1, -1)] * s["moves"].shape[0])[: s["moves"].shape[0]]
    whole_ = lambda x: np.array(x, np.int32)  # noqa: E731
    return (whole_(out), whole_(length), whole_(moves), whole_([n, used]), s["k"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn),
            s["k_scale"], s["v_scale"])


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "sample": _exact_sample}.get(case["op"], _exact_pages)(s)
