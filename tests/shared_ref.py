"""Plain definitions of attention over shared positions, of page tables that fork and compact, and of sampling with
settings per row (numpy and Python integers), which the tests hold the library to.  Written from
include/llm.h, sharing no code with the library (the exp of a weight is the oracle's)."""
import math

import numpy as np

import oracle

PAGE = 64


def attend_shared(r, q, length, groups, shared, count=None, table=None, scale=None, out=None):
    """As RefCache.attend of qcache_ref (r), for rows that take their positions below shared[i] from the places of
    the first row of their group: (result, mag, sens, flat)."""
    B, S, H, hd = q.shape
    g = H // r.kv
    scale = hd ** -0.5 if scale is None else scale
    res = np.zeros(q.shape) if out is None else out.copy()
    mag, sens, flat = np.zeros(q.shape), np.zeros((B, S, H, 1)), np.zeros((B, S, H, 1))
    for i in range(len(shared)):
        head = {}
        for b in range(groups[i], groups[i + 1]):
            n, L, sh = S if count is None else int(count[b]), int(length[b]), min(int(shared[i]), int(length[b]))
            if sh not in head:
                head[sh] = r.values(table, groups[i], sh)
            own = r.values(table, b, L - sh, first=sh)
            ks, vs = (np.concatenate(x, 1) for x in zip(head[sh], own))
            for t in range(n):
                end = L - n + t + 1
                res[b, t] = 0
                if end <= 0:
                    continue
                for j in range(r.kv):
                    x = q[b, t, j * g:(j + 1) * g]
                    k, v = ks[j, :end], vs[j, :end]
                    s = scale * (x @ k.T)
                    w = np.exp(s - s.max(-1, keepdims=True))
                    at = (b, t, slice(j * g, (j + 1) * g))
                    flat[at + (0,)] = np.abs(vs[j]).max(initial=0) * end / w.sum(-1)
                    w /= w.sum(-1, keepdims=True)
                    res[at] = w @ v
                    mag[at] = w @ np.abs(v)
                    sens[at + (0,)] = abs(scale) * np.abs(x).max(-1) * np.abs(k).sum(-1).max()
    return res, mag, sens, flat


def pages_of(n):
    return -(-n // PAGE)


def update(table, length, pages, parent=None, new=None):
    """(table, length, moves, [copies, pages in use]), or None where it cannot be done."""
    R, per = len(table), len(table[0])
    parent = list(range(R)) if parent is None else [int(p) for p in parent]
    if any(not -1 <= p < R for p in parent):
        return None
    new = [int(length[max(p, 0)]) for p in parent] if new is None else [int(n) for n in new]
    keep, mine = [0] * R, [[] for _ in range(R)]
    for r, p in enumerate(parent):
        if p < 0:
            new[r] = 0
            continue
        if not (0 <= length[p] <= per * PAGE and 0 <= new[r] <= per * PAGE):
            return None
        keep[r] = min(int(length[p]), new[r])
        mine[r] = [int(x) for x in table[p][:pages_of(keep[r])]]
        if any(not 0 <= x < pages for x in mine[r]):
            return None
    whole, opened = set(), {}
    for r in range(R):
        full = keep[r] // PAGE
        whole.update(mine[r][:full])
        if keep[r] % PAGE:
            opened.setdefault(mine[r][full], r)
    free = [x for x in range(pages) if x not in whole and x not in opened]
    moves, at = [], 0
    for r in range(R):
        copy = keep[r] % PAGE and (mine[r][-1] in whole or opened[mine[r][-1]] != r)
        need = bool(copy) + pages_of(new[r]) - len(mine[r])
        got = free[at:at + need]
        if len(got) < need:
            return None
        at += need
        if copy:
            moves.append([mine[r][-1], got[0]])
            mine[r][-1], got = got[0], got[1:]
        mine[r] += got
    return [m + [-1] * (per - len(m)) for m in mine], new, moves, [len(moves), len({x for m in mine for x in m})]


def compact(table, length, pages):
    R, per = len(table), len(table[0])
    if any(not 0 <= n <= per * PAGE for n in length):
        return None
    mine = [[int(x) for x in t[:pages_of(int(n))]] for t, n in zip(table, length)]
    held = {x for m in mine for x in m}
    if any(not 0 <= x < pages for x in held):
        return None
    used = len(held)
    moves = [list(m) for m in zip(sorted(x for x in held if x >= used), (x for x in range(used) if x not in held))]
    to = dict(moves)
    return [[to.get(x, x) for x in m] + [-1] * (per - len(m)) for m in mine], list(length), moves, [len(moves), used]


def sample(v, temp, k, p, min_p, u):
    """The id of one row of f32 logits."""
    v = np.asarray(v, np.float32)
    live = [i for i in range(len(v)) if not np.isnan(v[i]) and v[i] > -np.inf]
    if not live:
        return 0
    top = max(v[i] for i in live)
    if temp == 0:
        return next(i for i in live if v[i] == top)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        inverse = min(np.float32(1) / np.float32(temp), np.finfo(np.float32).max)
        far = {i: np.float32(0) if v[i] == top else np.float32(top - v[i]) * inverse for i in live}
    d = {i: math.floor(min(float(x), 30.0) * 2.0 ** 27) for i, x in far.items()}
    order = sorted(live, key=lambda i: (d[i], i))[:k]
    w = [int(np.rint(oracle.exp_s(-d[i] * 2.0 ** -27) * 2.0 ** 31)) for i in order]
    limit, cut, total = math.floor(float(p) * 2 ** 24) * sum(w) >> 24, 0, 0
    least = math.floor(float(min_p) * 2 ** 31)
    while cut < len(w) and (cut == 0 or total < limit) and w[cut] >= least:
        total += w[cut]
        cut += 1
    goal, run = math.floor(float(u) * 2 ** 24) * total >> 24, 0
    for i, x in zip(order, w):
        run += x
        if run > goal:
            return i
