"""Plain 64-bit definitions of the 8-bit cache operators and of draft verification (numpy), which the
tests hold the library to.  Written from include/llm.h, sharing no code with the library."""
import numpy as np

BLOCK, PAGE = 16, 64


def e4m3_table():
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v[(code & 127) == 127] = np.nan
    return np.where(code & 128, -v, v)


VALUE = e4m3_table()


def encode(x):
    """Codes of values |x| <= 448 (float64), nearest with ties to the even code; NaN is 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    pos = VALUE[:127]
    hi = np.searchsorted(pos, a).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    pick = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(x), 0x7f, pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def need_scale(x):
    """The least power of two >= 2^-126 with max |x| / s <= 448; NaN where a value is not finite."""
    if not np.isfinite(x).all():
        return np.nan
    top = float(np.max(np.abs(x), initial=0.0))
    s = 2.0 ** -126
    while top / s > 448.0:
        s *= 2.0
    return s


class RefCache:
    def __init__(self, rows, kv, cap, hd):
        self.k, self.v = (np.zeros((rows, kv, cap, hd), np.uint8) for _ in range(2))
        self.ks, self.vs = (np.zeros((rows, kv, cap // BLOCK)) for _ in range(2))
        self.rows, self.kv, self.cap, self.hd = rows, kv, cap, hd

    def slot(self, table, b, pos):
        if table is None:
            return b, pos
        page, per = int(table[b][pos // PAGE]), self.cap // PAGE
        return page // per, page % per * PAGE + pos % PAGE

    def write(self, k, v, pos, count=None, table=None):
        """k, v [B, S, kv, hd] float64 holding the f32 or bf16 values."""
        B, S = k.shape[:2]
        for b in range(B):
            n = S if count is None else int(count[b])
            p = int(pos[b])
            end = p + n
            at = p
            while at < end:
                stop = min(end, at // BLOCK * BLOCK + BLOCK)
                r, q = self.slot(table, b, at)
                t0, blk = q % BLOCK, q // BLOCK
                for h in range(self.kv):
                    for codes, scales, x in ((self.k, self.ks, k), (self.v, self.vs, v)):
                        new = x[b, at - p:stop - p, h]
                        s = need_scale(new)
                        old = scales[r, h, blk]
                        if t0 > 0:
                            s = np.nan if np.isnan(s) or np.isnan(old) else max(s, old)
                            if not np.isnan(s) and s > old:
                                kept = codes[r, h, q - t0:q]
                                codes[r, h, q - t0:q] = encode(VALUE[kept] * (old / s))
                        codes[r, h, q:q + stop - at] = 0 if np.isnan(s) else encode(new / s)
                        scales[r, h, blk] = s
                at = stop

    def values(self, table, b, n, first=0):
        """Keys and values [kv, n, hd] of positions first .. first + n - 1 of row b."""
        ks, vs = np.zeros((self.kv, n, self.hd)), np.zeros((self.kv, n, self.hd))
        for i in range(n):
            r, q = self.slot(table, b, first + i)
            ks[:, i] = VALUE[self.k[r, :, q]] * self.ks[r, :, q // BLOCK, None]
            vs[:, i] = VALUE[self.v[r, :, q]] * self.vs[r, :, q // BLOCK, None]
        return ks, vs

    def attend(self, q, length, count=None, table=None, scale=None, out=None):
        """q [B, S, H, hd] float64 -> (result, mag, sens, flat), the last three for tolerances: per element
        sum_t w_t |v_t| / sum w; per head the largest change of a score when every |q_d| changes by
        max |q|; and max |v| * positions / sum of weights relative to the largest weight."""
        B, S, H, hd = q.shape
        g = H // self.kv
        scale = hd ** -0.5 if scale is None else scale
        res = np.zeros(q.shape) if out is None else out.copy()
        mag, sens, flat = np.zeros(q.shape), np.zeros((B, S, H, 1)), np.zeros((B, S, H, 1))
        for b in range(B):
            n = S if count is None else int(count[b])
            ks, vs = self.values(table, b, int(length[b]))
            for i in range(n):
                end = int(length[b]) - n + i + 1
                res[b, i] = 0
                if end <= 0:
                    continue
                for j in range(self.kv):
                    x = q[b, i, j * g:(j + 1) * g]
                    k, v = ks[j, :end], vs[j, :end]
                    s = scale * (x @ k.T)
                    w = np.exp(s - s.max(-1, keepdims=True))
                    flat[b, i, j * g:(j + 1) * g, 0] = np.abs(vs[j]).max(initial=0) * end / w.sum(-1)
                    w /= w.sum(-1, keepdims=True)
                    res[b, i, j * g:(j + 1) * g] = w @ v
                    mag[b, i, j * g:(j + 1) * g] = w @ np.abs(v)
                    sens[b, i, j * g:(j + 1) * g, 0] = abs(scale) * np.abs(x).max(-1) * np.abs(k).sum(-1).max()
        return res, mag, sens, flat


def verify(p, q, drafts, count, u):
    """Kept drafts, the drawn token and the number kept of one row: p [S+1, V], q [S, V] or None."""
    S = len(drafts)
    n = S if count is None else min(max(int(count), 0), S)
    r = 0
    V = p.shape[1]
    while r < n:
        x = int(drafts[r])
        if not 0 <= x < V:
            break
        qx = 1.0 if q is None else float(q[r, x])
        if not float(u[r]) * qx < float(p[r, x]):
            break
        r += 1

    def units(w):
        w = np.where(w > 0, np.minimum(w, np.float32(1)), np.float32(0)).astype(np.float64)
        return [int(x) for x in np.floor(np.ldexp(w, 61))]

    w = p[r].copy()
    if r < n:
        if q is not None:
            w = (w - q[r]).astype(np.float32)
        elif 0 <= int(drafts[r]) < V:
            w[int(drafts[r])] = 0
    whole = units(w)
    if sum(whole) == 0:
        whole = units(p[r])
    total = sum(whole)
    last = 0
    if total:
        goal, run = int(np.floor(float(u[S]) * 2 ** 24)) * total >> 24, 0
        for last, x in enumerate(whole):
            run += x
            if run > goal:
                break
    return [int(x) for x in drafts[:r]] + [last] + [-1] * (S - r), r
