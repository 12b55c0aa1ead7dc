"""The 8-bit key/value cache on the GPU (llm_qcache_write / read / attend) against the 64-bit definitions
of tests/qcache_ref.py.  Codes, scales and read values must be equal; attention is held to a bound
derived from its roundings (attend_tolerance)."""
import math

import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
from tests import qcache_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16}


def stream():
    return torch.cuda.current_stream().cuda_stream


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def make(rows, kv, cap, hd, garbage=None):
    """A library cache and its reference; with `garbage`, every code and scale starts as dead data
    (codes of every pattern, NaN's among them; scales that are powers of two)."""
    c = pkg.QCache.empty(rows, kv, cap, hd)
    r = ref.RefCache(rows, kv, cap, hd)
    if garbage is not None:
        rng = np.random.default_rng(garbage)
        for codes, scales, t, ts in ((r.k, r.ks, c.tensors[0], c.tensors[2]), (r.v, r.vs, c.tensors[1], c.tensors[3])):
            codes[:] = rng.integers(0, 256, codes.shape)
            scales[:] = 2.0 ** rng.integers(-20, 20, scales.shape)
            t.copy_(torch.from_numpy(codes))
            ts.copy_(torch.from_numpy(scales.astype(np.float32)))
    return c, r


def same(c, r):
    for t, a in zip(c.tensors, (r.k, r.v, r.ks, r.vs)):
        got = t.cpu().numpy()
        if a.dtype == np.uint8:
            assert np.array_equal(got, a), f"{int((got != a).sum())} of {a.size} codes differ"
        else:
            assert np.array_equal(got.astype(np.float64), a, equal_nan=True)


def rows_of(rng, shape, dtype, spread=1.0):
    x = torch.from_numpy((rng.standard_normal(shape) * spread).astype(np.float32)).to(T[dtype]).cuda()
    return x, x.double().cpu().numpy()


def pages(rng, B, cap, rows):
    per = cap // 64
    return rng.permutation(rows * per)[:B * per].reshape(B, per).astype(np.int32)


# ---- writing and reading ----

@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("hd,kv,dtype", [(16, 3, "f32"), (32, 1, "bf16"), (64, 2, "bf16"), (128, 2, "f32"), (256, 1, "bf16"),
                                         (64, 5, "f32"), (128, 1, "bf16")])
def test_write_and_read_equal_the_definition(hd, kv, dtype, paged):
    rng = np.random.default_rng(hd * 10 + kv + paged)
    rows, cap = 4, 192
    c, r = make(rows, kv, cap, hd, garbage=hd)
    table = pages(rng, rows, cap, rows) if paged else None
    dt = None if table is None else i32(table)
    # chunks that end and start inside blocks and pages, with rows of no tokens, growing values (so
    # that kept tokens are rounded again) and a rewind
    at = np.array([0, 5, 16, 63])
    for step, (S, spread) in enumerate([(1, 0.1), (7, 1.0), (16, 30.0), (37, 0.01), (1, 1e4), (64, 2.0)]):
        count = np.minimum(rng.integers(0, S + 1, rows), cap - at)
        count[step % rows] = min(S, cap - at[step % rows])
        k, kn = rows_of(rng, (rows, S, kv, hd), dtype, spread)
        v, vn = rows_of(rng, (rows, S, kv, hd), dtype, spread / 3)
        c.write(k, v, i32(at), count=i32(count), table=dt, stream=stream())
        r.write(kn, vn, at, count, table)
        same(c, r)
        at = at + count
        if step == 3:
            at = np.maximum(at - 9, 0)
    for S in (1, 50):
        pos = np.array([3, 0, 40, 21])
        count = np.array([S, S // 2, 0, S])
        ko, vo = (torch.full((rows, S, kv, hd), 7.0, dtype=T[dtype], device="cuda") for _ in range(2))
        c.read(i32(pos), ko, vo, count=i32(count), table=dt, stream=stream())
        for b in range(rows):
            kr, vr = r.values(table, b, count[b], pos[b])
            for got, want in ((ko, kr), (vo, vr)):
                g = got[b].double().cpu().numpy()
                assert np.array_equal(g[:count[b]], want.swapaxes(0, 1), equal_nan=True)
                assert (g[count[b]:] == 7.0).all()  # rows behind the last token stay as they were


def test_write_one_token_at_a_time_and_at_once_agree_within_a_rounding():
    rng = np.random.default_rng(3)
    kv, hd, n = 2, 64, 50
    k, kn = rows_of(rng, (1, n, kv, hd), "f32")
    one, r1 = make(1, kv, 64, hd)
    for i in range(n):
        one.write(k[:, i:i + 1], k[:, i:i + 1], i32([i]), stream=stream())
        r1.write(kn[:, i:i + 1], kn[:, i:i + 1], [i])
    same(one, r1)
    both, _ = make(1, kv, 64, hd)
    both.write(k, k, i32([0]), stream=stream())
    # the last scale is the same power of two; a value rounded twice is off only where the first
    # scale's code became subnormal: by half a step of 2^-9 scale at most
    for a, b, s in ((one.tensors[0], both.tensors[0], both.tensors[2]),):
        assert torch.equal(one.tensors[2][..., :3], both.tensors[2][..., :3])
        x, y = (t.view(torch.float8_e4m3fn).float() for t in (a, b))
        assert ((x - y).abs() <= 2.0 ** -9).all()


def test_write_takes_slices_of_wider_rows():
    rng = np.random.default_rng(4)
    B, S, kv, hd = 2, 5, 2, 32
    wide, wn = rows_of(rng, (B, S, 3 * kv * hd), "bf16")
    c, r = make(B, kv, 64, hd)
    c.write(wide[..., kv * hd:2 * kv * hd], wide[..., 2 * kv * hd:], i32([1, 30]), stream=stream())
    r.write(wn[..., kv * hd:2 * kv * hd].reshape(B, S, kv, hd), wn[..., 2 * kv * hd:].reshape(B, S, kv, hd), [1, 30])
    same(c, r)


def test_values_that_are_not_finite_and_extreme_ones():
    kv, hd = 1, 64
    c, r = make(1, kv, 128, hd)
    k = np.zeros((1, 96, kv, hd), np.float32)
    k[0, :16] = 3.4e38
    k[0, 16:32] = 1e-42                       # subnormal f32 (the scale stops at 2^-126)
    k[0, 32:48, 0, 5] = np.nan
    k[0, 48:64, 0, 0] = -np.inf
    k[0, 64:80] = np.float32(448.0)           # exactly the largest code
    k[0, 80:96] = np.nextafter(np.float32(448.0), np.float32(1e9))
    t = torch.from_numpy(k).cuda()
    c.write(t, -t, i32([0]), stream=stream())
    with np.errstate(invalid="ignore"):
        r.write(k.astype(np.float64), -k.astype(np.float64), [0])
        same(c, r)
        # a block stays NaN while its first position is kept, and is whole again once it is not
        x = torch.ones(1, 1, kv, hd, device="cuda")
        for pos in (40, 33, 32):
            c.write(x, x, i32([pos]), stream=stream())
            r.write(np.ones((1, 1, kv, hd)), np.ones((1, 1, kv, hd)), [pos])
            same(c, r)
    assert torch.isfinite(c.tensors[2][0, 0, 2])


def test_bad_positions_counts_and_pages_are_reported_and_skipped():
    rng = np.random.default_rng(6)
    B, S, kv, hd, cap = 4, 3, 2, 64, 128
    k, kn = rows_of(rng, (B, S, kv, hd), "f32")
    good = np.array([3, 60, 100, 0])
    table = np.arange(B * 2, dtype=np.int32).reshape(B, 2)

    def run(pos, count=None, tab=None):
        c, r = make(B, kv, cap, hd, garbage=1)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.write(k, k, i32(pos), count=None if count is None else i32(count), table=None if tab is None else i32(tab),
                status=st, stream=stream())
        return c, r, int(st)

    for bad in (-1, cap - 2, cap, 1 << 30, -(1 << 31)):
        pos = good.copy()
        pos[1] = bad
        c, r, st = run(pos)
        assert st == pkg.LLM_ERR_POS_RANGE
        r.write(kn, kn, good, np.array([S, 0, S, S]))
        same(c, r)
    for bad in (-1, S + 1):
        c, r, st = run(good, [S, bad, 1, S])
        assert st == pkg.LLM_ERR_ARG
        r.write(kn, kn, good, np.array([S, 0, 1, S]))
        same(c, r)
    for bad in (-1, B * 2, 1 << 30):
        tab = table.copy()
        tab[1, 0] = bad                       # row 1's tokens 60..62 lie in its first page
        c, r, st = run(good, None, tab)
        assert st == pkg.LLM_ERR_ARG
        r.write(kn, kn, good, np.array([S, 0, S, S]), table)
        same(c, r)
    c, r, st = run(good, [S, 0, 1, S], table)
    assert st == 0
    # reading: the rows that are out of range stay as they were
    out = torch.full((B, S, kv, hd), 5.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.read(i32([0, cap - 1, -4, 2]), out, out.clone(), status=st, stream=stream())
    assert int(st) == pkg.LLM_ERR_POS_RANGE and (out[1:3] == 5.0).all()


# ---- attention ----

def attend_tolerance(dtype, hd, want, mag, sens, flat):
    """|error| of an output, from the roundings of the operator.

    Scores: a query enters to 2^-19 of its largest element (f32) or 2^-21 (bf16 queries), the hd
    products are summed in f32 and a few more f32 roundings follow (scales, the exponent's argument):
    |ds| <= sens * (2^-19 + (hd + 32) 2^-24).  A weight and the sum of weights each move by
    exp(ds) - 1: together 2.2 ds.  A weight enters the product over the values rounded to at least 16
    (f32) or 8 (bf16) significant bits, but never finer than 2^-22 (2^-14) of the largest weight times
    the largest value scale; codes reach twice the largest value under it: 2 flat of that.  The sum
    itself is f32: under 2^-20 of mag for the lengths here.  A bf16 output is off by half a step, 2^-8."""
    ds = sens * (2.0 ** -19 + (hd + 32) * 2.0 ** -24)
    if dtype == "f32":
        return mag * (2.2 * ds + 2.0 ** -16 + 2.0 ** -20) + 2 * flat * 2.0 ** -22 + 1e-37
    return mag * (2.2 * ds + 2.0 ** -8 + 2.0 ** -20) + 2 * flat * 2.0 ** -14 + np.abs(want) * 2.0 ** -8 + 1e-37


def check_attend(c, r, rng, B, S, g, dtype, length, count=None, table=None, scale=None, spread=1.0, ws=None):
    hd = r.hd
    q, qn = rows_of(rng, (B, S, r.kv * g, hd), dtype, spread)
    out = torch.full_like(q, 9.0)
    ws = c.workspace(g, B, S) if ws is None else ws
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.attend(q, i32(length), out, ws, count=None if count is None else i32(count),
             table=None if table is None else i32(table), scale=scale, status=st, stream=stream())
    want, mag, sens, flat = r.attend(qn, length, count, table, scale, out=np.full(q.shape, 9.0))
    got = out.double().cpu().numpy()
    assert int(st) == 0
    err, tol = np.abs(got - want), attend_tolerance(dtype, hd, want, mag, sens, flat)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}, "
                           f"worst {float(np.nanmax(err / tol)):.3g} of the tolerance, largest {float(np.nanmax(err)):.3g}")
    return out


def fill(c, r, rng, n, table=None, spread=1.0):
    """n positions of every row of the call written in odd chunks."""
    B = r.rows if table is None else len(table)
    for lo, hi in ((0, n // 3), (n // 3, n)):
        if hi > lo:
            k, kn = rows_of(rng, (B, hi - lo, r.kv, r.hd), "f32", spread)
            v, vn = rows_of(rng, (B, hi - lo, r.kv, r.hd), "f32")
            c.write(k, v, i32([lo] * B), table=None if table is None else i32(table), stream=stream())
            r.write(kn, vn, [lo] * B, None, table)


SHAPES = [(16, 3, 2), (32, 2, 5), (64, 2, 1), (64, 3, 3), (64, 1, 16), (128, 2, 4), (128, 1, 8), (128, 3, 1), (128, 1, 7),
          (256, 2, 2), (64, 2, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,kv,g", SHAPES)
def test_attend_lengths_at_every_edge(hd, kv, g, dtype):
    rng = np.random.default_rng(hd + 100 * g)
    rows, cap = 14, 320
    c, r = make(rows, kv, cap, hd, garbage=7)
    fill(c, r, rng, 300)
    length = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 257, 300]
    check_attend(c, r, rng, rows, 1, g, dtype, length)
    # several tokens per row, some of them before the row's first position, padded rows among them
    check_attend(c, r, rng, rows, 5, g, dtype, length, count=[5, 5, 5, 0, 1, 2, 3, 4, 5, 5, 0, 5, 1, 5])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,kv,g,S", [(64, 2, 2, 1), (128, 2, 4, 3), (128, 1, 1, 40), (64, 1, 3, 75), (32, 1, 2, 4)])
def test_attend_through_scattered_pages(hd, kv, g, S, dtype):
    rng = np.random.default_rng(hd + S)
    rows, cap, B = 5, 256, 4
    c, r = make(rows, kv, cap, hd, garbage=8)
    table = pages(rng, B, cap, rows)
    fill(c, r, rng, 200, table)
    length = [200, 129, 64, 97]
    # pages behind a row's length are not looked at
    view = table.copy()
    for b, n in enumerate(length):
        view[b, -(-n // 64):] = [-1, 1 << 30, rows * 4][b % 3]
    check_attend(c, r, rng, B, S, g, dtype, length, table=view)
    # rows that share the same pages
    check_attend(c, r, rng, B, S, g, dtype, [200, 150, 200, 101], table=table[[0, 0, 1, 0]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_long_rows_many_parts(dtype):
    rng = np.random.default_rng(11)
    c, r = make(2, 2, 5008, 128, garbage=9)
    fill(c, r, rng, 5001)
    ws = c.workspace(4, 2, 2)
    for length in ([5001, 3], [4097, 4999], [1, 2], [2048, 5000]):  # one workspace, used again and again
        check_attend(c, r, rng, 2, 2, 4, dtype, length, ws=ws)


@pytest.mark.parametrize("hd", [16, 64, 128])
@pytest.mark.parametrize("rows,kv,cap", [(1, 1, 16), (1, 1, 48), (3, 1, 80), (1, 2, 112)])
def test_caches_smaller_than_a_tile_and_with_ragged_ends(hd, rows, kv, cap):
    # tiles of 128 positions reach past the row, the head and the whole cache
    rng = np.random.default_rng(hd + cap)
    c, r = make(rows, kv, cap, hd, garbage=5)
    fill(c, r, rng, cap)
    for dtype in ("f32", "bf16"):
        check_attend(c, r, rng, rows, 1, 2, dtype, [cap - b for b in range(rows)])
        check_attend(c, r, rng, rows, 3, 2, dtype, [1 + b for b in range(rows)])


def test_attend_takes_slices_of_wider_rows_and_many_rows():
    # queries as slices of fused rows; more rows than lanes of the warp that shares the work out
    rng = np.random.default_rng(21)
    B, kv, g, hd, cap = 70, 2, 3, 64, 144
    c, r = make(B, kv, cap, hd, garbage=6)
    fill(c, r, rng, 140)
    wide, wn = rows_of(rng, (B, 2, (kv * g + 2 * kv) * hd), "f32")
    n = kv * g * hd
    out = torch.full((B, 2, n + 8), 9.0, device="cuda")
    length = [(b * 29) % 141 for b in range(B)]
    c.attend(wide[..., :n], i32(length), out[..., 8:], c.workspace(g, B, 2), stream=stream())
    want, mag, sens, flat = r.attend(wn[..., :n].reshape(B, 2, kv * g, hd), length)
    got = out[..., 8:].reshape(B, 2, kv * g, hd).double().cpu().numpy()
    assert (np.abs(got - want) <= attend_tolerance("f32", hd, want, mag, sens, flat)).all()
    assert (out[..., :8] == 9.0).all()


def test_attend_scores_that_rise_along_the_row_and_other_scales():
    # running maxima move at every tile; the scale argument is used as given (zero and negative too)
    rng = np.random.default_rng(12)
    kv, hd, n = 1, 128, 1000
    c, r = make(1, kv, 1008, hd)
    base = rng.standard_normal((1, 1, kv, hd)).astype(np.float32)
    k = (base * np.linspace(0.01, 4.0, n)[None, :, None, None]).astype(np.float32)
    v, vn = rows_of(rng, (1, n, kv, hd), "f32")
    c.write(torch.from_numpy(k).cuda(), v, i32([0]), stream=stream())
    r.write(k.astype(np.float64), vn, [0])
    for scale in (None, 0.0, -0.05, 0.3):
        check_attend(c, r, rng, 1, 2, 4, "f32", [n], scale=scale, spread=2.0)


def test_attend_value_scales_far_apart():
    # a block of values 2^12 larger than the rest at a small weight, and blocks of zeros
    rng = np.random.default_rng(13)
    kv, hd, n = 1, 64, 400
    c, r = make(1, kv, 400, hd)
    k, kn = rows_of(rng, (1, n, kv, hd), "f32")
    v, _ = rows_of(rng, (1, n, kv, hd), "f32")
    v[:, 160:176] *= 4096.0
    v[:, 0:48] = 0.0
    vn = v.double().cpu().numpy()
    c.write(k, v, i32([0]), stream=stream())
    r.write(kn, vn, [0])
    for length in ([n], [48], [177]):
        check_attend(c, r, rng, 1, 3, 4, "f32", length)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_heavy_position_and_a_long_flat_tail(dtype):
    # position 0 weighs 2^15 to 2^19 times one of the 4095 others, which share a score and have values of
    # one sign: whatever is lost of their weights adds up.  320 (row, kv head) pairs of 32 tiles keep a
    # CTA on one of them for most of its tiles.
    B, kv, g, hd, n = 40, 8, 4, 64, 4096
    c = pkg.QCache.empty(B, kv, n, hd)
    gen = torch.Generator(device="cuda").manual_seed(15)
    k = torch.zeros(B, n, kv, hd, device="cuda")
    k[..., 0] = 1.0
    k[:, 0, :, 0] = 2.0
    v = 0.5 + 0.5 * torch.rand(B, n, kv, hd, device="cuda", generator=gen)
    c.write(k, v, i32([0] * B), stream=stream())
    q = torch.zeros(B, 1, kv * g, hd, device="cuda")
    q[..., 0] = 15.0 + 4.0 * torch.rand(B, 1, kv * g, device="cuda", generator=gen)
    q = (q * math.log(2.0) * hd ** 0.5).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    out = torch.empty_like(q)
    c.attend(q, i32([n] * B), out, c.workspace(g, B, 1), stream=stream())
    c.read(i32([0] * B), k, v, stream=stream())
    for b in range(0, B, 13):
        x = q[b, 0].double().reshape(kv, g, hd)
        kd, vd = k[b].double().transpose(0, 1), v[b].double().transpose(0, 1)   # [kv][n][hd]
        w = torch.softmax(hd ** -0.5 * x @ kd.transpose(1, 2), -1)
        want = (w @ vd).cpu().numpy()
        top = w.amax(-1, keepdim=True).cpu().numpy()
        sens = (hd ** -0.5 * x.abs().amax(-1, keepdim=True) * kd.abs().sum(-1).max()).cpu().numpy()
        # as attend_tolerance (all values are positive: mag is the result), but for the weights' last
        # digit: 2^-27 (bf16 2^-20) of the largest weight, times values of up to 2 under their scale, n times
        ds = sens * (2.0 ** -19 + (hd + 32) * 2.0 ** -24)
        last, digits, half = (2.0 ** -27, 2.0 ** -16, 0.0) if dtype == "f32" else (2.0 ** -20, 2.0 ** -8, 2.0 ** -8)
        tol = want * (2.2 * ds + digits + 2.0 ** -20 + half) + 2 * n * top * last
        err = np.abs(out[b, 0].double().reshape(kv, g, hd).cpu().numpy() - want)
        assert (err <= tol).all(), f"worst {float((err / tol).max()):.3g} of the tolerance"


@pytest.mark.parametrize("hd,kv,g", [(128, 2, 4), (256, 2, 2)])
def test_pages_beyond_32_bit_offsets(hd, kv, g):
    # codes of 8.6 GB each, written and attended to through pages at both ends; the reference holds those alone
    rng = np.random.default_rng(22)
    per = (1 << 33) // (kv * hd * 64) + 1
    c = pkg.QCache.empty(1, kv, per * 64, hd)
    r = ref.RefCache(1, kv, 6 * 64, hd)
    far = np.array([[per - 1, 0, per - 2], [1, per - 3, per // 2 + 1]], np.int32)
    near = np.arange(6, dtype=np.int32).reshape(2, 3)
    k, kn = rows_of(rng, (2, 150, kv, hd), "f32")
    v, vn = rows_of(rng, (2, 150, kv, hd), "f32")
    c.write(k, v, i32([0, 7]), table=i32(far), stream=stream())
    r.write(kn, vn, [0, 7], None, near)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    c.read(i32([0, 7]), kb, vb, table=i32(far), stream=stream())
    for b, n in ((0, 0), (1, 7)):
        kk, vv = r.values(near, b, 150, n)
        assert np.array_equal(kb[b].double().cpu().numpy(), kk.transpose(1, 0, 2))
        assert np.array_equal(vb[b].double().cpu().numpy(), vv.transpose(1, 0, 2))
    for dtype in ("f32", "bf16"):
        q, qn = rows_of(rng, (2, 3, kv * g, hd), dtype)
        out = torch.empty_like(q)
        c.attend(q, i32([150, 157]), out, c.workspace(g, 2, 3), table=i32(far), stream=stream())
        want, mag, sens, flat = r.attend(qn, [150, 157], table=near)
        assert (np.abs(out.double().cpu().numpy() - want) <= attend_tolerance(dtype, hd, want, mag, sens, flat)).all()


def test_one_row_of_more_than_2_to_the_25_positions():
    # zeros but for the last 16 positions, which weigh about as much as all the others together
    rng = np.random.default_rng(23)
    hd, g, n = 128, 4, (1 << 25) + 1000
    c = pkg.QCache.empty(1, 1, (n + 15) // 16 * 16, hd)
    v, vn = rows_of(rng, (1, 16, 1, hd), "f32")
    k = torch.ones(1, 16, 1, hd, device="cuda")
    c.write(k, v, i32([n - 16]), stream=stream())
    c.read(i32([n - 16]), k, v, stream=stream())
    q = torch.full((1, 1, g, hd), 15.0 / hd ** 0.5, device="cuda")
    out = torch.empty_like(q)
    c.attend(q, i32([n]), out, c.workspace(g, 1, 1), stream=stream())
    s = hd ** -0.5 * float(q[0, 0, 0].double().sum())
    vd = v[0, :, 0].double().cpu().numpy()
    total = n - 16 + 16 * math.exp(s)
    want, mag = math.exp(s) * vd.sum(0) / total, math.exp(s) * np.abs(vd).sum(0) / total
    # zero values lose nothing with their weights, so 16 positions count for flat; a lane adds up at most
    # 2^9 weights of a CTA's tiles in f32, each addition off by half a step
    tol = attend_tolerance("f32", hd, want, mag, s, np.abs(vd).max() * 16 * math.exp(s) / total) + mag * 2.0 ** -15
    assert (np.abs(out[0, 0].double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("hd", [32, 64, 128])
def test_calls_without_any_visible_position(hd):
    kv, g, B = 2, 4, 3
    c, r = make(B, kv, 64, hd, garbage=2)
    ws = c.workspace(g, B, 2)
    q = torch.ones(B, 2, kv * g, hd, device="cuda")
    for length, count, want in (([0] * B, None, 0.0), ([0] * B, [0] * B, 9.0), ([40, 64, 1], [0] * B, 9.0)):
        out = torch.full_like(q, 9.0)
        c.attend(q, i32(length), out, ws, count=None if count is None else i32(count), stream=stream())
        assert (out == want).all()
    x = torch.ones(B, 2, kv, hd, device="cuda")
    c.write(x, x, i32([0, 63, 64]), count=i32([0] * B), stream=stream())   # nothing to write, anywhere
    same(c, r)
    rng = np.random.default_rng(24)                                        # the workspace is as it was
    fill(c, r, rng, 64)
    check_attend(c, r, rng, B, 2, g, "f32", [64, 1, 33], ws=ws)


def test_nan_reaches_only_the_tokens_that_see_it():
    rng = np.random.default_rng(14)
    for hd, g in ((128, 4), (64, 1), (32, 2)):
        kv, n = 2, 160
        c, r = make(1, kv, 192, hd)
        fill(c, r, rng, n)
        bad = torch.zeros(1, 1, kv, hd, device="cuda")
        bad[0, 0, 1, 3] = float("nan")        # head 1 of the token at position 160, alone in its block
        zero = torch.zeros_like(bad)
        for k, v in ((bad, zero), (zero, bad)):
            c.write(k, v, i32([160]), stream=stream())
            q, _ = rows_of(rng, (1, 3, kv * g, hd), "f32")
            out = torch.zeros_like(q)
            c.attend(q, i32([161]), out, c.workspace(g, 1, 3), stream=stream())
            assert torch.isfinite(out[0, :2]).all()          # positions ..158 and ..159
            assert torch.isfinite(out[0, 2, :g]).all()       # head 0
            assert torch.isnan(out[0, 2, g:]).all()


def test_bad_lengths_and_pages_leave_the_other_rows_right():
    rng = np.random.default_rng(15)
    for hd in (128, 32):
        kv, g, cap, B = 2, 4, 256, 4
        c, r = make(B, kv, cap, hd, garbage=3)
        table = np.arange(B * 4, dtype=np.int32).reshape(B, 4)
        fill(c, r, rng, 250)
        q, qn = rows_of(rng, (B, 2, kv * g, hd), "f32")

        def run(length, tab=None, count=None):
            out = torch.full_like(q, 9.0)
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            c.attend(q, i32(length), out, c.workspace(g, B, 2), table=None if tab is None else i32(tab),
                     count=None if count is None else i32(count), status=st, stream=stream())
            return out.double().cpu().numpy(), int(st)

        want, mag, sens, flat = r.attend(qn, [250, 100, 64, 3])
        tol = attend_tolerance("f32", hd, want, mag, sens, flat)
        for bad in (-1, cap + 1, 1 << 30, -(1 << 31)):
            got, st = run([250, bad, 64, 3])
            assert st == pkg.LLM_ERR_POS_RANGE and (got[1] == 0).all()
            assert (np.abs(got - want)[[0, 2, 3]] <= tol[[0, 2, 3]]).all()
        got, st = run([250, 100, 64, 3], count=[2, 3, 2, 2])
        assert st == pkg.LLM_ERR_ARG and (got[1] == 9).all()
        # a page outside the pool: its positions are not seen
        for bad in (-1, B * 4, 1 << 30):
            tab = table.copy()
            tab[1, 0] = bad
            got, st = run([250, 100, 64, 3], tab)
            assert st == pkg.LLM_ERR_ARG
            assert (np.abs(got - want)[[0, 2, 3]] <= tol[[0, 2, 3]]).all()
            hole = ref.RefCache(1, kv, cap, hd)
            hole.k[0], hole.v[0], hole.ks[0], hole.vs[0] = r.k[1], r.v[1], r.ks[1], r.vs[1]
            for i in range(2):                # positions 64 .. of row 1 alone
                kk, vv = hole.values(None, 0, 99 + i - 64, 64)
                for j in range(kv):
                    s = hd ** -0.5 * qn[1, i, j * g:(j + 1) * g] @ kk[j].T
                    w = np.exp(s - s.max(-1, keepdims=True))
                    o = w @ vv[j] / w.sum(-1, keepdims=True)
                    assert (np.abs(got[1, i, j * g:(j + 1) * g] - o) <= 2 * tol[1].max()).all()


def test_captured_calls_replay_with_new_lengths_and_streams_of_their_own():
    rng = np.random.default_rng(16)
    kv, g, hd, B = 2, 4, 128, 3
    c, r = make(B, kv, 512, hd)
    fill(c, r, rng, 500)
    q, qn = rows_of(rng, (B, 2, kv * g, hd), "f32")
    side = torch.cuda.Stream()
    length = i32([10, 20, 30])
    new, newn = rows_of(rng, (B, 2, kv, hd), "f32")
    pos = i32([8, 18, 28])
    outs, spaces, graphs = [], [], []
    for _ in range(2):                        # two graphs, each with its own workspace
        outs.append(torch.zeros_like(q))
        spaces.append(c.workspace(g, B, 2))
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            s = torch.cuda.current_stream().cuda_stream
            c.write(new, new, pos, stream=s)
            c.attend(q, length, outs[-1], spaces[-1], stream=s)
        graphs.append(gr)
    for want_len in ([10, 20, 30], [500, 2, 257], [129, 384, 65]):
        length.copy_(i32(want_len))
        pos.copy_(i32([n - 2 for n in want_len]))
        r.write(newn, newn, [n - 2 for n in want_len])
        torch.cuda.synchronize()
        graphs[0].replay()                    # (the second write changes nothing: same values, same place)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        want, mag, sens, flat = r.attend(qn, want_len)
        for o in outs:
            assert (np.abs(o.double().cpu().numpy() - want) <= attend_tolerance("f32", hd, want, mag, sens, flat)).all()
        assert torch.equal(outs[0], outs[1])  # the same bits, whatever else ran
        same(c, r)


def test_wrappers_refuse_shapes_types_and_devices_that_do_not_fit():
    c = pkg.QCache.empty(2, 2, 64, 64)
    x = torch.zeros(2, 3, 2, 64, device="cuda")
    pos = i32([0, 0])
    q = torch.zeros(2, 1, 8, 64, device="cuda")
    ws = c.workspace(4, 2, 1)
    for f in (lambda: c.write(x, x.bfloat16(), pos), lambda: c.write(x.half(), x.half(), pos), lambda: c.write(x, x[:, :2], pos),
              lambda: c.write(x, x.cpu(), pos), lambda: c.write(x, x, pos.long()), lambda: c.write(x, x, i32([0])),
              lambda: c.write(x, x, None), lambda: c.write(x, x, pos, count=i32([1])), lambda: c.write(x, x, pos, table=i32([0, 1])),
              lambda: c.write(x.transpose(2, 3), x, pos), lambda: c.write(x[..., :32], x[..., :32], pos),
              lambda: c.attend(q, pos, q.bfloat16(), ws), lambda: c.attend(q, pos, q[:, :, :4], ws),
              lambda: c.attend(q[:, :, :3], pos, q[:, :, :3].clone(), ws), lambda: c.attend(q, pos.cpu(), q.clone(), ws),
              lambda: c.workspace(17, 1, 1), lambda: c.workspace(4, 0, 1)):
        with pytest.raises(pkg.LlmError):
            f()
    need = c.workspace(4, 2, 1).numel()
    if need > 16:
        with pytest.raises(pkg.LlmError):
            c.attend(q, pos, q.clone(), ws[:need - 16])
