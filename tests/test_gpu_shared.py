"""Attention over shared positions (llm_qcache_attend_shared) on the GPU against the 64-bit definition of
tests/shared_ref.py, within a bound derived from its roundings."""
import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
from tests import qcache_ref, shared_ref
from tests.test_gpu_qcache import T, fill, i32, make, pages, rows_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def tolerance(dtype, hd, want, mag, sens):
    """|error| of an output.  A query enters to 2^-17 of its largest element (bf16: exact above 2^-10 of it, else off by
    2^-18 of it; f32: four e4m3 pieces leave 2^-17 of an element); hd products are summed in f32, and the score meets a few more f32
    roundings: |ds| <= sens (2^-17 + (hd + 32) 2^-24).  A weight and the sum of weights each move by exp(ds) - 1, together
    2.2 ds; the exponential is off by 2^-21; a weight enters as bf16 pieces, off by 2^-26 (f32: three) or 2^-17 (bf16:
    two) of itself; sums are f32: 2^-19 of the sum of magnitudes for the lengths here.  A bf16 output is
    off by half a step, 2^-8."""
    ds = sens * (2.0 ** -17 + (hd + 32) * 2.0 ** -24)
    digits = 2.0 ** -26 if dtype == "f32" else 2.0 ** -17
    return mag * (2.2 * ds + 2.0 ** -21 + digits + 2.0 ** -19) + (np.abs(want) * 2.0 ** -8 if dtype == "bf16" else 0) + 1e-37


def wide_table(r, B, table=None):
    """The rows' page table, or that of rows in place, with columns for 2^18 positions, which no row has."""
    per = r.k.shape[2] // 64
    table = np.arange(B)[:, None] * per + np.arange(per)[None] if table is None else np.asarray(table)
    return np.concatenate([table, np.full((B, 4096 - table.shape[1]), -1)], 1).astype(np.int32)


def check(c, r, rng, S, g, dtype, length, groups, shared, count=None, table=None, scale=None, spread=1.0, ws=None, status=0, want_with=None):
    B, hd = len(length), r.hd
    q, qn = rows_of(rng, (B, S, r.kv * g, hd), dtype, spread)
    out = torch.full_like(q, 9.0)
    ws = c.workspace_shared(g, B, S, len(shared)) if ws is None else ws
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.attend_shared(q, i32(length), i32(groups), i32(shared), out, ws, count=None if count is None else i32(count),
                    table=None if table is None else i32(table), scale=scale, status=st)
    outs = [out]
    if status == 0 and r.k.shape[2] % 64 == 0:
        # the same through a page table that has room for far more, which calls that read the shared positions once go by
        outs.append(torch.full_like(q, 9.0))
        t = wide_table(r, B) if table is None else wide_table(r, B, table)
        c.attend_shared(q, i32(length), i32(groups), i32(shared), outs[1], ws, count=None if count is None else i32(count),
                        table=i32(t), scale=scale, status=st)
    length, groups, shared = want_with or (length, groups, shared)
    want, mag, sens, _ = shared_ref.attend_shared(r, qn, length, groups, shared, count, table, scale, out=np.full(q.shape, 9.0))
    assert int(st) == status
    got = np.stack([x.double().cpu().numpy() for x in outs])
    err, tol = np.abs(got - want), tolerance(dtype, hd, want, mag, sens)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0].tolist()}, "
                           f"worst {float(np.nanmax(err / tol)):.3g} of the tolerance, largest {float(np.nanmax(err)):.3g}")
    return out


SHAPES = [(16, 2, 2), (32, 1, 5), (64, 2, 1), (64, 3, 3), (64, 1, 16), (128, 2, 4), (128, 1, 8), (128, 3, 1), (128, 1, 7), (256, 1, 2)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,kv,g", SHAPES)
def test_lengths_and_shared_parts_at_every_edge(hd, kv, g, dtype):
    # rows in place: the group's first row holds the shared positions, the others' own places below them hold dead data
    rng = np.random.default_rng(hd + g)
    rows, cap = 11, 320
    c, r = make(rows, kv, cap, hd, garbage=7)
    fill(c, r, rng, 300)
    length = [300, 65, 200, 129, 1, 64, 128, 130, 0, 257, 300]
    for groups, shared in (([0, 11], [64]), ([0, 11], [0]), ([0, 11], [129]), ([0, 3, 3, 10, 11], [63, 300, 128, 16]),
                           ([0, 11], [300]), (list(range(12)), [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 300])):
        check(c, r, rng, 1, g, dtype, length, groups, shared)
    check(c, r, rng, 5, g, dtype, length, [0, 4, 11], [130, 60], count=[5, 5, 0, 1, 5, 2, 3, 4, 5, 5, 1])
    check(c, r, rng, 3, g, dtype, length, [0, 11], [100])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,kv,g,S", [(64, 2, 2, 1), (128, 2, 4, 3), (128, 1, 1, 40), (64, 1, 3, 75), (128, 1, 8, 33), (32, 1, 2, 4)])
def test_pages_of_the_first_row_and_of_each_row(hd, kv, g, S, dtype):
    rng = np.random.default_rng(hd + S)
    rows, cap, B = 6, 256, 5
    c, r = make(rows, kv, cap, hd, garbage=8)
    table = pages(rng, B, cap, rows)
    fill(c, r, rng, 200, table)
    length = [200, 129, 80, 97, 193]
    groups, shared = [0, 2, 5], [129, 77]
    # pages behind a row's length, and whole pages of what the others of a group share, are not looked at
    view = table.copy()
    for b, n in enumerate(length):
        view[b, -(-n // 64):] = [-1, 1 << 30, rows * 4][b % 3]
    view[1, :2], view[3, :1], view[4, :1] = -5, 1 << 29, -1
    check(c, r, rng, S, g, dtype, length, groups, shared, table=view)
    # the same pages named by all: what the ordinary attention gives
    for b, lead, n in ((1, 0, 2), (3, 2, 1), (4, 2, 1)):
        table[b, :n] = table[lead, :n]
    q, _ = rows_of(rng, (B, S, kv * g, hd), dtype)
    a, b_ = torch.empty_like(q), torch.empty_like(q)
    c.attend(q, i32(length), a, c.workspace(g, B, S), table=i32(table))
    c.attend_shared(q, i32(length), i32(groups), i32([128, 64]), b_, c.workspace_shared(g, B, S, 2), table=i32(table))
    assert (a.float() - b_.float()).abs().max() <= (2e-2 if dtype == "bf16" else 2e-3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd", [64, 128])
def test_many_rows_and_long_parts(hd, dtype):
    # groups of more rows than a tile has columns, units cut over many CTAs, workspaces used again
    rng = np.random.default_rng(11)
    B, kv, g, cap = 70, 2, 4, 2048
    c, r = make(2, kv, cap, hd, garbage=9)
    table = np.zeros((B, 30), np.int32)
    fill(c, r, rng, 1920, np.arange(30, dtype=np.int32)[None])
    for b in range(B):
        table[b] = np.roll(np.arange(30), 0 if b in (0, 66) else b) if b else np.arange(30)
    ws = c.workspace_shared(g, B, 2, 3)
    for length in ([1900 - 3 * b for b in range(B)], [1500 + b % 5 for b in range(B)]):
        check(c, r, rng, 2, g, dtype, length, [0, 66, 67, 70], [1500, 3, 1200], table=table, ws=ws)


def test_slices_of_wider_rows_and_other_scales():
    rng = np.random.default_rng(21)
    B, kv, g, hd, cap = 9, 2, 3, 64, 144
    c, r = make(B, kv, cap, hd, garbage=6)
    fill(c, r, rng, 140)
    wide, wn = rows_of(rng, (B, 2, (kv * g + 2 * kv) * hd), "f32")
    n = kv * g * hd
    out = torch.full((B, 2, n + 8), 9.0, device="cuda")
    length = [140 - b for b in range(B)]
    c.attend_shared(wide[..., :n], i32(length), i32([0, B]), i32([100]), out[..., 8:], c.workspace_shared(g, B, 2, 1))
    want, mag, sens, _ = shared_ref.attend_shared(r, wn[..., :n].reshape(B, 2, kv * g, hd), length, [0, B], [100])
    got = out[..., 8:].reshape(B, 2, kv * g, hd).double().cpu().numpy()
    assert (np.abs(got - want) <= tolerance("f32", hd, want, mag, sens)).all()
    assert (out[..., :8] == 9.0).all()
    for scale in (0.0, -0.05, 0.3, 2.0):
        check(c, r, rng, 1, g, "f32", length, [0, B], [100], scale=scale, spread=2.0)


@pytest.mark.parametrize("wide", [False, True])
def test_bad_groups_shared_parts_lengths_and_pages(wide):
    rng = np.random.default_rng(15)
    for hd in (128, 64, 32):
        kv, g, cap, B = 2, 4, 256, 4
        c, r = make(B, kv, cap, hd, garbage=3)
        fill(c, r, rng, 256)
        t, most = (wide_table(r, B), 1 << 18) if wide else (None, cap)
        L = [256, 200, 70, 130]
        # bounds that do not ascend from 0 to B: no row shares
        for groups in ([0, 3], [1, 4], [0, 5], [0, 3, 2, 4], [0, 4, 4, 3], [-1, 4], [0, 1 << 30, 4], [0, -5, 4]):
            n = len(groups) - 1
            check(c, r, rng, 1, g, "f32", L, groups, [64] * n, status=pkg.LLM_ERR_ARG, want_with=(L, [0, 4], [0]) if n == 1 else (L, [0, 4], [0]), table=t)
        # shared parts out of range: the rows of that group share nothing
        for bad in (-1, most + 1, 1 << 30):
            check(c, r, rng, 1, g, "f32", L, [0, 2, 4], [bad, 60], status=pkg.LLM_ERR_POS_RANGE, want_with=(L, [0, 2, 4], [0, 60]), table=t)
        # lengths and counts out of range: those rows are empty
        check(c, r, rng, 1, g, "f32", [256, -1, most + 1, 130], [0, 4], [100], status=pkg.LLM_ERR_POS_RANGE,
              want_with=([256, 0, 0, 130], [0, 4], [100]), table=t)
        # a page of the shared part outside the pool is unseen by all, one of a row's own by that row
        table = wide_table(r, B) if wide else np.arange(B * 4, dtype=np.int32).reshape(B, 4)
        for b, i in ((0, 1), (3, 1)):
            bad = table.copy()
            bad[b, i] = B * 4
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            q, _ = rows_of(rng, (B, 1, kv * g, hd), "f32")
            out, fine = torch.empty_like(q), torch.empty_like(q)
            ws = c.workspace_shared(g, B, 1, 1)
            c.attend_shared(q, i32(L), i32([0, 4]), i32([100]), out, ws, table=i32(bad), status=st)
            c.attend_shared(q, i32(L), i32([0, 4]), i32([100]), fine, ws, table=i32(table))
            assert int(st) == pkg.LLM_ERR_ARG and torch.isfinite(out).all()
            same_rows = [x for x in range(B) if torch.allclose(out[x], fine[x], atol=1e-5)]
            assert same_rows == ([] if b == 0 else [0, 1, 2])


@pytest.mark.parametrize("hd", [32, 64, 128])
def test_shared_parts_out_of_range_are_reported_whoever_has_them(hd):
    # a group without rows, one of empty rows, one whose rows have no tokens in the call; each way a call can go
    kv, g, B = 2, 4, 4
    c, r = make(B, kv, 128, hd, garbage=2)
    fill(c, r, np.random.default_rng(16), 100)
    q = torch.ones(B, 1, kv * g, hd, device="cuda")
    for table in (None, wide_table(r, B)):
        for groups, shared, length, count in (([0, 2, 2, 4], [10, -1, 20], [100] * 4, None), ([0, 2, 4, 4], [10, 20, 1 << 30], [100] * 4, None),
                                              ([0, 2, 4], [10, -7], [100, 100, 0, 0], None), ([0, 2, 4], [1 << 29, 10], [100] * 4, [0, 0, 1, 1])):
            st, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full_like(q, 9.0)
            c.attend_shared(q, i32(length), i32(groups), i32(shared), out, c.workspace_shared(g, B, 1, len(shared)),
                            count=None if count is None else i32(count), table=None if table is None else i32(table), status=st)
            want, mag, sens, _ = shared_ref.attend_shared(r, q.double().cpu().numpy(), length, groups, [0 if not 0 <= n <= 128 else n for n in shared],
                                                          count, None, out=np.full(q.shape, 9.0))
            assert int(st) == pkg.LLM_ERR_POS_RANGE
            assert (np.abs(out.double().cpu().numpy() - want) <= tolerance("f32", hd, want, mag, sens)).all()


@pytest.mark.parametrize("hd", [32, 64, 128])
@pytest.mark.parametrize("wide", [False, True])
def test_nothing_to_see(hd, wide):
    kv, g, B = 2, 4, 3
    c, r = make(B, kv, 64, hd, garbage=2)
    ws, table = c.workspace_shared(g, B, 2, 2), i32(wide_table(r, B)) if wide else None
    q = torch.ones(B, 2, kv * g, hd, device="cuda")
    for length, count, shared, want in (([0] * B, None, [0, 0], 0.0), ([0] * B, None, [64, 30], 0.0), ([0] * B, [0] * B, [10, 0], 9.0),
                                        ([40, 64, 1], [0] * B, [40, 64], 9.0)):
        out = torch.full_like(q, 9.0)
        c.attend_shared(q, i32(length), i32([0, 1, 3]), i32(shared), out, ws, count=None if count is None else i32(count), table=table)
        assert (out == want).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_reaches_only_the_tokens_that_see_it(dtype, wide):
    rng = np.random.default_rng(14)
    for hd, g in ((128, 4), (64, 1), (32, 2)):
        kv, n, B = 2, 160, 3
        c, r = make(B, kv, 192, hd)
        fill(c, r, rng, n)
        table = i32(wide_table(r, B)) if wide else None
        bad, zero = torch.zeros(1, 1, kv, hd, device="cuda"), torch.zeros(1, 1, kv, hd, device="cuda")
        bad[0, 0, 1, 3] = float("nan")        # head 1 of the first row's token at position 160, alone in its block
        for k, v in ((bad, zero), (zero, bad)):
            c.write(k, v, i32([160]))
            q, _ = rows_of(rng, (B, 3, kv * g, hd), dtype)
            out = torch.zeros_like(q)
            # shared: seen by the last token of the rows that reach it; not shared: by the first row's alone
            for shared, seers in (([176], (0, 2)), ([160], (0,)), ([16], (0,))):
                c.attend_shared(q, i32([161, 160, 161]), i32([0, B]), i32(shared), out, c.workspace_shared(g, B, 3, 1), table=table)
                for b in range(B):
                    for i in range(3):
                        sees = b in seers and i == 2
                        assert torch.isfinite(out[b, i, :g]).all()
                        assert torch.isnan(out[b, i, g:]).all() if sees else torch.isfinite(out[b, i, g:]).all()
        # a query that is not finite: its head and token alone
        for value in (float("nan"), float("inf")):
            c.write(zero, zero, i32([160]))
            q, _ = rows_of(rng, (B, 3, kv * g, hd), dtype)
            q[1, 1, g, 5] = value
            out = torch.zeros_like(q)
            c.attend_shared(q, i32([160] * B), i32([0, B]), i32([100]), out, c.workspace_shared(g, B, 3, 1), table=table)
            wrong = ~torch.isfinite(out)
            assert wrong[1, 1, g].all() and int(wrong.sum()) == hd


def test_captured_graphs_streams_and_two_workspaces():
    rng = np.random.default_rng(31)
    B, kv, g, hd, cap = 6, 2, 4, 128, 640
    c, r = make(B, kv, cap, hd, garbage=4)
    fill(c, r, rng, 600)
    length, groups, shared = i32([600 - 7 * b for b in range(B)]), i32([0, 2, B]), i32([300, 500])
    q, _ = rows_of(rng, (B, 1, kv * g, hd), "bf16")
    ws = [c.workspace_shared(g, B, 1, 2) for _ in range(2)]
    out = [torch.zeros_like(q) for _ in range(2)]
    for i in range(2):
        ws[i].fill_(255)
        c.attend_shared(q, length, groups, shared, out[i], ws[i])
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.attend_shared(q, length, groups, shared, out[i], ws[i])
        graphs.append(gr)
    s = [torch.cuda.Stream() for _ in range(2)]
    for L, sh in (([600] * B, [300, 500]), ([250, 600, 0, 64, 500, 10], [64, 65]), ([600 - 7 * b for b in range(B)], [0, 600])):
        length.copy_(i32(L))
        shared.copy_(i32(sh))
        want = torch.zeros_like(q)
        c.attend_shared(q, length, groups, shared, want, c.workspace_shared(g, B, 1, 2))
        torch.cuda.synchronize()
        for _ in range(10):
            for i in range(2):
                with torch.cuda.stream(s[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], want)
        ref, mag, sens, _ = shared_ref.attend_shared(r, q.double().cpu().numpy(), L, [0, 2, B], sh)
        assert (np.abs(want.double().cpu().numpy() - ref) <= tolerance("bf16", hd, ref, mag, sens)).all()


def test_the_wrapper_refuses_what_does_not_fit():
    c = pkg.QCache.empty(2, 2, 128, 64)
    q = torch.zeros(2, 1, 4, 64, device="cuda")
    good = dict(q=q, length=i32([1, 1]), groups=i32([0, 2]), shared=i32([0]), out=torch.zeros_like(q), workspace=c.workspace_shared(2, 2, 1, 1))
    c.attend_shared(**good)
    for kw in (dict(groups=i32([0, 1, 2])), dict(groups=None), dict(shared=None), dict(shared=i32([0, 0, 0])), dict(groups=i32([0, 2]).long()),
               dict(shared=torch.zeros(1, device="cuda")), dict(out=torch.zeros_like(q).bfloat16()), dict(length=i32([1])),
               dict(q=torch.zeros(2, 1, 5, 64, device="cuda")), dict(table=i32([0, 1])), dict(scale=float("inf")),
               dict(shared=i32([]), groups=i32([0]))):
        with pytest.raises(pkg.LlmError):
            c.attend_shared(**{**good, **kw})


def test_a_run_of_fork_write_attention_and_draws():
    # one prompt, forked into four continuations that go on by themselves: pages forked and copied, tokens written,
    # attended to behind the shared pages, and drawn from, against the same steps in plain form
    rng = np.random.default_rng(41)
    R, per, kv, g, hd, V, n = 4, 6, 2, 2, 64, 300, 150
    c, r = make(2, kv, 12 * 64, hd)
    book = [pkg.Pages.empty(R, per, 24) for _ in range(2)]
    pws = book[0].workspace()
    moves, counts, st = torch.zeros(R, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    head = torch.from_numpy(rng.standard_normal((kv * g * hd, V)).astype(np.float32)).cuda()
    table, length = [[-1] * per for _ in range(R)], [0] * R
    layers = pkg.QCacheLayers([c])

    def update(parent, new):
        nonlocal table, length
        book[0].update(book[1], moves, counts, pws, parent=i32(parent), length=i32(new), status=st)
        layers.copy(moves, counts=counts, status=st)
        book.reverse()
        table, length, steps, _ = shared_ref.update(table, length, 24, parent, new)
        for a, b in steps:
            for x, m in ((r.k, 64), (r.v, 64), (r.ks, 4), (r.vs, 4)):
                x[b // 12, :, b % 12 * m:(b % 12 + 1) * m] = x[a // 12, :, a % 12 * m:(a % 12 + 1) * m]
        assert book[0].table.tolist() == table and int(st) == 0

    def write(rows, pos, S):
        k, kn = rows_of(rng, (len(rows), S, kv, hd), "bf16")
        v, vn = rows_of(rng, (len(rows), S, kv, hd), "bf16")
        t = [table[b] for b in rows]
        c.write(k, v, i32(pos), table=i32(t), status=st)
        r.write(kn, vn, pos, None, t)

    update([0, -1, -1, -1], [n, 0, 0, 0])
    write([0], [0], n)
    update([0] * R, [n + 1] * R)
    ws = c.workspace_shared(g, R, 1, 1)
    for step in range(6):
        write(range(R), [x - 1 for x in length], 1)
        q, qn = rows_of(rng, (R, 1, kv * g, hd), "bf16")
        out = torch.empty_like(q)
        c.attend_shared(q, book[0].length, i32([0, R]), i32([128]), out, ws, table=book[0].table, status=st)
        want, mag, sens, _ = shared_ref.attend_shared(r, qn, length, [0, R], [128], None, table)
        assert (np.abs(out.double().cpu().numpy() - want) <= tolerance("bf16", hd, want, mag, sens)).all()
        logits = out.flatten(1).float() @ head
        ids, u = torch.empty(R, dtype=torch.int32, device="cuda"), rng.random(R).astype(np.float32)
        pkg.llm_sample_rows(logits, torch.full((R,), 0.8, device="cuda"), torch.from_numpy(u).cuda(), ids, min_p=torch.full((R,), 0.02, device="cuda"), status=st)
        x = logits.cpu().numpy()
        assert ids.tolist() == [shared_ref.sample(x[b], np.float32(0.8), V, np.float32(1), np.float32(0.02), u[b]) for b in range(R)]
        # the best two go on twice, as a search with beams does
        parent = [0, 1, 2, 3] if step % 2 else [1, 1, 3, 0]
        update(parent, [length[p] + 1 for p in parent])
    assert int(st) == 0
    update([0, -1, 0, -1], [length[0], 0, 65, 0])
    assert counts.tolist()[1] == shared_ref.pages_of(length[0]) + 1


@pytest.mark.parametrize("dtype,hd,S", [("bf16", 128, 1), ("f32", 64, 3)])
def test_captured_calls_that_read_the_shared_positions_once(dtype, hd, S):
    # as above, for calls whose tables have room for more: several kernels each, workspaces that held anything
    rng = np.random.default_rng(32)
    B, kv, g, cap = 7, 2, 4, 640
    c, r = make(B, kv, cap, hd, garbage=4)
    fill(c, r, rng, 600)
    table = i32(wide_table(r, B))
    length, groups, shared = i32([600 - 7 * b for b in range(B)]), i32([0, 2, B]), i32([300, 500])
    q, _ = rows_of(rng, (B, S, kv * g, hd), dtype)
    ws = [c.workspace_shared(g, B, S, 2) for _ in range(2)]
    out = [torch.zeros_like(q) for _ in range(2)]
    graphs = []
    for i in range(2):
        ws[i].fill_(255)
        c.attend_shared(q, length, groups, shared, out[i], ws[i], table=table)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            c.attend_shared(q, length, groups, shared, out[i], ws[i], table=table)
    s = [torch.cuda.Stream() for _ in range(2)]
    for L, sh in (([600] * B, [300, 500]), ([250, 600, 0, 64, 500, 10, 3], [64, 65]), ([600 - 7 * b for b in range(B)], [0, 600])):
        length.copy_(i32(L))
        shared.copy_(i32(sh))
        want, few = torch.zeros_like(q), torch.zeros_like(q)
        c.attend_shared(q, length, groups, shared, want, ws[0], table=table)
        c.attend_shared(q, length, groups, shared, few, ws[0])      # (the other way: the same workspace)
        torch.cuda.synchronize()
        for _ in range(10):
            for i in range(2):
                with torch.cuda.stream(s[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], want)
        ref, mag, sens, _ = shared_ref.attend_shared(r, q.double().cpu().numpy(), L, [0, 2, B], sh)
        for x in (want, few):
            assert (np.abs(x.double().cpu().numpy() - ref) <= tolerance(dtype, hd, ref, mag, sens)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_beside_many_columns(dtype):
    # a group of 132 columns, whose shared positions the kernel for many takes: a NaN among them, behind what some rows see;
    # a query that is not finite
    rng = np.random.default_rng(17)
    hd, kv, g, B = 128, 2, 4, 33
    c, r = make(1, kv, 640, hd)
    fill(c, r, rng, 592)          # (whole blocks: a value that is not finite makes its block's scale NaN)
    bad, zero = torch.zeros(1, 1, kv, hd, device="cuda"), torch.zeros(1, 1, kv, hd, device="cuda")
    bad[0, 0, 1, 3] = float("nan")
    table = i32(np.concatenate([np.tile(np.arange(10), (B, 1)), np.full((B, 4086), -1)], 1))
    length = [593 if b % 3 == 0 else 592 if b % 3 == 1 else 77 for b in range(B)]
    for k, v in ((bad, zero), (zero, bad)):
        c.write(k, v, i32([592]))
        q, _ = rows_of(rng, (B, 1, kv * g, hd), dtype)
        out = torch.zeros_like(q)
        c.attend_shared(q, i32(length), i32([0, B]), i32([593]), out, c.workspace_shared(g, B, 1, 1), table=table)
        wrong = ~torch.isfinite(out[:, 0])
        assert not wrong[:, :g].any()
        for b in range(B):
            assert wrong[b, g:].all() if length[b] == 593 else not wrong[b].any()
    c.write(zero, zero, i32([592]))
    for value in (float("nan"), float("inf")):
        q, _ = rows_of(rng, (B, 1, kv * g, hd), dtype)
        q[31, 0, 5, 100] = value
        out = torch.zeros_like(q)
        c.attend_shared(q, i32([592] * B), i32([0, B]), i32([590]), out, c.workspace_shared(g, B, 1, 1), table=table)
        wrong = ~torch.isfinite(out)
        assert wrong[31, 0, 5].all() and int(wrong.sum()) == hd


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 1000])
def test_calls_of_many_units(G, dtype):
    # thousands of units, whose counts lie where the first tiles go: one group (the kernel for many columns, the rows' own
    # positions on that for few), and groups of four rows (the kernel for few); the same bits every time
    rng = np.random.default_rng(18)
    B, kv, g, hd, n = 4000, 2, 1, 64, 150
    c, r = make(2, kv, 256, hd, garbage=5)
    fill(c, r, rng, 256, np.arange(8).reshape(2, 4))
    table = np.full((B, 4096), -1)
    table[:, :3] = rng.integers(0, 8, (B, 3))
    length = (n - np.arange(B) % 37).tolist()
    groups, shared = np.linspace(0, B, G + 1).astype(int).tolist(), (100 + np.arange(G) % 29).tolist()
    q, qn = rows_of(rng, (B, 1, kv * g, hd), dtype)
    ws, outs = c.workspace_shared(g, B, 1, G), []
    for i in range(8):
        outs.append(torch.full_like(q, 9.0))
        c.attend_shared(q, i32(length), i32(groups), i32(shared), outs[i], ws, table=i32(table))
        ws.fill_(255 if i % 2 else 0)
    want, mag, sens, _ = shared_ref.attend_shared(r, qn, length, groups, shared, None, table[:, :3])
    assert (np.abs(outs[0].double().cpu().numpy() - want) <= tolerance(dtype, hd, want, mag, sens)).all()
    assert all(torch.equal(x, outs[0]) for x in outs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,g,S", [(32, 2, 1), (64, 1, 3), (128, 4, 1), (128, 8, 33), (64, 4, 128)])
def test_rows_without_tokens_have_no_pages(hd, g, S, dtype):
    # rows that take no part in a call, whole groups of them and single ones, whose tables were never set: nothing of theirs is
    # looked at or reported, and their outputs stay; a group's first row holds its pages with or without tokens of its own.  128
    # tokens of 4 heads: the kernel for many columns
    rng = np.random.default_rng(hd + S)
    rows, kv, B = 6, 2, 8
    c, r = make(rows, kv, 256, hd, garbage=8)
    table = np.zeros((B, 4), np.int32)
    table[[0, 3, 6]] = pages(rng, 3, 256, rows)
    fill(c, r, rng, 256, table[[0, 3, 6]])
    for b, lead in ((1, 0), (2, 0), (4, 3), (5, 3), (7, 6)):
        table[b] = table[lead]
    length, groups, shared = [250, 249, 170, 200, 190, 180, 256, 140], [0, 3, 6, 8], [129, 100, 64]
    q, qn = rows_of(rng, (B, S, kv * g, hd), dtype)
    ws = c.workspace_shared(g, B, S, 3)
    for count in ([S, 0, 1, 0, 0, 0, 0, S], [0, 0, S, 0, 0, 0, (S + 1) // 2, 0], [0] * B):
        view = table.copy()
        for b in range(B):
            i = max(x for x in range(3) if groups[x] <= b)
            if count[b] == 0 and (b != groups[i] or not any(count[groups[i]:groups[i + 1]])):
                view[b] = -1 if b % 2 else 1 << 30
        want, mag, sens, _ = shared_ref.attend_shared(r, qn, length, groups, shared, count, table, out=np.full(q.shape, 9.0))
        for t in (view, wide_table(r, B, view)):
            out, st = torch.full_like(q, 9.0), torch.zeros(1, dtype=torch.int32, device="cuda")
            c.attend_shared(q, i32(length), i32(groups), i32(shared), out, ws, count=i32(count), table=i32(t), status=st)
            assert int(st) == 0
            assert (np.abs(out.double().cpu().numpy() - want) <= tolerance(dtype, hd, want, mag, sens)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,g,B,S,per", [(64, 1, 4096, 1, 160), (64, 1, 4097, 1, 160), (128, 1, 4500, 1, 3), (64, 16, 4, 2048, 512), (64, 16, 4, 2050, 512)])
def test_both_sides_of_the_most_units(hd, g, B, S, per, dtype):
    # up to 4096 units a side the shared positions can be read once; calls of more go row by row, as the ordinary attention takes them
    rng = np.random.default_rng(B + S)
    kv, n = 1, 140
    c, r = make(2, kv, 320, hd, garbage=5)
    fill(c, r, rng, 320, np.arange(10).reshape(2, 5))
    table = np.full((B, per), -1)
    table[:, :3] = rng.integers(0, 10, (B, 3))
    length, G = (n - np.arange(B) % 37).tolist(), min(B, 9) // 3
    groups, shared = np.linspace(0, B, G + 1).astype(int).tolist(), (60 + np.arange(G) * 5).tolist()
    count = None if S == 1 else [S, 1, 3, 2][:B]
    if S > 1:
        length = [140, 120, 133, 64]
    q, qn = rows_of(rng, (B, S, kv * g, hd), dtype)
    out, st = torch.full_like(q, 9.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    c.attend_shared(q, i32(length), i32(groups), i32(shared), out, c.workspace_shared(g, B, S, G), table=i32(table), status=st,
                    count=None if count is None else i32(count))
    assert int(st) == 0
    want, mag, sens, _ = shared_ref.attend_shared(r, qn, length, groups, shared, count, table[:, :3], out=np.full(q.shape, 9.0))
    assert (np.abs(out.double().cpu().numpy() - want) <= tolerance(dtype, hd, want, mag, sens)).all()


def test_a_call_that_no_way_takes_is_refused():
    c = pkg.QCache.empty(1, 8, 64, 64)
    q = torch.zeros(1, 1, 8, 64, device="cuda").expand(4096, 1, 8, 64)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda").expand(4096, 1 << 16)
    lib, P = pkg.lib(), q.data_ptr()          # (refused on the host: nothing is read)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    for B, S, G in ((1 << 20, 1 << 10, 1), (1 << 20, 1 << 10, 1 << 20)):
        st = lib.llm_qcache_attend_shared(c._c, P, 0, 512, 1, B, S, P, None, table.data_ptr(), 1 << 16, P, P, G, 0.1, P, 512, ws.data_ptr(),
                                          1 << 60, None, None)
        assert st == pkg.LLM_ERR_ARG and b"too large" in lib.llm_last_error(None)


@pytest.mark.parametrize("hd", [32, 64, 128])
def test_a_zeroed_workspace_serves_both_attentions_by_turns(hd):
    rng = np.random.default_rng(19)
    B, kv, g, cap = 5, 2, 4, 640
    c, r = make(B, kv, cap, hd, garbage=4)
    fill(c, r, rng, 600)
    table = i32(wide_table(r, B))
    length, groups, shared = i32([600 - 7 * b for b in range(B)]), i32([0, 2, B]), i32([300, 500])
    q, _ = rows_of(rng, (B, 8, kv * g, hd), "bf16")
    ws = torch.zeros(max(c.workspace(g, B, 8).numel(), c.workspace_shared(g, B, 8, 2).numel()), dtype=torch.uint8, device="cuda")
    want, out, other = (torch.empty_like(q) for _ in range(3))
    c.attend(q, length, want, c.workspace(g, B, 8))
    for t in (table, None, table, table):
        c.attend_shared(q, length, groups, shared, other, ws, table=t)
        for _ in range(2):
            out.fill_(9.0)
            c.attend(q, length, out, ws)
            assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,g,S", [(64, 2, 1), (128, 4, 1), (128, 4, 4)])
def test_uneven_groups_and_empty_ones(hd, g, S, dtype):
    # as many groups as rows, most of them empty (all rows in the first, in the last, in one between); one group of most rows beside single
    # ones; more empty groups than others
    rng = np.random.default_rng(20)
    kv, B = 2, 40
    c, r = make(B, kv, 256, hd, garbage=6)
    fill(c, r, rng, 250)
    length = [250 - 3 * (b % 7) for b in range(B)]
    for groups, shared in (([0] + [B] * B, [200] + [70] * (B - 1)), ([0] * B + [B], [70] * (B - 1) + [200]),
                           ([0] * 11 + [B] * (B - 10), [70] * 10 + [200] + [70] * (B - 11)),
                           ([0, 31] + list(range(32, B + 1)), [200] + [129] * (B - 31)), ([0, 0, 0, 3, 3, 3, 39, 39, 39, 40], [1, 2, 130, 3, 4, 200, 5, 6, 60])):
        check(c, r, rng, S, g, dtype, length, groups, shared)


def test_workspaces_of_calls_that_go_row_by_row():
    # as many groups as rows, or more rows than are counted: as much as the ordinary attention needs
    c = pkg.QCache.empty(2, 8, 256, 128)
    for g, B, S, G in ((4, 5000, 1, 7), (4, 64, 1, 64), (4, 600, 64, 1)):
        assert c.workspace_shared(g, B, S, G).numel() == c.workspace(g, B, S).numel()
    assert c.workspace_shared(4, 64, 1, 63).numel() > c.workspace(4, 64, 1).numel()
