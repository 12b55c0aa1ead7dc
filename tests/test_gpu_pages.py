"""Page tables that fork, shrink, grow and compact, and copies of pages, on the GPU against the plain
definitions of tests/shared_ref.py: everything must be equal."""
import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
import synth
from synth import WORKLOADS
from tests import shared_ref as ref
from tests.test_gpu_qcache import i32, make, same

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Book:
    def __init__(self, rows, per, pages):
        self.now, self.then = (pkg.Pages.empty(rows, per, pages) for _ in range(2))
        self.ws = self.now.workspace()
        self.ws.fill_(-77)
        self.table, self.length, self.rows, self.pages = [[-1] * per for _ in range(rows)], [0] * rows, rows, pages

    def load(self, table, length):
        self.table, self.length = [list(map(int, t)) for t in table], [int(n) for n in length]
        self.now.table.copy_(i32(table))
        self.now.length.copy_(i32(length))

    def check(self, want, m, moves, counts, status, code):
        if want is None:
            assert int(status) == code
            assert counts.tolist() == [0, -1] and (moves == -1).all()
            assert torch.equal(self.then.table, self.now.table) and torch.equal(self.then.length, self.now.length)
            return False
        assert int(status) == 0
        table, length, steps, n = want
        assert counts.tolist() == n
        assert moves.tolist() == [list(x) for x in steps] + [[-1, -1]] * (m - len(steps))
        assert self.then.table.tolist() == table and self.then.length.tolist() == list(length)
        self.now, self.then, self.table, self.length = self.then, self.now, table, list(length)
        return True

    def update(self, parent=None, length=None, code=pkg.LLM_ERR_OOM):
        moves = torch.full((self.rows, 2), 7, dtype=torch.int32, device="cuda")
        counts, status = torch.full((2,), 7, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.then.table.fill_(5)
        self.now.update(self.then, moves, counts, self.ws, parent=None if parent is None else i32(parent),
                        length=None if length is None else i32(length), status=status)
        return self.check(ref.update(self.table, self.length, self.pages, parent, length), self.rows, moves, counts, status, code)

    def compact(self, code=pkg.LLM_ERR_ARG):
        m = max(1, self.pages // 2)
        moves = torch.full((m, 2), 7, dtype=torch.int32, device="cuda")
        counts, status = torch.full((2,), 7, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.then.table.fill_(5)
        self.now.compact(self.then, moves, counts, self.ws, status=status)
        return self.check(ref.compact(self.table, self.length, self.pages), m, moves, counts, status, code)


@pytest.mark.parametrize("rows,per,pages", [(1, 1, 1), (1, 5, 4), (4, 3, 7), (7, 9, 40), (33, 18, 400), (64, 300, 9000), (1500, 5, 3001),
                                            (3, 2100, 6000), (2, 1, 70000)])
def test_random_forks_rewinds_growth_and_frees(rows, per, pages):
    rng = np.random.default_rng(rows + per)
    b, done = Book(rows, per, pages), 0
    for step in range(12):
        parent = rng.integers(-1, rows, rows) if step % 3 else None
        most = per * 64 if step % 2 else max(1, per * 16)
        length = np.minimum(per * 64, rng.integers(0, most + 1, rows) // rng.choice([1, 1, 64], rows) * rng.choice([1, 64], rows))
        if step == 7:
            length = None
        done += b.update(parent, length)
        b.compact()
    assert done > 0


def test_the_pool_runs_out_exactly():
    b = Book(3, 4, 6)
    assert b.update(length=[128, 65, 64])       # 2 + 2 + 1 pages
    assert b.update(length=[129, 65, 64])       # the last one
    assert not b.update(length=[129, 129, 64])  # one too many
    assert b.update(parent=[0, -1, 0])          # a row gone, a fork of 3 pages: one copied
    assert not b.update(parent=[0, 0, 0], length=[129, 193, 129 + 64])
    assert b.update(parent=[-1, -1, -1])


@pytest.mark.parametrize("big", [False, True])
def test_what_is_out_of_range_leaves_everything_as_it_was(big):
    R, per, pages = (40, 500, 30000) if big else (4, 5, 30)  # (one cluster, one CTA)
    b = Book(R, per, pages)
    assert b.update(length=[100] * R)
    for parent, length, code in [([R] + [0] * (R - 1), None, pkg.LLM_ERR_ARG), ([0] * (R - 1) + [-2], None, pkg.LLM_ERR_ARG),
                                 (None, [-1] + [5] * (R - 1), pkg.LLM_ERR_POS_RANGE),
                                 (None, [5] * (R - 1) + [per * 64 + 1], pkg.LLM_ERR_POS_RANGE)]:
        assert not b.update(parent, length, code)
    for at, page in ((0, pages), (1, -1), (1, 1 << 30)):
        table = [list(t) for t in b.table]
        table[R - 1][at] = page
        old = b.table
        b.load(table, b.length)
        assert not b.update(code=pkg.LLM_ERR_ARG) and not b.compact()
        assert b.update(parent=[0] * R, length=[64] * R)     # (pages that no new row keeps are not looked at)
        b.load(old, [100] * R)
    b.load(b.table, [100] * (R - 1) + [per * 64 + 1])
    assert not b.compact(pkg.LLM_ERR_POS_RANGE) and not b.update(code=pkg.LLM_ERR_POS_RANGE)
    # entries behind a row's pages mean nothing
    table = [list(t) for t in b.table]
    for t in table:
        t[2:] = [-9, 1 << 30, 0][: per - 2] + [3] * (per - 5)
    b.load(table, [100] * R)
    assert b.update() and b.compact()


def test_no_status_word_and_one_workspace_for_both():
    b = Book(2, 2, 3)
    assert b.update(length=[70, 10])
    moves, counts = torch.zeros(2, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    b.now.update(b.then, moves, counts, b.ws, length=i32([128, 128]))
    assert counts.tolist() == [0, -1]
    assert b.compact()


def test_a_captured_update_follows_its_inputs():
    b = Book(6, 4, 40)
    assert b.update(length=[100, 0, 0, 70, 0, 0])
    parent, length = i32([0, 0, 0, 3, 3, 3]), i32([101, 101, 101, 71, 71, 71])
    moves, counts = torch.zeros(6, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    b.now.update(b.then, moves, counts, b.ws, parent=parent, length=length)  # (loads the kernel)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.now.update(b.then, moves, counts, b.ws, parent=parent, length=length)
    for p, n in (([0, 0, 0, 3, 3, 3], [101, 101, 101, 71, 71, 71]), ([3, -1, 0, 0, 3, 5], [10, 0, 200, 64, 65, 1])):
        parent.copy_(i32(p))
        length.copy_(i32(n))
        g.replay()
        want = ref.update(b.table, b.length, 40, p, n)
        assert b.then.table.tolist() == want[0] and b.then.length.tolist() == want[1] and counts.tolist() == want[3]
        assert moves.tolist()[: want[3][0]] == [list(x) for x in want[2]]


# ---- copies ----

@pytest.mark.parametrize("hd,kv,rows,cap", [(16, 1, 1, 128), (32, 3, 2, 192), (64, 2, 3, 256), (128, 8, 4, 128), (256, 1, 2, 320)])
def test_copied_pages_equal_and_nothing_else_changes(hd, kv, rows, cap):
    rng = np.random.default_rng(hd)
    pairs = [make(rows, kv, cap, hd, garbage=hd + i) for i in range(3)]
    layers = pkg.QCacheLayers([c for c, _ in pairs])
    per, pool = cap // 64, rows * cap // 64
    for step in range(4):
        order = rng.permutation(pool)
        n = pool // 2
        moves = [[int(a), int(b)] for a, b in zip(order[:n], order[n:2 * n])]
        if step == 1 and n > 1:
            moves[1][0] = moves[0][0]            # one source twice
        listed = moves + [[-1, -1], [-1, -1]]
        took = n if step < 3 else n - 1          # the count says how many of them there are
        counts = i32([took, 99]) if step > 1 else None
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        layers.copy(i32(listed), counts=counts, status=status)
        assert int(status) == 0
        for c, r in pairs:
            for a, b in moves[:took]:
                for x, m in ((r.k, 64), (r.v, 64), (r.ks, 4), (r.vs, 4)):
                    x[b // per, :, b % per * m:(b % per + 1) * m] = x[a // per, :, a % per * m:(a % per + 1) * m]
            same(c, r)


def test_captured_copies_behind_a_fill_a_copy_of_memory_and_an_update():
    # what a copy of pages follows in a captured graph: a memory copy of its moves, an update that writes them, another copy
    rng = np.random.default_rng(9)
    R, per, pages = 3, 4, 16
    c = pkg.QCache.empty(1, 2, pages * 64, 64)
    layers = pkg.QCacheLayers([c])
    book = [pkg.Pages.empty(R, per, pages) for _ in range(2)]
    ws = book[0].workspace()
    counts = torch.zeros(2, dtype=torch.int32, device="cuda")
    moves, given, second = (torch.zeros(R, 2, dtype=torch.int32, device="cuda") for _ in range(3))
    parent, length = (torch.zeros(R, dtype=torch.int32, device="cuda") for _ in range(2))
    second.copy_(torch.tensor([[1, 11], [-1, -1], [11, 12]], dtype=torch.int32))

    def run():
        moves.copy_(given)                      # (a memory copy)
        layers.copy(moves)
        layers.copy(second[:1].contiguous())
        layers.copy(second[2:].contiguous())
        book[0].update(book[1], moves, counts, ws, parent=parent, length=length)
        layers.copy(moves, counts=counts)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for trial in range(6):
        codes = torch.from_numpy(rng.integers(0, 256, (1, 2, pages * 64, 64)).astype(np.uint8)).cuda()
        c.tensors[0].copy_(codes)
        first = rng.permutation(10)[:6].reshape(3, 2)
        given.copy_(torch.from_numpy(first.astype(np.int32)))
        # row 0 holds pages 13 and 14, the latter in part; the others go on from it
        book[0].table.fill_(-1)
        book[0].table[0, :2] = torch.tensor([13, 14])
        book[0].length.copy_(torch.tensor([64 + 10 + trial, 0, 0]))
        length.fill_(64 + 10 + trial)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = codes.cpu().numpy().reshape(2, pages, 64, 64).copy()
        for a, b in [*[(a, b) for a, b in first], (1, 11), (11, 12), *moves.tolist()[:int(counts[0])]]:
            want[:, b] = want[:, a]
        assert int(counts[0]) == 2 and moves[:2, 0].tolist() == [14, 14]
        assert (c.tensors[0].cpu().numpy().reshape(want.shape) == want).all()


def test_pages_outside_the_pool_are_reported_and_skipped():
    c, r = make(2, 2, 128, 64, garbage=1)
    for move in ([4, 0], [0, 4], [-1, 0], [0, -1], [1 << 30, 1], [0, -(1 << 31)]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkg.QCacheLayers([c]).copy(i32([move, [3, 2]]), status=status)
        assert int(status) == pkg.LLM_ERR_ARG
        r.k[1, :, :64], r.v[1, :, :64] = r.k[1, :, 64:], r.v[1, :, 64:]
        r.ks[1, :, :4], r.vs[1, :, :4] = r.ks[1, :, 4:], r.vs[1, :, 4:]
        same(c, r)


def test_more_layers_than_one_launch_takes():
    n = 2 * 96 + 5
    caches = [pkg.QCache.empty(1, 1, 128, 16) for _ in range(n)]
    for i, c in enumerate(caches):
        c.tensors[0][:, :, :64] = i % 100
        c.tensors[3][:, :, :4] = float(i)
    pkg.QCacheLayers(caches).copy(i32([[0, 1]]))
    for i, c in enumerate(caches):
        assert (c.tensors[0] == i % 100).all() and (c.tensors[3] == float(i)).all()


def test_the_wrappers_refuse_what_does_not_fit():
    b = Book(4, 3, 20)
    moves, counts = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for kw in (dict(moves=moves[:3]), dict(moves=moves.long()), dict(counts=counts[:1]), dict(workspace=b.ws[:-1]), dict(moves=None),
               dict(out=b.now), dict(parent=i32([0] * 3)), dict(length=i32([0] * 5)), dict(status=counts)):
        args = dict(out=b.then, moves=moves, counts=counts, workspace=b.ws)
        args.update(kw)
        with pytest.raises(pkg.LlmError):
            b.now.update(**args)
    with pytest.raises(pkg.LlmError):
        b.now.compact(b.then, moves, counts, b.ws)          # (moves for 10 are wanted)
    for table, length in ((b.now.table[:, :2], b.now.length), (b.now.table, b.now.length[:3]), (b.now.table.long(), b.now.length)):
        with pytest.raises(pkg.LlmError):
            pkg.Pages(table, length, 20)
    c = pkg.QCache.empty(1, 1, 128, 64)
    for bad in (lambda: pkg.QCacheLayers([]), lambda: pkg.QCacheLayers([c]).copy(moves.long()),
                lambda: pkg.QCacheLayers([c]).copy(moves.flatten()), lambda: pkg.QCacheLayers([c]).copy(moves, counts=counts[:1])):
        with pytest.raises(pkg.LlmError):
            bad()
    pkg.QCacheLayers([c]).copy(moves[:0])                    # nothing to do


# ---- a handle's pool ----

@pytest.mark.parametrize("cache_type", [pkg.LLM_CACHE_MODEL, pkg.LLM_CACHE_E4M3])
@pytest.mark.parametrize("bf16", [False, True])
def test_a_forked_row_of_a_handle_goes_on_like_its_parent(bf16, cache_type):
    # prompts run through pages, row 2 is forked from row 0 (whole pages together, the open one copied); fed what
    # row 0 is fed, it gets the same logits bit for bit, and a row fed something else does not disturb the others
    w = WORKLOADS["tiny_f32"]
    s = synth.shrink(w.shape, bf16=bf16) if bf16 else w.shape
    m = pkg.Model(s, synth.model_blob(s, w.seed_weights), max_batch=4, max_seq=192, cache_type=cache_type)
    per = 3
    b = Book(4, per, 12)
    toks = synth.tokens(w.seed_tokens, 0, 400, s.vocab)
    n = 100
    assert b.update(length=[n, 70, 0, 0])
    for t in range(n):
        rows = [0, 1] if t < 70 else [0]
        m.decode_paged([toks[r * 100 + t] for r in rows], [t] * len(rows), np.array([b.table[r] for r in rows], np.int32).clip(min=0))
    assert b.update(parent=[0, 1, 0, 1], length=[n + 3, 73, n + 3, 73])
    m.copy_pages([[b.table[0][1], b.table[2][1]], [b.table[1][1], b.table[3][1]]])
    feed = synth.tokens(w.seed_tokens, 3, 3, s.vocab)
    table = np.array(b.table, np.int32).clip(min=0)
    for i in range(3):
        x = [feed[i], feed[i], feed[i], (feed[i] + 1) % s.vocab]
        got = m.decode_paged(x, [n + i, 70 + i, n + i, 70 + i], table)
        assert np.array_equal(got[0], got[2])
        assert not np.array_equal(got[1], got[3])
    for bad in ([[0, 0]], [[0, 1], [2, 1]], [[0, 1], [1, 2]], [[1, 2], [0, 1]], [[0, 12]], [[-1, 3]]):
        with pytest.raises(pkg.LlmError) as e:
            m.copy_pages(bad)
        assert e.value.status == pkg.LLM_ERR_ARG
    m.copy_pages(np.zeros((0, 2), np.int32))
    m.close()


def test_every_page_of_a_handle_can_be_moved_at_once():
    w = WORKLOADS["tiny_f32"]
    s = w.shape
    m = pkg.Model(s, synth.model_blob(s, w.seed_weights), max_batch=2, max_seq=192)
    rng = np.random.default_rng(3)
    k = rng.standard_normal((s.layers, 2, s.kv, 192, s.hd)).astype(np.float32)
    for l in range(s.layers):
        for r in range(2):
            m.kv_import(l, r, 0, k[l, r], -k[l, r])
    m.copy_pages([[0, 5], [0, 1], [4, 2], [0, 3]])          # (more than half the pool)
    page = lambda x, p: x[:, p // 3, :, p % 3 * 64:p % 3 * 64 + 64]  # noqa: E731
    for a, b in ((0, 5), (0, 1), (4, 2), (0, 3)):
        page(k, b)[:] = page(k, a)
    for l in range(s.layers):
        for r in range(2):
            got = m.kv_export(l, r, 0, 192)
            assert np.array_equal(got[0], k[l, r]) and np.array_equal(got[1], -k[l, r])
    m.close()
    m = pkg.Model(s, synth.model_blob(s, w.seed_weights), max_batch=1, max_seq=80)
    with pytest.raises(pkg.LlmError) as e:
        m.copy_pages([[0, 1]])
    assert e.value.status == pkg.LLM_ERR_CONFIG
    m.close()


@pytest.mark.parametrize("pinned", [False, True])
def test_moves_are_read_before_the_call_returns(pinned):
    # the handle's stream is busy when pages are copied, and the array is used again at once, from ordinary memory and from
    # memory that the device reads by itself; few moves, and more than one transfer takes
    w = WORKLOADS["tiny_f32"]
    s = w.shape
    for rows, seq, moves, later in ((2, 192, [[0, 5], [0, 1], [4, 2], [0, 3]], [[4, 5], [4, 1], [0, 2], [4, 3]]),
                                    (16, 1 << 16, [[3, p] for p in range(1 << 14) if p not in (3, 4)], [[4, p] for p in range(1 << 14) if p not in (3, 4)])):
        m = pkg.Model(s, synth.model_blob(s, w.seed_weights), max_batch=rows, max_seq=seq)
        per = seq // 64
        k = np.random.default_rng(4).standard_normal((s.layers, s.kv, min(seq, 320), s.hd)).astype(np.float32)
        for l in range(s.layers):
            for r in range(2 if rows == 2 else 1):
                m.kv_import(l, r, 0, k[l] * (1 + r), -k[l])
        page = lambda l, p: k[l, :, p % per * 64:p % per * 64 + 64] * (1 + p // per)  # noqa: E731
        host = torch.tensor(moves, dtype=torch.int32)
        host = host.pin_memory() if pinned else host
        with torch.cuda.stream(torch.cuda.ExternalStream(pkg.llm_stream(m.h))):
            torch.cuda._sleep(200_000_000)
        pkg.llm_copy_pages(m.h, host, len(moves))
        host.copy_(torch.tensor(later, dtype=torch.int32))
        m.synchronize()
        for l in range(s.layers):
            for a, b in moves[:2] + moves[-2:] + moves[len(moves) // 3::1000]:
                got = m.kv_export(l, b // per, b % per * 64, 64)
                assert np.array_equal(got[0], page(l, a)), (a, b)
        m.close()
