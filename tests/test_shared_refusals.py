"""Refusals of the entries for shared positions, pages and per-row sampling that the host makes before any GPU
work, and the plain definitions the GPU tests use (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
from llama_architecture_kv_gb300 import build as pkg_build
from tests import shared_ref as ref
from tests.test_qcache_refusals import CACHES, cache

ARG, CONFIG, BATCH = pkg.LLM_ERR_ARG, pkg.LLM_ERR_CONFIG, pkg.LLM_ERR_BATCH
P = 0x10000  # an aligned address that is never followed: every case below is refused on the host


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return pkg.lib()


def test_shared_attention_refuses_bad_arguments(lib):
    def attend(c=None, q=P, dtype=1, q_stride=256, group=2, B=2, S=1, length=P, count=None, table=None, pages=0, groups=P,
               shared=P, G=1, scale=0.125, out=P, out_stride=256, ws=P, nbytes=1 << 40, status=None):
        return lib.llm_qcache_attend_shared(c or cache(), q, dtype, q_stride, group, B, S, length, count, table, pages, groups,
                                            shared, G, scale, out, out_stride, ws, nbytes, status, None)
    for kw, code in CACHES:
        assert attend(c=cache(**kw)) == code, kw
    for kw, code in [(dict(group=0), CONFIG), (dict(group=17), CONFIG), (dict(q=None), ARG), (dict(out=None), ARG),
                     (dict(q_stride=255), ARG), (dict(out_stride=248), ARG), (dict(dtype=-1), ARG), (dict(length=None), ARG),
                     (dict(scale=float("nan")), ARG), (dict(B=0), BATCH), (dict(B=3), BATCH), (dict(S=0), ARG),
                     (dict(groups=None), ARG), (dict(shared=None), ARG), (dict(groups=P + 2), ARG), (dict(shared=P + 1), ARG),
                     (dict(G=0), ARG), (dict(G=3), ARG), (dict(G=-1), ARG), (dict(status=P + 2), ARG),
                     (dict(table=P, pages=0), ARG), (dict(count=P + 3), ARG)]:
        assert attend(**kw) == code, kw
    n = ctypes.c_uint64()
    for kw, args, code in [(dict(rows=0), (1, 1, 1, 1), CONFIG), (dict(), (0, 1, 1, 1), CONFIG), (dict(), (1, 0, 1, 1), BATCH),
                           (dict(), (1, 2, 0, 1), ARG), (dict(), (1, 2, 1, 0), ARG), (dict(), (1, 2, 1, 3), ARG)]:
        assert lib.llm_qcache_shared_workspace(cache(**kw), *args, ctypes.byref(n)) == code, (kw, args)
    assert lib.llm_qcache_shared_workspace(cache(), 1, 1, 1, 1, None) == ARG


def book(table=P, length=P << 8, rows=4, per=8, pages=64):
    return ctypes.byref(pkg.LlmPages(table, length, rows, per, pages))


def test_page_tables_refuse_bad_arguments(lib):
    n = ctypes.c_uint64()
    bad = [(dict(table=None), ARG), (dict(length=None), ARG), (dict(table=P + 2), ARG), (dict(rows=0), CONFIG), (dict(per=0), CONFIG),
           (dict(pages=0), CONFIG), (dict(pages=(1 << 28) + 1), CONFIG), (dict(rows=1 << 20, per=1 << 12), CONFIG), (dict(per=(1 << 24) + 1), CONFIG)]
    for kw, code in bad:
        assert lib.llm_pages_workspace(book(**kw), ctypes.byref(n)) == code, kw
    assert lib.llm_pages_workspace(book(), ctypes.byref(n)) == pkg.LLM_OK
    need = n.value
    to = dict(table=P << 4, length=P << 10)

    def update(x=None, y=None, parent=None, length=None, moves=P, counts=P, ws=P, nbytes=need, status=None):
        return lib.llm_pages_update(x or book(), y or book(**to), parent, length, moves, counts, ws, nbytes, status, None)

    def compact(x=None, y=None, moves=P, counts=P, ws=P, nbytes=need, status=None):
        return lib.llm_pages_compact(x or book(), y or book(**to), moves, counts, ws, nbytes, status, None)

    for call in (update, compact):
        for kw, code in bad:
            assert call(x=book(**kw)) == code, kw
        for kw in (dict(rows=5), dict(per=9), dict(pages=65)):
            assert call(y=book(**{**to, **kw})) == CONFIG, kw
        # tables and lengths that overlap, by an end
        for kw in (dict(table=P), dict(table=P + 4 * 31), dict(table=P - 4), dict(length=P << 8), dict(length=(P << 8) + 12),
                   dict(table=(P << 8) - 4), dict(length=P + 124)):
            assert call(y=book(**{**to, **kw})) == ARG, kw
        for kw in (dict(moves=None), dict(counts=None), dict(moves=P + 1), dict(counts=P + 2), dict(ws=None), dict(ws=P + 2),
                   dict(nbytes=need - 1), dict(status=P + 1)):
            assert call(**kw) == ARG, kw
    assert update(parent=P + 2) == ARG and update(length=P + 2) == ARG


def test_page_copies_refuse_bad_arguments(lib):
    def copy(c=None, n=1, moves=P, m=1, counts=None, status=None):
        return lib.llm_qcache_copy_pages(c or cache(), n, moves, m, counts, status, None)
    for kw, code in CACHES:
        assert copy(c=cache(**kw)) == code, kw
    for kw in (dict(n=0), dict(moves=None), dict(m=0), dict(m=-1), dict(moves=P + 2), dict(counts=P + 1), dict(status=P + 2), dict(m=1 << 30)):
        assert copy(**kw) == ARG, kw
    assert copy(c=cache(max_seq=80)) == CONFIG
    one = dict(k=P, v=P, k_scale=P, v_scale=P, rows=2, kv_heads=2, max_seq=128, head=64)
    for kw in (dict(rows=3), dict(kv_heads=1), dict(max_seq=192), dict(head=128)):
        two = (pkg.LlmQcache * 2)(*[pkg.LlmQcache(*d.values()) for d in (one, {**one, **kw})])
        assert lib.llm_qcache_copy_pages(two, 2, P, 1, None, None, None) == CONFIG, kw
    assert lib.llm_copy_pages(None, P, 1) == ARG


def test_sampling_refuses_bad_arguments(lib):
    def draw(logits=P, stride=100, B=2, V=100, temp=P, k=P, p=P, min_p=P, u=P, ids=P, status=None):
        return lib.llm_sample_rows(logits, stride, B, V, temp, k, p, min_p, u, ids, status, None)
    for kw, code in [(dict(logits=None), ARG), (dict(u=None), ARG), (dict(ids=None), ARG), (dict(B=0), BATCH), (dict(B=(1 << 24) + 1), BATCH),
                     (dict(V=0), ARG), (dict(V=524281, stride=524281), ARG), (dict(stride=99), ARG), (dict(stride=-100), ARG)]:
        assert draw(**kw) == code, kw
    for name in ("logits", "temp", "k", "p", "min_p", "u", "ids", "status"):
        assert draw(**{name: P + 2}) == ARG, name
    assert b"aligned" in lib.llm_last_error(None)


def test_the_plain_updates_keep_what_rows_hold():
    # random forks, rewinds, growth and frees: every row's kept positions stay readable through the new table, no two
    # rows can write one page, and a compaction leaves the front of the pool in use
    rng = np.random.default_rng(5)
    for _ in range(60):
        R, per, pages = int(rng.integers(1, 9)), int(rng.integers(1, 6)), int(rng.integers(1, 60))
        table, length = [[-1] * per for _ in range(R)], [0] * R
        data = {}                                        # (page, place) -> what was written there
        seen = [[] for _ in range(R)]                    # what each row should read
        for step in range(8):
            parent = rng.integers(-1, R, R)
            new = rng.integers(0, per * 64 + 1, R)
            got = ref.update(table, length, pages, parent, new)
            if got is None:
                continue
            table, length, moves, (n, used) = got
            assert n == len(moves) and not {a for a, _ in moves} & {b for _, b in moves} and len({b for _, b in moves}) == n
            for a, b in moves:
                for i in range(64):
                    data[b, i] = data.get((a, i))
            seen = [seen[p][:m] if p >= 0 else [] for p, m in zip(parent, new)]
            for r in range(R):
                assert [data.get((table[r][i // 64], i % 64)) for i in range(len(seen[r]))] == seen[r]
                for i in range(len(seen[r]), length[r]):
                    data[table[r][i // 64], i % 64] = (step, r, i)
                    seen[r].append((step, r, i))
            for r in range(R):
                assert [data[table[r][i // 64], i % 64] for i in range(length[r])] == seen[r]
            table2, _, moves, (n, held) = ref.compact(table, length, pages)
            assert held == used and {x for t in table2 for x in t if x >= 0} == set(range(used))
