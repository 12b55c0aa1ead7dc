"""Refusals of the 8-bit cache and verification entries that the host makes before any GPU work, and the
64-bit definitions the GPU tests use (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
from llama_architecture_kv_gb300 import build as pkg_build
from tests import qcache_ref as ref

ARG, CONFIG, BATCH = pkg.LLM_ERR_ARG, pkg.LLM_ERR_CONFIG, pkg.LLM_ERR_BATCH
P = 0x10000  # an aligned address that is never followed: every case below is refused on the host


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return pkg.lib()


def cache(**kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, rows=2, kv_heads=2, max_seq=128, head=64)
    d.update(kw)
    return ctypes.byref(pkg.LlmQcache(*[d[n] for n, _ in pkg.LlmQcache._fields_]))


def write(lib, c=None, k=P, v=P, dtype=1, stride=128, B=2, S=3, pos=P, count=None, table=None, pages=0, status=None):
    return lib.llm_qcache_write(c or cache(), k, v, dtype, stride, B, S, pos, count, table, pages, status, None)


def read(lib, c=None, k=P, v=P, dtype=1, stride=128, B=2, S=3, pos=P, count=None, table=None, pages=0, status=None):
    return lib.llm_qcache_read(c or cache(), B, S, pos, count, table, pages, k, v, dtype, stride, status, None)


CACHES = [(dict(k=None), ARG), (dict(v_scale=None), ARG), (dict(k=P + 8), ARG), (dict(k_scale=P + 2), ARG),
          (dict(rows=0), CONFIG), (dict(kv_heads=0), CONFIG), (dict(head=48), CONFIG), (dict(max_seq=100), CONFIG),
          (dict(max_seq=0), CONFIG), (dict(max_seq=-16), CONFIG), (dict(rows=1 << 20, max_seq=1 << 20), CONFIG)]
ROWS = [(dict(B=0), BATCH), (dict(B=3), BATCH), (dict(S=0), ARG), (dict(pos=None), ARG), (dict(pos=P + 1), ARG),
        (dict(S=1 << 30), ARG), (dict(dtype=2), ARG),
        (dict(k=None), ARG), (dict(v=P + 4), ARG), (dict(stride=120), ARG), (dict(stride=132), ARG),
        (dict(table=P, pages=0), ARG), (dict(table=P, pages=1 << 30), ARG), (dict(status=P + 2), ARG),
        (dict(table=P, pages=1 << 24), ARG), (dict(table=P, pages=-1), ARG)]


@pytest.mark.parametrize("call", [write, read])
def test_cache_calls_refuse_bad_arguments(lib, call):
    for kw, code in CACHES:
        assert call(lib, c=cache(**kw)) == code, kw
    for kw, code in ROWS:
        assert call(lib, **kw) == code, kw
    # pages need whole pages per row
    assert call(lib, c=cache(max_seq=80), table=P, pages=1) == CONFIG
    assert lib.llm_last_error(None)


@pytest.mark.parametrize("call", [write, read])
def test_cache_calls_refuse_more_warps_than_a_launch_has(lib, call):
    # blocks that 2^31 - 1 tokens can touch times 16 heads, and the neighbours of the bound of 2^30
    wide = dict(rows=1, kv_heads=16, max_seq=16)
    for S in ((1 << 31) - 1, (1 << 31) - 16, 1 << 30, ((1 << 26) - 2) * 16 + 2):
        assert call(lib, c=cache(**wide), B=1, S=S, stride=1024) == ARG, S
        assert b"too large" in lib.llm_last_error(None)


def test_attention_refuses_bad_arguments(lib):
    def attend(c=None, q=P, dtype=1, q_stride=256, group=2, B=2, S=1, length=P, count=None, table=None, pages=0,
               scale=0.125, out=P, out_stride=256, ws=P, nbytes=1 << 40, status=None):
        return lib.llm_qcache_attend(c or cache(), q, dtype, q_stride, group, B, S, length, count, table, pages, scale,
                                     out, out_stride, ws, nbytes, status, None)
    for kw, code in CACHES:
        assert attend(c=cache(**kw)) == code, kw
    for kw, code in [(dict(group=0), CONFIG), (dict(group=17), CONFIG), (dict(q=None), ARG), (dict(out=None), ARG),
                     (dict(q_stride=255), ARG), (dict(out_stride=248), ARG), (dict(dtype=-1), ARG),
                     (dict(length=None), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
                     (dict(B=0), BATCH), (dict(B=3), BATCH), (dict(S=0), ARG)]:
        assert attend(**kw) == code, kw
    assert attend(c=cache(head=128), group=9, q_stride=4096, out_stride=4096) == CONFIG  # group * head > 1024
    n = ctypes.c_uint64()
    for kw, args, code in [(dict(rows=0), (1, 1, 1), CONFIG), (dict(), (0, 1, 1), CONFIG), (dict(), (1, 0, 1), BATCH),
                           (dict(), (1, 1, 0), ARG)]:
        assert lib.llm_qcache_workspace(cache(**kw), *args, ctypes.byref(n)) == code
    assert lib.llm_qcache_workspace(cache(), 1, 1, 1, None) == ARG


def test_verification_refuses_bad_arguments(lib):
    def verify(p=P, q=None, drafts=P, count=None, B=1, S=1, V=8, u=P, ids=P, accepted=P):
        return lib.llm_verify(p, q, drafts, count, B, S, V, u, ids, accepted, None)
    for kw, code in [(dict(p=None), ARG), (dict(drafts=None), ARG), (dict(u=None), ARG), (dict(ids=None), ARG),
                     (dict(accepted=None), ARG), (dict(B=0), BATCH), (dict(S=0), ARG), (dict(S=65536), ARG),
                     (dict(V=0), ARG), (dict(V=(1 << 30) + 1), ARG), (dict(B=(1 << 24) + 1), BATCH), (dict(p=P + 2), ARG), (dict(ids=P + 1), ARG)]:
        assert verify(**kw) == code, kw


def test_create_refuses_an_unknown_cache_type(lib):
    from synth.configs import TINY
    c = pkg.config(TINY, 1, 16, cache_type=2)
    h = ctypes.c_void_p()
    buf = np.zeros(4, np.uint8)
    n = pkg.llm_weight_count(c) * 4
    assert lib.llm_create(ctypes.byref(c), buf.ctypes.data, n, 0, None, ctypes.byref(h)) == CONFIG
    # the types that exist pass this check (and fail on the blob's size, before any GPU work)
    for t in (pkg.LLM_CACHE_MODEL, pkg.LLM_CACHE_E4M3):
        c = pkg.config(TINY, 1, 16, cache_type=t)
        assert lib.llm_create(ctypes.byref(c), buf.ctypes.data, n + 4, 0, None, ctypes.byref(h)) == pkg.LLM_ERR_WEIGHTS_SIZE


def test_python_wrappers_refuse_tensors_of_the_cpu():
    torch = pytest.importorskip("torch")
    with pytest.raises(pkg.LlmError):
        pkg.QCache(torch.zeros(1, 1, 16, 16, dtype=torch.uint8), torch.zeros(1, 1, 16, 16, dtype=torch.uint8),
                   torch.zeros(1, 1, 1), torch.zeros(1, 1, 1))
    with pytest.raises(pkg.LlmError):
        pkg.llm_verify(torch.zeros(1, 2, 4), None, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2),
                       torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


# ---- the definitions themselves ----

def test_reference_codes_round_to_nearest_even():
    assert ref.VALUE[0x7e] == 448 and ref.VALUE[1] == 2.0 ** -9 and ref.VALUE[8] == 2.0 ** -6
    assert np.isnan(ref.VALUE[0x7f]) and np.isnan(ref.VALUE[0xff])
    codes = np.array([c for c in range(256) if (c & 127) != 127], np.uint8)
    assert np.array_equal(ref.encode(ref.VALUE[codes]), codes)  # every code is a fixed point (-0 too)
    assert ref.encode([1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10]).tolist() == [0x38, 0x3a, 0xb8, 0, 2]
    x = np.random.default_rng(1).uniform(-448, 448, 2000)
    err = np.abs(ref.VALUE[ref.encode(x)] - x)
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10)).all()


def test_reference_scale_places_the_largest_value():
    for top in (448.0, 448.0 + 2.0 ** -14, 1.0, 1e-30, 3.4e38, 0.0, 1e-44):
        s = ref.need_scale(np.array([top, -top / 2]))
        assert top / s <= 448 and (s == 2.0 ** -126 or top / (s / 2) > 448)
    assert np.isnan(ref.need_scale(np.array([1.0, np.inf])))


def test_reference_verification_keeps_the_target_distribution():
    # all (draft, draw) outcomes of a tiny case, weighted by their probabilities, sum to p
    p = np.array([[0.5, 0.25, 0.125, 0.125], [0.25, 0.25, 0.25, 0.25]], np.float32)
    q = np.array([[0.125, 0.5, 0.25, 0.125]], np.float32)
    first = np.zeros(4)
    grid = (np.arange(64) + 0.5) / 64
    for x in range(4):
        for u0 in grid:
            for u1 in grid:
                ids, r = ref.verify(p, q, [x], None, [u0, u1])
                first[ids[0]] += q[0, x] / 64 ** 2
    assert np.abs(first - p[0]).max() <= 1 / 32  # the grid's resolution
