"""Verification of drafted tokens on the GPU (llm_verify) against the exact definition in
tests/qcache_ref.py: ids and counts are integers and must be equal."""
import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
from tests import qcache_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def run(p, q, drafts, u, count=None):
    B, S = drafts.shape
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    ids = torch.full((B, S + 1), -7, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    pkg.llm_verify(dev(p), dev(q), dev(drafts.astype(np.int32)), dev(u.astype(np.float32)), ids, acc,
                   count=None if count is None else dev(np.asarray(count, np.int32)),
                   stream=torch.cuda.current_stream().cuda_stream)
    return ids.cpu().numpy(), acc.cpu().numpy()


def check(p, q, drafts, u, count=None):
    ids, acc = run(p, q, drafts, u, count)
    for b in range(len(drafts)):
        want = ref.verify(p[b], None if q is None else q[b], drafts[b], None if count is None else count[b], u[b])
        assert (ids[b].tolist(), int(acc[b])) == want, b
    return ids, acc


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (2, 1, 3), (5, 4, 7), (3, 2, 130), (4, 3, 1000), (2, 5, 49152), (1, 7, 50001),
                                   (2, 2, 128256), (9, 13, 2048), (1, 1, 262147)])
def test_ids_equal_the_definition(B, S, V, drawn):
    rng = np.random.default_rng(B * 1000 + V)
    logits = rng.standard_normal((B, S + 1, V)) * 3
    p = softmax(logits)
    near = logits[:, :S] + rng.standard_normal((B, S, V)) * 0.3
    q = softmax(near) if drawn else None
    drafts = np.array([[rng.choice(V, p=softmax(near[b, i]).astype(np.float64) / softmax(near[b, i]).astype(np.float64).sum())
                        for i in range(S)] for b in range(B)])
    u = (rng.integers(0, 1 << 24, (B, S + 1)) / (1 << 24)).astype(np.float32)
    check(p, q, drafts, u)
    check(p, q, drafts, u, count=[(b * 2 + 1) % (S + 1) for b in range(B)])
    # the ends of the draw: 0 and the largest float below 1
    u[:, S] = np.where(np.arange(B) % 2, np.float32(0), np.nextafter(np.float32(1), np.float32(0)))
    check(p, q, drafts, u)
    u[:, :S] = 0.999
    check(p, q, drafts, u)


def test_edges():
    V, S = 64, 3
    rng = np.random.default_rng(5)
    p = softmax(rng.standard_normal((6, S + 1, V)))
    q = p[:, :S].copy()                       # p == q: always kept, and where not, nothing is left over
    d = rng.integers(0, V, (6, S))
    u = np.full((6, S + 1), 0.5, np.float32)
    ids, acc = check(p, q, d, u)
    assert (acc == S).all()
    d2 = d.copy()
    d2[0, 0], d2[1, 1], d2[2, 2], d2[3, 0] = -1, V, 1 << 30, -(1 << 31)
    ids, acc = check(p, q, d2, u)             # ids outside the vocabulary are never kept
    assert acc[:4].tolist() == [0, 1, 2, 0]
    check(p, None, d2, u)
    zero = np.zeros_like(p)
    ids, acc = check(zero, None, d, u)        # no weight at all
    assert (acc == 0).all() and (ids[:, 0] == 0).all()
    one = np.zeros_like(p)
    one[:, :, 17] = 1.0                       # one-hot targets (greedy)
    ids, acc = check(one, None, np.full((6, S), 17), u)
    assert (acc == S).all() and (ids == 17).all()
    ids, acc = check(one, None, np.where(np.arange(S) == 1, 3, 17) * np.ones((6, 1), int), u)
    assert (acc == 1).all() and (ids[:, 1] == 17).all()
    sick = p.copy()
    sick[:, 0, ::3] = np.nan
    sick[:, 0, 1::3] = -1.0
    check(sick, q, d, u)
    sick[:, 0] = np.inf
    run(sick, q, d, u)
    # u outside [0, 1) cannot lead outside the vocabulary
    ids, acc = run(p, q, d, np.full((6, S + 1), 7.0, np.float32), count=[0] * 6)
    assert ((ids[:, 0] >= 0) & (ids[:, 0] < V)).all()
    ids, acc = run(p, q, d, np.full((6, S + 1), np.nan, np.float32), count=[-3, 0, 9, 1, 2, 3])
    assert ((ids[:, 0] >= 0) & (ids[:, 0] < V)).all()


def test_rows_that_start_off_16_byte_boundaries():
    # contiguous tensors at odd offsets of their storage
    rng = np.random.default_rng(6)
    B, S, V = 3, 2, 1003
    p, q = softmax(rng.standard_normal((B, S + 1, V)) * 3), softmax(rng.standard_normal((B, S, V)) * 3)
    d = rng.integers(0, V, (B, S)).astype(np.int32)
    u = (rng.integers(0, 1 << 24, (B, S + 1)) / (1 << 24)).astype(np.float32)

    def off(a, by):
        flat = torch.zeros(a.size + by, dtype=torch.from_numpy(a).dtype, device="cuda")
        flat[by:] = torch.from_numpy(a).cuda().reshape(-1)
        return flat[by:].view(a.shape)

    ids, acc = off(np.full((B, S + 1), -7, np.int32), 1), off(np.full(B, -7, np.int32), 3)
    pkg.llm_verify(off(p, 1), off(q, 3), off(d, 1), off(u, 2), ids, acc, stream=torch.cuda.current_stream().cuda_stream)
    for b in range(B):
        assert (ids[b].tolist(), int(acc[b])) == ref.verify(p[b], q[b], d[b], None, u[b])


def test_tokens_are_distributed_like_the_target():
    # the first token of many independent rows: each id's frequency is binomial around p
    V, B = 11, 40000
    rng = np.random.default_rng(8)
    pt, qt = softmax(rng.standard_normal((2, V)) * 1.5), softmax(rng.standard_normal((1, V)) * 1.5)
    p, q = np.broadcast_to(pt, (B, 2, V)).copy(), np.broadcast_to(qt, (B, 1, V)).copy()
    u = (rng.integers(0, 1 << 24, (B, 2)) / (1 << 24)).astype(np.float32)
    drafts = rng.choice(V, size=(B, 1), p=qt[0].astype(np.float64) / qt[0].astype(np.float64).sum())
    ids, _ = run(p, q, drafts, u)
    freq = np.bincount(ids[:, 0], minlength=V) / B
    # five standard deviations of a binomial frequency
    assert (np.abs(freq - pt[0]) <= 5 * np.sqrt(pt[0] * (1 - pt[0]) / B)).all(), (freq, pt[0])


def test_captured_call_replays():
    V, S, B = 1000, 2, 3
    rng = np.random.default_rng(9)
    p, q = softmax(rng.standard_normal((B, S + 1, V))), softmax(rng.standard_normal((B, S, V)))
    tp, tq = torch.from_numpy(p).cuda(), torch.from_numpy(q).cuda()
    d = torch.zeros(B, S, dtype=torch.int32, device="cuda")
    u = torch.zeros(B, S + 1, device="cuda")
    ids, acc = torch.zeros(B, S + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        pkg.llm_verify(tp, tq, d, u, ids, acc, stream=torch.cuda.current_stream().cuda_stream)
    for k in range(4):
        dn = rng.integers(0, V, (B, S))
        un = rng.random((B, S + 1)).astype(np.float32)
        d.copy_(torch.from_numpy(dn.astype(np.int32)))
        u.copy_(torch.from_numpy(un))
        gr.replay()
        torch.cuda.synchronize()
        for b in range(B):
            assert (ids[b].tolist(), int(acc[b])) == ref.verify(p[b], q[b], dn[b], None, un[b])


@pytest.mark.parametrize("V", [5, 7, 64, 1000, 50001])
@pytest.mark.parametrize("big", [np.inf, 1e30, 3.0])
def test_rows_that_are_no_probabilities_draw_an_id_of_the_vocabulary(V, big):
    # weights above 1 count as 1: up to seven of them are drawn from as defined, more give some id
    rng = np.random.default_rng(V)
    B, S = 16, 3
    p = np.full((B, S + 1, V), big, np.float32)
    q = softmax(rng.standard_normal((B, S, V)))
    d = rng.integers(0, V, (B, S))
    kept = np.arange(B) % (S + 1)
    d[np.arange(B), np.minimum(kept, S - 1)] = np.where(kept < S, -1, d[np.arange(B), S - 1])   # lost there, or nowhere
    u = (rng.integers(0, 1 << 24, (B, S + 1)) / (1 << 24)).astype(np.float32)
    for draft in (q, None):
        ids, acc = run(p, draft, d, u)
        assert np.array_equal(acc, kept)
        for b in range(B):
            r = kept[b]
            assert ids[b, :r].tolist() == d[b, :r].tolist() and (ids[b, r + 1:] == -1).all()
            assert 0 <= ids[b, r] < V
            if V <= 7:
                assert (ids[b].tolist(), r) == ref.verify(p[b], None if draft is None else draft[b], d[b], None, u[b])
