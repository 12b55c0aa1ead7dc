"""One token per row with settings of its own (llm_sample_rows) on the GPU against the definition in Python
integers (tests/shared_ref.py): ids must be equal."""
import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
from tests import shared_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def draw(v, temp, k, p, min_p, u, stream=None):
    dev = lambda x, t: None if x is None else torch.as_tensor(np.asarray(x, t)).cuda()  # noqa: E731
    logits = v if isinstance(v, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(v, np.float32)).cuda()
    ids, status = torch.full((logits.shape[0],), -5, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pkg.llm_sample_rows(logits, dev(temp, np.float32), dev(u, np.float32), ids, k=dev(k, np.int32), p=dev(p, np.float32),
                        min_p=dev(min_p, np.float32), status=status, stream=stream)
    return ids.tolist(), int(status)


def check(v, temp, k, p, min_p, u):
    v = np.asarray(v, np.float32)
    got, status = draw(v, temp, k, p, min_p, u)
    want = [ref.sample(v[b], np.float32(temp[b]), int(k[b]), np.float32(p[b]), np.float32(min_p[b]), np.float32(u[b])) for b in range(len(v))]
    assert status == 0 and got == want, [(b, x, y) for b, (x, y) in enumerate(zip(got, want)) if x != y][:5]


def settings(rng, B, V):
    return (rng.choice([0.0, 0.3, 0.7, 1.0, 1.7, 30.0], B), rng.choice([1, 2, 5, 40, V // 2 + 1, V, V + 7, 1 << 30], B),
            rng.choice([1.0, 0.999, 0.9, 0.5, 1e-6, 1e-9], B), rng.choice([0.0, 0.0, 1e-4, 0.05, 0.5, 1.0], B),
            np.floor(rng.random(B) * 2 ** 24) / 2 ** 24)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 33, 511, 4096, 4099, 20001])
@pytest.mark.parametrize("spread", [0.0, 1e-3, 2.5, 40.0])
def test_ids_equal_the_definition(V, spread):
    rng = np.random.default_rng(V)
    B = 24 if V > 4000 else 60
    v = rng.standard_normal((B, V)) * spread
    if V > 2:
        v[::3] = np.round(v[::3])        # ties
    check(v, *settings(rng, B, V))


@pytest.mark.parametrize("V", [49152, 128256, 524280])
def test_large_vocabularies(V):
    rng = np.random.default_rng(V)
    B = 4
    check(rng.standard_normal((B, V)) * 2.5, [1.0, 0.8, 0.0, 2.0], [V, 50, 1, V // 3], [0.95, 1.0, 1.0, 0.9], [0, 0, 0, 1e-3], rng.random(B))


@pytest.mark.parametrize("B,V", [(20, 32771), (39, 16387), (153, 2049), (40, 100003), (3, 65537)])
def test_numbers_of_rows_and_ids(B, V):
    # rows take fewer CTAs the more there are, and more where a part of a row has no room on chip
    rng = np.random.default_rng(B)
    check(rng.standard_normal((B, V)) * rng.choice([0.5, 2.5, 6.0], (B, 1)), *settings(rng, B, V))


def test_places_whose_candidates_just_fit_or_just_do_not():
    # n logits in one of the 2048 steps into which the distances are sorted first, n about the room for a place's
    # and for all places' candidates, the rest far apart
    rng = np.random.default_rng(6)
    for n in (1000, 1023, 1024, 1025, 2046, 2047, 2048, 2049, 2100):
        V = n + 500
        v = np.concatenate([[0.0], np.linspace(-20, -1, V - n - 1), -0.5 - 1e-4 * rng.random(n)])
        v = np.stack([rng.permutation(v) for _ in range(6)])
        check(v, [1.0] * 6, [V, n // 2, n + 1, V, 3, V], [0.9, 1.0, 0.5, 1.0, 0.9, 0.3], [0, 0, 0.1, 0.6, 0.6065, 0.60651], rng.random(6))


@pytest.mark.parametrize("k", [1, 2, 1000, 1023, 1024, 1025, 2000])
def test_top_k_about_the_room_for_its_candidates(k):
    # as many candidates in the k-th one's step as just fit with those before, or do not; with each of the other settings
    rng = np.random.default_rng(k)
    V = 6000
    for n in (1, 900, 1500, 2500):
        v = np.concatenate([np.linspace(0, -2, k - 1), np.full(n, -2.5), np.linspace(-9, -25, V - n - k + 1)])
        v = np.stack([rng.permutation(v) for _ in range(6)])
        check(v, [1.0, 0.7, 1.3, 1.0, 0.0, 1.0], [k] * 6, [1.0, 0.9, 1.0, 0.5, 1.0, 0.999], [0, 0, np.exp(-2.5), 0.3, 0, 0.0820849], rng.random(6))


def test_equal_logits_and_logits_within_a_step():
    # every candidate at one distance, more than are put in order at once; and distances of a few units of 2^-27
    V, rng = 20000, np.random.default_rng(1)
    u = np.array([0.0, 0.25, 0.5, 1 - 2.0 ** -24, 0.99, 0.3])
    check(np.full((6, V), 3.25), [1.0] * 6, [V, V, 100, 7000, V, 1], [1, 0.5, 1, 0.3, 1e-5, 1], [0, 0.3, 1, 0, 0, 0], u)
    near = 1.0 + rng.integers(0, 7, (6, V)) * 2.0 ** -23
    check(near, [1.0] * 6, [V, V, 100, 7000, V, 1], [1, 0.5, 1, 0.3, 1e-5, 1], [0, 0.3, 1, 0, 0, 0], u)
    check(rng.standard_normal((6, V)) * 1e-6, [1e-3, 1.0, 50.0, 1e4, 1e30, 1e-30], [V, V, 100, 7000, V, 9], [1, 0.5, 1, 0.3, 0.9, 1], [0] * 6, u)
    # half the row at one distance far from the top, the rest beyond every weight
    v = np.full((6, V), -1e4)
    v[:, ::2] = -3.0
    v[:, 77] = 0.0
    check(v, [1.0] * 6, [V, V, 100, 7000, V, 1], [1, 0.9, 1, 0.9999, 0.99, 1], [0, 0, 0, 0.01, 0, 0], u)


def test_infinities_and_nan():
    inf, nan = np.inf, np.nan
    v = np.array([[nan, 1.0, 2.0, -inf, nan, 0.5], [-inf] * 6, [nan] * 6, [nan, -inf, nan, -inf, nan, -inf], [1, inf, 3, inf, -inf, nan],
                  [-inf, -inf, -1e30, -inf, nan, -inf], [3e38, -3e38, 3e38, 1, 2, 3], [-0.0, 0.0, -0.0, 0.0, -1, -1]], np.float32)
    for temp in (0.0, 1e-38, 0.7, 1e38):
        for u in (0.0, 0.4, 0.999):
            for k in (1, 2, 6):
                check(v, [temp] * 8, [k] * 8, [0.9] * 8, [0.0] * 8, [u] * 8)


def test_settings_out_of_range_give_no_id_and_are_reported():
    v = np.random.default_rng(2).standard_normal((3, 300)).astype(np.float32)
    fine = dict(temp=1.0, k=5, p=0.9, min_p=0.1, u=0.5)
    nan = float("nan")
    want = [ref.sample(x, np.float32(1), 5, np.float32(0.9), np.float32(0.1), np.float32(0.5)) for x in v]
    for name, bad in [("temp", -1.0), ("temp", nan), ("temp", float("inf")), ("k", 0), ("k", -3), ("p", 0.0), ("p", 1.5), ("p", nan),
                      ("min_p", -0.1), ("min_p", 1.1), ("min_p", nan), ("u", 1.0), ("u", -0.5), ("u", nan)]:
        args = {n: [x] * 3 for n, x in fine.items()}
        args[name][1] = bad
        got, status = draw(v, args["temp"], args["k"], args["p"], args["min_p"], args["u"])
        assert status == pkg.LLM_ERR_ARG and got == [want[0], -1, want[2]], name
    # a greedy row looks at its temperature alone
    got, status = draw(v, [0.0] * 3, [0] * 3, [nan] * 3, [2.0] * 3, [5.0] * 3)
    assert status == 0 and got == v.argmax(-1).tolist()


def test_left_out_settings_and_rows_of_a_wider_tensor():
    rng = np.random.default_rng(3)
    wide = torch.from_numpy(rng.standard_normal((5, 1009)).astype(np.float32)).cuda()
    for lo, hi in ((0, 1000), (1, 1001), (3, 1009)):
        v = wide[:, lo:hi]
        u = rng.random(5)
        got, status = draw(v, None, None, None, None, u)
        x = v.cpu().numpy()
        assert status == 0 and got == [ref.sample(x[b], np.float32(1), hi, np.float32(1), np.float32(0), np.float32(u[b])) for b in range(5)]
    for bad in (dict(logits=wide.double()), dict(logits=wide[:, ::2]), dict(logits=wide[0]), dict(u=torch.zeros(4, device="cuda")),
                dict(ids=torch.zeros(5, device="cuda")), dict(temp=torch.zeros(5, device="cuda").double()),
                dict(k=torch.zeros(5, device="cuda")), dict(ids=None)):
        args = dict(logits=wide, temp=None, u=torch.zeros(5, device="cuda"), ids=torch.zeros(5, dtype=torch.int32, device="cuda"))
        args.update(bad)
        with pytest.raises(pkg.LlmError):
            pkg.llm_sample_rows(**args)


def test_draws_follow_the_distribution():
    # 2^13 evenly spaced draws of a row: every id as often as its share says, within one of each end of its run
    V, n = 300, 1 << 13
    v = torch.from_numpy(np.random.default_rng(4).standard_normal(V).astype(np.float32) * 2).cuda().expand(n, V).contiguous()
    u = (np.arange(n) + 0.5) / n
    got, _ = draw(v, [0.9] * n, [100] * n, [0.97] * n, [0.001] * n, u)
    w = np.exp(v[0].double().cpu().numpy() / 0.9)
    order = np.argsort(-w)[:100]
    c = np.cumsum(w[order]) / w[order].sum()
    kept = order[: int(np.searchsorted(c, 0.97)) + 1]
    kept = kept[w[kept] >= 0.001 * w.max()]
    share = w[kept] / w[kept].sum()
    count = np.bincount(got, minlength=V)
    assert set(np.flatnonzero(count)) <= set(kept)
    assert (np.abs(count[kept] - share * n) <= 1.01).all()


def test_captured_calls_and_other_streams():
    rng = np.random.default_rng(5)
    V, B = 5000, 3
    v = torch.from_numpy(rng.standard_normal((B, V)).astype(np.float32)).cuda()
    temp, u, ids = torch.ones(B, device="cuda"), torch.zeros(B, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    pkg.llm_sample_rows(v, temp, u, ids)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.llm_sample_rows(v, temp, u, ids)
    for x in (0.1, 0.6, 0.95):
        u.fill_(x)
        v.copy_(torch.from_numpy(rng.standard_normal((B, V)).astype(np.float32)))
        g.replay()
        want = [ref.sample(v[b].cpu().numpy(), np.float32(1), V, np.float32(1), np.float32(0), np.float32(x)) for b in range(B)]
        assert ids.tolist() == want
    # two streams at once, no workspace between them
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    out = []
    for i in range(20):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                x = torch.full_like(ids, -9)
                pkg.llm_sample_rows(v, temp, u, x)
                out.append(x)
    torch.cuda.synchronize()
    assert all(x.tolist() == want for x in out)
