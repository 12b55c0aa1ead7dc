"""Handles with an 8-bit cache (cache_type LLM_CACHE_E4M3) and verification steps.

What a step stores must be the quantisation of what a handle with a plain cache stores (layer 0, whose
keys and values depend on nothing the caches change); what its attention computes must be the attention
over the values read back; and the other entries must agree with the plain step.
"""
import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
import oracle
import synth
from synth import WORKLOADS, shrink
from synth.configs import TINY
from tests import qcache_ref as ref
from tests.test_gpu_qcache import attend_tolerance

pytestmark = pytest.mark.gpu

F32_TOL = 1e-4      # of the logit range, as the parity tests hold the f32 model
BF16_ABS = 3e-2     # absolute, bf16 weights
E4M3 = pkg.LLM_CACHE_E4M3
LLAMA8 = WORKLOADS["llama8b_b1"].shape

SHAPES = [
    # name, shape, rows, tc_min_batch
    ("f32_hd16", shrink(TINY, kv=2, g=2), 2, 0),
    ("f32_hd64_g3", shrink(TINY, kv=2, g=3, half=32, ffn=200, vocab=300), 2, 0),
    ("bf16_hd128_g4", shrink(LLAMA8, layers=2, kv=2, ffn=512, vocab=1000), 3, 0),
    ("bf16_hd64_g1_tc", shrink(LLAMA8, layers=2, kv=4, g=1, half=32, ffn=512, vocab=1000), 17, 1),
]


def make(shape, seed, B, cap, wstd=None, **kw):
    blob = synth.model_blob(shape, seed, wstd=wstd if wstd else (0.1 if not shape.bf16 else 0.02))
    return pkg.Model(shape, blob, max_batch=B, max_seq=cap, **kw)


def wide(x):
    """Cache elements (bf16 bits or f32) as float64."""
    return (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64) if x.dtype == np.uint16 else x.astype(np.float64)


def close(a, b, shape):
    err = float(np.max(np.abs(a - b)))
    return err <= (BF16_ABS if shape.bf16 else F32_TOL * float(b.max() - b.min()))


@pytest.mark.parametrize("name,shape,B,tc", SHAPES, ids=[s[0] for s in SHAPES])
def test_steps_store_the_quantised_keys_and_values(name, shape, B, tc):
    P, steps, cap = 37, 6, 96
    toks = synth.tokens(702, 0, B * (P + steps), shape.vocab).reshape(B, P + steps)
    plain, q8 = make(shape, 701, B, cap, tc_min_batch=tc), make(shape, 701, B, cap, tc_min_batch=tc, cache_type=E4M3)
    for g in (plain, q8):
        g.prefill(toks[:, :P], 0, logits=False)
        for s in range(steps):
            g.decode(toks[:, P + s], P + s)
    for b in (0, B - 1):
        k, v = plain.kv_export(0, b, 0, P + steps)
        want = ref.RefCache(1, shape.kv, cap // 16 * 16, shape.hd)
        kk, vv = (wide(x).swapaxes(0, 1)[None] for x in (k, v))
        want.write(kk[:, :P], vv[:, :P], [0])
        for s in range(steps):
            want.write(kk[:, P + s:P + s + 1], vv[:, P + s:P + s + 1], [P + s])
        wk, wv = want.values(None, 0, P + steps)
        gk, gv = q8.kv_export(0, b, 0, P + steps)
        assert np.array_equal(wide(gk), wk) and np.array_equal(wide(gv), wv)
        assert q8.filled(b) == P + steps
    plain.close()
    q8.close()


@pytest.mark.parametrize("name,shape,B,tc", SHAPES, ids=[s[0] for s in SHAPES])
def test_steps_of_rows_at_their_own_positions_store_across_block_and_tile_edges(name, shape, B, tc):
    # rows around position 128, the first of a block and of a tile among theirs
    P, steps, cap = 131, 14, 192
    toks = synth.tokens(712, 0, B * (P + steps), shape.vocab).reshape(B, P + steps)
    first = np.array([P - 5 * (b % 3) for b in range(B)])
    plain, q8 = make(shape, 711, B, cap, tc_min_batch=tc), make(shape, 711, B, cap, tc_min_batch=tc, cache_type=E4M3)
    logits, prompt = [], {}
    for g in (plain, q8):
        g.prefill(toks[:, :P], 0, logits=False)
        prompt = prompt or {b: g.kv_export(0, b, 0, P) for b in {0, 1, B - 1}}
        for s in range(steps):
            lg = g.decode_rows(np.ascontiguousarray(toks[np.arange(B), first + s]), first + s)
        logits.append(lg)
    for b, (k0, v0) in prompt.items():
        n = int(first[b]) + steps
        k, v = plain.kv_export(0, b, 0, n)
        k0, v0, kk, vv = (wide(x).swapaxes(0, 1)[None] for x in (k0, v0, k, v))
        want = ref.RefCache(1, shape.kv, cap, shape.hd)
        want.write(k0, v0, [0])               # (the steps rewrite its tokens from first[b] on)
        for p in range(int(first[b]), n):
            want.write(kk[:, p:p + 1], vv[:, p:p + 1], [p])
        wk, wv = want.values(None, 0, n)
        gk, gv = q8.kv_export(0, b, 0, n)
        assert np.array_equal(wide(gk), wk) and np.array_equal(wide(gv), wv)
    # a step's graph replayed: the same bits
    again = q8.decode_rows(np.ascontiguousarray(toks[np.arange(B), first + steps - 1]), first + steps - 1)
    assert np.array_equal(again, logits[1])
    plain.close()
    q8.close()


@pytest.mark.parametrize("name,shape,B,tc", SHAPES, ids=[s[0] for s in SHAPES])
def test_attention_of_every_layer_is_that_over_the_values_read_back(name, shape, B, tc):
    n, cap = 150, 192
    toks = synth.tokens(712, 0, B * n, shape.vocab).reshape(B, n)
    g = make(shape, 711, B, cap, debug_trace=True, cache_type=E4M3)
    g.prefill(toks[:, :n - 1], 0, logits=False)
    g.decode(toks[:, n - 1], n - 1)
    for layer in range(shape.layers):
        qr, attn = g.trace(layer, "qr"), g.trace(layer, "attn")
        for b in (0, B - 1):
            k, v = (wide(x) for x in g.kv_export(layer, b, 0, n))
            c = ref.RefCache(1, shape.kv, cap, shape.hd)
            c.values = lambda table, row, m, first=0: (k, v)
            q = qr[b].astype(np.float64).reshape(1, 1, shape.heads, shape.hd)
            want, mag, sens, flat = c.attend(q, [n], scale=float(np.float32(1) / np.sqrt(np.float32(shape.hd))))
            got = attn[b].reshape(1, 1, shape.heads, shape.hd)
            assert (np.abs(got - want) <= attend_tolerance("f32", shape.hd, want, mag, sens, flat)).all(), (layer, b)
    g.close()


@pytest.mark.parametrize("name,shape,B,tc", SHAPES, ids=[s[0] for s in SHAPES])
def test_a_prefill_pass_attends_like_single_steps(name, shape, B, tc):
    # the last token of a prefill, again as a decode step over the cache that the prefill left (moved to
    # another handle by export and import, which keep every value)
    n, cap = 131, 192
    toks = synth.tokens(722, 0, B * n, shape.vocab).reshape(B, n)
    a, c = make(shape, 721, B, cap, tc_min_batch=tc, cache_type=E4M3), make(shape, 721, B, cap, cache_type=E4M3)
    lg = a.prefill(toks[:, :77], 0)          # two passes, the second starting inside a block
    lg = a.prefill(toks[:, 77:], 77)
    for layer in range(shape.layers):
        for b in range(B):
            k, v = a.kv_export(layer, b, 0, n - 1)
            c.kv_import(layer, b, 0, k, v)
            k2, v2 = c.kv_export(layer, b, 0, n - 1)
            assert np.array_equal(k, k2) and np.array_equal(v, v2)
    again = c.decode(toks[:, n - 1], n - 1)
    for b in range(B):
        assert close(again[b], lg[b], shape), b
    a.close()
    c.close()


@pytest.mark.parametrize("name,shape,B,tc", SHAPES[1:], ids=[s[0] for s in SHAPES[1:]])
def test_pages_rows_and_generation_agree_with_plain_steps(name, shape, B, tc):
    cap, n = 192, 70
    toks = synth.tokens(732, 0, B * (n + 1), shape.vocab).reshape(B, n + 1)
    one, two = make(shape, 731, B, cap, tc_min_batch=tc, cache_type=E4M3), make(shape, 731, B, cap, tc_min_batch=tc, cache_type=E4M3)
    per = cap // 64
    table = np.random.default_rng(733).permutation(B * per).astype(np.int32).reshape(B, per)
    for s in range(n):
        x = one.decode_paged(toks[:, s], np.full(B, s, np.int32), table)
        y = two.decode_rows(toks[:, s], np.full(B, s, np.int32))
        assert np.array_equal(x.view(np.uint32), y.view(np.uint32)), s
    # rows at their own positions, one of them rewound into a block
    pos = np.array([n - 11 * (b % 3) for b in range(B)], np.int32)
    x = two.decode_rows(toks[np.arange(B), pos], pos)
    assert np.isfinite(x).all()
    u = synth.uniforms(734, 0, 5 * B)
    two.prefill(toks[:, :n], 0, logits=False)
    ids = two.generate(toks[:, n], n, 5, 0.9, 20, 0.9, u)
    two.prefill(toks[:, :n], 0, logits=False)
    cur = toks[:, n]
    for s in range(5):
        cur = two.step(cur, n + s, 0.9, 20, 0.9, u[s * B:(s + 1) * B])
        assert np.array_equal(cur, ids[s]), s
    one.close()
    two.close()


def test_packed_prompts_agree_with_their_own_prefill():
    for name, shape, B, tc in SHAPES[1:]:
        cap = 128
        a = make(shape, 741, 2, cap, tc_min_batch=tc, cache_type=E4M3)
        t0, t1, t2 = (synth.tokens(742 + i, 0, m, shape.vocab) for i, m in enumerate((45, 20, 13)))
        # row 0: a prompt at 0..44; row 1: prompts at 0..19 and 37..49 (both end inside blocks)
        lg = a.prefill_packed(np.concatenate([t0, t1, t2]), [0] * 45 + [1] * 33,
                              list(range(45)) + list(range(20)) + list(range(37, 50)), [5] * 45 + [6] * 20 + [7] * 13,
                              [44, 64, 77])
        b = make(shape, 741, 2, cap, tc_min_batch=tc, cache_type=E4M3)
        for i, t in ((0, t0), (1, t1)):
            want = b.prefill(t[None], 0)[0]
            assert close(lg[i], want, shape), (name, i)
        # a prompt that ends inside a block whose later positions are filled is refused
        with pytest.raises(pkg.LlmError) as e:
            a.prefill_packed(t1[:5], [1] * 5, list(range(5)), [1] * 5, [4])
        assert e.value.status == pkg.LLM_ERR_POS_RANGE
        a.prefill_packed(t1[:16], [1] * 16, list(range(16)), [1] * 16, [15])  # a whole block is not
        with pytest.raises(pkg.LlmError) as e:
            a.kv_import(0, 0, 0, *a.kv_export(0, 0, 0, 20))
        assert e.value.status == pkg.LLM_ERR_POS_RANGE
        a.kv_import(0, 0, 0, *a.kv_export(0, 0, 0, 45))
        a.close()
        b.close()


# ---- verification steps ----

@pytest.mark.parametrize("cache", [pkg.LLM_CACHE_MODEL, E4M3], ids=["model", "e4m3"])
@pytest.mark.parametrize("name,shape,B,tc", SHAPES, ids=[s[0] for s in SHAPES])
def test_verification_steps_follow_the_model(name, shape, B, tc, cache):
    cap, n, S = 128, 21, 4
    toks = synth.tokens(762, 0, B * n, shape.vocab).reshape(B, n)
    kw = dict(tc_min_batch=tc, cache_type=cache, wstd=0.2 if not shape.bf16 else 0.06)
    g = make(shape, 761, B, cap, **kw)
    g.prefill(toks[:, :n - 1], 0, logits=False)
    greedy = g.generate(toks[:, n - 1], n - 1, S + 2).T.copy()         # [B][S + 2]
    u = np.full((B, S + 1), 0.5, np.float32)
    # greedy drafts that the model itself would draw are all kept, and one more token comes
    g.prefill(toks[:, :n - 1], 0, logits=False)
    block = np.concatenate([toks[:, n - 1:], greedy[:, :S]], 1)
    ids, acc, p = g.verify_step(block, np.full(B, n - 1), u)
    assert (acc == S).all() and np.array_equal(ids, greedy[:, :S + 1])
    assert np.array_equal(np.sort(p, -1)[..., -1], np.ones((B, S + 1))) and (p.sum(-1) == 1).all()
    # from there on the handle goes on after the kept drafts
    nxt = g.step(ids[:, S], n - 1 + S + 1)
    assert np.array_equal(nxt, greedy[:, S + 1])
    # a wrong draft ends the row's run there, rows at their own positions; the next step rewinds
    pos = np.array([n - 1 - (b % 2) * 3 for b in range(B)])
    g.prefill(toks[:, :n - 1], 0, logits=False)
    start = toks[np.arange(B), pos]
    chain = np.empty((B, S + 1), np.int32)
    cur = start
    for s in range(S + 1):
        cur = g.step_rows(cur, pos + s)
        chain[:, s] = cur
    wrong = chain.copy()
    at = np.arange(B) % S
    wrong[np.arange(B), at] = (wrong[np.arange(B), at] + 1) % shape.vocab
    ids, acc, p = g.verify_step(np.concatenate([start[:, None], wrong[:, :S]], 1), pos, u)
    assert np.array_equal(acc, at)
    for b in range(B):
        assert ids[b, :at[b] + 1].tolist() == chain[b, :at[b] + 1].tolist() and (ids[b, at[b] + 1:] == -1).all()
    # sampled drafts: the outcome is the definition's on the returned probabilities, and those are the
    # softmax of the model's logits
    rng = np.random.default_rng(763)
    q = rng.dirichlet(np.ones(shape.vocab), (B, S)).astype(np.float32)
    drafts = np.array([[rng.choice(shape.vocab) for _ in range(S)] for _ in range(B)], np.int32)
    uu = rng.random((B, S + 1)).astype(np.float32)
    g.prefill(toks[:, :n - 1], 0, logits=False)
    ids, acc, p = g.verify_step(np.concatenate([start[:, None], drafts], 1), pos, uu, temp=0.7, q=q)
    for b in range(B):
        assert (ids[b].tolist(), int(acc[b])) == ref.verify(p[b], q[b], drafts[b], None, uu[b])
    g.prefill(toks[:, :n - 1], 0, logits=False)
    lg = g.decode_rows(start, pos)
    want = np.exp((lg.astype(np.float64) - lg.max(-1, keepdims=True)) / 0.7)
    want /= want.sum(-1, keepdims=True)
    # a logit off by e moves a probability by at most exp(2 e / temp) - 1 of it
    e = BF16_ABS if shape.bf16 else F32_TOL * (lg.max(-1) - lg.min(-1)).max()
    assert (np.abs(p[:, 0] - want) <= want * np.expm1(2 * e / 0.7) + 1e-7).all()
    g.close()


def test_more_rows_than_one_activation_tile_through_the_head():
    # 70 rows are two tiles of the tensor-core head; on this vocabulary (as on the 8B shape's) the tile
    # height that fills the SMs best differs between one tile and two, and the head's map has one height
    shape = shrink(LLAMA8, layers=1, kv=1, g=2, ffn=256, vocab=128256)
    B, S, n = 14, 4, 9
    g = make(shape, 781, 80, 64, wstd=0.06)
    toks = synth.tokens(782, 0, 80 * n, shape.vocab).reshape(80, n)
    g.prefill(toks[:, :n - 1], 0, logits=False)
    chain = g.generate(toks[:, n - 1], n - 1, S + 1).T.copy()           # 80 rows in one step
    g.prefill(toks[:B, :n - 1], 0, logits=False)
    assert np.array_equal(g.generate(toks[:B, n - 1], n - 1, S + 1).T, chain[:B])
    g.prefill(toks[:B, :n - 1], 0, logits=False)
    ids, acc, p = g.verify_step(np.concatenate([toks[:B, n - 1:], chain[:B, :S]], 1), np.full(B, n - 1),
                                np.full((B, S + 1), 0.5, np.float32))
    assert (acc == S).all() and np.array_equal(ids, chain[:B])
    g.close()


def test_verification_step_refusals():
    shape = SHAPES[0][1]
    g = make(shape, 771, 2, 64, max_tokens=8)
    g.prefill(synth.tokens(772, 0, 20, shape.vocab).reshape(2, 10), 0, logits=False)
    ok = np.zeros((2, 4), np.int32)
    u = np.zeros((2, 4), np.float32)
    for toks, pos, temp, code in [
            (ok, [11, 0], 0.0, pkg.LLM_ERR_POS_RANGE), (ok, [-1, 0], 0.0, pkg.LLM_ERR_POS_RANGE),
            (ok, [10, 10], -1.0, pkg.LLM_ERR_ARG), (ok, [10, 10], float("inf"), pkg.LLM_ERR_ARG),
            (ok + shape.vocab, [10, 10], 0.0, pkg.LLM_ERR_TOKEN_RANGE)]:
        with pytest.raises(pkg.LlmError) as e:
            g.verify_step(toks, np.array(pos), u, temp)
        assert e.value.status == code
    with pytest.raises(pkg.LlmError) as e:
        g.verify_step(np.zeros((2, 5), np.int32), np.array([10, 10]), np.zeros((2, 5), np.float32))  # 10 tokens, passes of 8
    assert e.value.status == pkg.LLM_ERR_BATCH
    with pytest.raises(pkg.LlmError) as e:
        g.verify_step(np.zeros((2, 1), np.int32), np.array([10, 10]), np.zeros((2, 1), np.float32))
    assert e.value.status == pkg.LLM_ERR_ARG
    assert g.filled(0) == 10
    # probabilities at an address that the head's 16-byte stores could not use
    import torch
    p = torch.zeros(2 * 4 * shape.vocab + 4, device="cuda")
    i4, f4 = torch.zeros(16, dtype=torch.int32, device="cuda"), torch.zeros(16, device="cuda")
    with pytest.raises(pkg.LlmError) as e:
        pkg.llm_verify_step(g.h, ok, 2, 3, np.array([10, 10], np.int32), 0.0, None, f4, p[1:], i4, i4[8:])
    assert e.value.status == pkg.LLM_ERR_ARG
    g.close()
    h = make(shape, 771, 2, 12)
    h.prefill(synth.tokens(772, 0, 20, shape.vocab).reshape(2, 10), 0, logits=False)
    with pytest.raises(pkg.LlmError) as e:
        h.verify_step(ok, np.array([9, 10]), u)
    assert e.value.status == pkg.LLM_ERR_POS_RANGE
    h.close()
    t = make(shape, 771, 2, 64, debug_trace=True)
    with pytest.raises(pkg.LlmError) as e:
        t.verify_step(ok, np.array([0, 0]), u)
    assert e.value.status == pkg.LLM_ERR_ARG
    t.close()
