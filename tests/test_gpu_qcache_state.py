"""What a handle with an 8-bit cache keeps between calls, and what may not depend on it: waits that ran
out, dead data of earlier sequences, drafts that were not kept."""
import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
import synth
from synth import shrink
from synth.configs import TINY
from tests.test_gpu_qcache_model import E4M3, LLAMA8, SHAPES, make

pytestmark = pytest.mark.gpu

# with the head sizes of the attention on CUDA cores
ALL = SHAPES + [("f32_hd32", shrink(TINY, kv=3, g=2, half=16, ffn=200, vocab=300), 3, 0),
                ("bf16_hd256", shrink(LLAMA8, layers=2, kv=1, g=2, half=128, ffn=512, vocab=1000), 4, 1)]


def bits(x):
    return np.ascontiguousarray(x).view(np.uint32)


@pytest.mark.parametrize("half,cap", [(8, 64), (8, 192), (16, 64), (32, 64), (64, 300), (128, 64)])
def test_a_wait_that_ran_out_leaves_the_handle_as_it_was(half, cap):
    # heads of 16, 32 and 256 need no attention workspace on caches this small
    shape = shrink(TINY, kv=2, g=2, half=half)
    g = make(shape, 801, 1, cap, cache_type=E4M3)
    toks = synth.tokens(802, 0, 12, shape.vocab)
    first = g.prefill(toks[None, :9], 0)
    step = g.decode(toks[9:10], 9)
    pkg.llm_check_wait_timeout(g.h, 5000)
    with pytest.raises(pkg.LlmError) as e:
        g.synchronize()
    assert e.value.status == pkg.LLM_ERR_DEVICE_TIMEOUT
    g.synchronize()                            # reported once, then cleared
    assert np.array_equal(bits(g.decode(toks[9:10], 9)), bits(step))
    assert np.array_equal(bits(g.prefill(toks[None, :9], 0)), bits(first))
    g.close()


def sick(rng, shape, n, how):
    """Cache elements [kv][n][hd] of an earlier sequence: large, or not finite."""
    x = (rng.standard_normal((shape.kv, n, shape.hd)) * 2.0 ** 12).astype(np.float32)
    if how == "nan":
        x[:, ::3, 1] = np.nan
    return (x.view(np.uint32) >> 16).astype(np.uint16) if shape.bf16 else x


@pytest.mark.parametrize("how", ["large", "nan"])
@pytest.mark.parametrize("reset", [True, False], ids=["reset", "rewound"])
@pytest.mark.parametrize("name,shape,B,tc", SHAPES, ids=[s[0] for s in SHAPES])
def test_dead_data_decides_nothing_for_prompts_and_imports_that_start_inside_blocks(name, shape, B, tc, reset, how):
    cap, rng = 192, np.random.default_rng(812)
    t0, t1, t2, t3 = (synth.tokens(813 + i, 0, m, shape.vocab) for i, m in enumerate((10, 13, 20, 3)))
    got = []
    for old in (True, False):
        g = make(shape, 811, 2, cap, tc_min_batch=tc, cache_type=E4M3)
        if old:
            for layer in range(shape.layers):
                for row in range(2):
                    g.kv_import(layer, row, 0, sick(rng, shape, 150, how), sick(rng, shape, 150, how))
        if reset:
            pkg.llm_reset(g.h)
        # (without a reset: row 0 rewound to nothing kept but its first 10 positions, row 1 too)
        g.prefill(np.stack([t0, t0]), 0, logits=False)
        # row 0: 37..49 in a block of dead positions; row 1: 52..54, then 55..74 of another prompt in the same block
        lg = g.prefill_packed(np.concatenate([t1, t3, t2]), [0] * 13 + [1] * 23, list(range(37, 50)) + list(range(52, 75)),
                              [1] * 13 + [2] * 3 + [3] * 20, [12, 15, 35])
        out = [bits(lg)]
        k, v = sick(np.random.default_rng(5), shape, 9, "large"), sick(np.random.default_rng(6), shape, 9, "large")
        for layer in range(shape.layers):
            out += [g.kv_export(layer, 0, 37, 13), g.kv_export(layer, 1, 52, 23)]
        for layer in range(shape.layers):
            g.kv_import(layer, 0, 133, k, v)   # positions 128 .. 132 are dead
            out.append(g.kv_export(layer, 0, 133, 9))
        got.append(out)
        g.close()
    for a, b in zip(*got):
        assert all(np.array_equal(x, y, equal_nan=np.asarray(x).dtype == np.float32) for x, y in zip(a, b))


def test_dead_data_of_the_block_is_kept_where_it_is_live():
    # a prompt that starts right behind filled positions keeps what they hold
    name, shape, B, tc = SHAPES[2]
    g = make(shape, 821, 2, 128, tc_min_batch=tc, cache_type=E4M3)
    t = synth.tokens(822, 0, 60, shape.vocab)
    g.prefill(np.stack([t[:37], t[:37]]), 0, logits=False)
    k0, v0 = g.kv_export(0, 0, 0, 37)
    g.prefill_packed(t[37:40], [0] * 3, [37, 38, 39], [1] * 3, [2])
    k1, v1 = g.kv_export(0, 0, 0, 37)
    # codes are rounded again at most where the scale grew: by 2^-4 of a value at most, or a step of the block
    for a, b in ((k0, k1), (v0, v1)):
        a, b = ((x.astype(np.uint32) << 16).view(np.float32) for x in (a, b))
        assert np.array_equal(a[:, :32], b[:, :32])
        assert (np.abs(a - b) <= np.abs(a) * 2.0 ** -4 + np.abs(b).max() * 2.0 ** -14).all() and np.abs(b[:, 32:]).max() > 0
    g.close()


@pytest.mark.parametrize("tokens", [8, 16, 20, 0])
@pytest.mark.parametrize("name,shape,B,tc", SHAPES[:3], ids=[s[0] for s in SHAPES[:3]])
def test_imports_are_one_write_whatever_a_pass_holds(name, shape, B, tc, tokens):
    # values that grow inside blocks: a write of the whole range rounds each of them once
    from tests import qcache_ref as ref
    from tests.test_gpu_qcache_model import wide
    g = make(shape, 831, 2, 128, max_tokens=tokens, cache_type=E4M3)
    rng = np.random.default_rng(832)
    n, at = 75, 5
    grow = 2.0 ** (np.arange(n) * 0.7 % 9)[None, :, None]
    k, v = ((rng.standard_normal((shape.kv, n, shape.hd)) * grow).astype(np.float32) for _ in range(2))
    if shape.bf16:
        k, v = ((x.view(np.uint32) >> 16).astype(np.uint16) for x in (k, v))
    want = ref.RefCache(1, shape.kv, 128, shape.hd)
    kk, vv = (wide(x).swapaxes(0, 1)[None] for x in (k, v))
    want.write(kk, vv, [at])
    wk, wv = want.values(None, 0, n, at)
    for layer in range(shape.layers):
        g.kv_import(layer, 1, at, k, v)
        gk, gv = g.kv_export(layer, 1, at, n)
        assert np.array_equal(wide(gk), wk) and np.array_equal(wide(gv), wv)
    g.close()


# ---- drafts ----

def chain_of(g, start, pos, n):
    out = np.empty((len(start), n), np.int32)
    cur = start
    for s in range(n):
        cur = g.step_rows(cur, pos + s)
        out[:, s] = cur
    return out


@pytest.mark.parametrize("cache", [pkg.LLM_CACHE_MODEL, E4M3], ids=["model", "e4m3"])
@pytest.mark.parametrize("name,shape,B,tc", ALL, ids=[s[0] for s in ALL])
def test_probabilities_do_not_depend_on_later_drafts(name, shape, B, tc, cache):
    n, S, cap = 24, 5, 128
    g = make(shape, 841, B, cap, tc_min_batch=tc, cache_type=cache, wstd=0.2 if not shape.bf16 else 0.06)
    toks = synth.tokens(842, 0, B * n, shape.vocab).reshape(B, n)
    pos = np.array([n - 1 - 3 * (b % 4) for b in range(B)])
    start = toks[np.arange(B), pos]
    rng = np.random.default_rng(843)
    u = rng.random((B, S + 1)).astype(np.float32)
    base = rng.integers(0, shape.vocab, (B, S)).astype(np.int32)
    first = None
    for at in (S - 1, S - 1, S - 1, 2, 0):     # the draft from which on this list differs from the first
        drafts = base.copy()
        if first is not None:
            drafts[:, at:] = rng.integers(0, shape.vocab, (B, S - at))
        g.prefill(toks[:, :n - 1], 0, logits=False)
        _, _, p = g.verify_step(np.concatenate([start[:, None], drafts], 1), pos, u, temp=0.8)
        if first is None:
            first = p
        else:
            assert np.array_equal(bits(p[:, :at + 1]), bits(first[:, :at + 1])), at
    g.close()


@pytest.mark.parametrize("name,shape,B,tc", ALL, ids=[s[0] for s in ALL])
def test_drafts_that_are_not_kept_leave_nothing_behind(name, shape, B, tc):
    from tests import qcache_ref as ref
    from tests.test_gpu_qcache_model import wide
    n, S, cap = 40, 9, 128
    kw = dict(tc_min_batch=tc, wstd=0.2 if not shape.bf16 else 0.06)
    g = make(shape, 851, B, cap, cache_type=E4M3, **kw)
    toks = synth.tokens(852, 0, B * n, shape.vocab).reshape(B, n)
    pos = np.array([n - 1 - 3 * (b % 5) for b in range(B)])   # some rows cross from one block into the next
    start = toks[np.arange(B), pos]
    g.prefill(toks[:, :n - 1], 0, logits=False)
    chain = chain_of(g, start, pos, S + 2)
    kept = (np.arange(B) * 2 + 1) % (S + 1)
    u = np.full((B, S + 1), 0.5, np.float32)
    rng = np.random.default_rng(853)
    seen, lists = [], []
    for trial in range(3):
        drafts = chain[:, :S].copy()
        for b in range(B):
            tail = rng.integers(0, shape.vocab, S - kept[b])
            if kept[b] < S:
                tail[0] = (chain[b, kept[b]] + 1 + trial) % shape.vocab
            drafts[b, kept[b]:] = tail
        lists.append(drafts)
        g.prefill(toks[:, :n - 1], 0, logits=False)
        ids, acc, p = g.verify_step(np.concatenate([start[:, None], drafts], 1), pos, u)
        if trial == 0:
            # (a draft may be lost to a near tie between the steps' logits and the pass's: the lists agree up to it)
            assert (acc <= kept).all() and 2 * (acc == kept).sum() > B and (acc < S).any()
            kept = acc.copy()
        assert np.array_equal(acc, kept)
        out = [g.kv_export(layer, b, 0, int(pos[b] + kept[b]) + 1) for layer in range(shape.layers) for b in range(B)]
        nxt = g.decode_rows(ids[np.arange(B), kept], pos + kept + 1)
        seen.append((out, bits(nxt)))
    for out, nxt in seen[1:]:
        assert np.array_equal(nxt, seen[0][1])
        for (k, v), (k0, v0) in zip(out, seen[0][0]):
            assert np.array_equal(k, k0) and np.array_equal(v, v0)
    # what layer 0 holds: the kept tokens written one by one (its keys and values depend on no cache)
    plain = make(shape, 851, B, cap, **kw)
    plain.prefill(toks[:, :n - 1], 0, logits=False)
    prompt = {b: plain.kv_export(0, b, 0, n - 1) for b in range(B)}
    plain.verify_step(np.concatenate([start[:, None], lists[0]], 1), pos, u)
    for b in range(B):
        end = int(pos[b] + kept[b]) + 1
        k0, v0, kk, vv = (wide(x).swapaxes(0, 1)[None] for x in (*prompt[b], *plain.kv_export(0, b, 0, end)))
        want = ref.RefCache(1, shape.kv, cap, shape.hd)
        want.write(k0, v0, [0])
        for q in range(int(pos[b]), end):
            want.write(kk[:, q:q + 1], vv[:, q:q + 1], [q])
        wk, wv = want.values(None, 0, end)
        gk, gv = seen[0][0][b]
        assert np.array_equal(wide(gk), wk) and np.array_equal(wide(gv), wv), b
    plain.close()
    g.close()


@pytest.mark.parametrize("name,shape,B,tc", ALL, ids=[s[0] for s in ALL])
def test_blocks_of_lost_drafts_alone_are_empty(name, shape, B, tc):
    from tests.test_gpu_qcache_model import wide
    n, S, cap = 31, 20, 128
    g = make(shape, 871, B, cap, tc_min_batch=tc, cache_type=E4M3, wstd=0.2 if not shape.bf16 else 0.06)
    toks = synth.tokens(872, 0, B * n, shape.vocab).reshape(B, n)
    g.prefill(toks[:, :n], 0, logits=False)
    pos = np.array([n - b % 17 for b in range(B)])             # 15 .. 31: the last of a block among them
    drafts = synth.tokens(873, 0, B * (S + 1), shape.vocab).reshape(B, S + 1)
    drafts[:, 0] = toks[np.arange(B), np.minimum(pos, n - 1)]
    # no probability is above a draw times 1 that is above 1: nothing is kept
    _, acc, _ = g.verify_step(drafts, pos, np.full((B, S + 1), 2.0, np.float32))
    assert (acc == 0).all()
    for b in range(B):
        behind, end = int(pos[b]) // 16 * 16 + 16, int(pos[b]) + S + 1
        for layer in range(shape.layers):
            k, v = g.kv_export(layer, b, behind, end - behind)
            assert (wide(k) == 0).all() and (wide(v) == 0).all()   # (codes keep their signs)
    g.close()
