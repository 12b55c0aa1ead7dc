"""Attention over the 8-bit cache where a few positions outweigh, or outscale, all the others: the rest may
be small beside them and still be the whole result (a position that draws most of the weight often has a
value near zero).  What is lost of a small weight has to be small beside that weight, not beside the largest."""
import math

import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
from tests.test_gpu_qcache import i32, stream

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LN2 = math.log(2.0)


def want_and_bound(q, k, v, scale, dtype):
    """Attention of q [g, hd] over k, v [n, hd] (float64, as stored), and the bound on an output's error:
    a query enters to 2^-19 of its largest element and hd products are summed in f32, which moves a score by
    ds and a weight and the sum by exp(ds) - 1 each (2.2 ds); the exponential itself is off by 2^-21; a weight
    enters as three bf16 pieces (f32 queries) or two (bf16), off by 2^-26 or 2^-17 of itself, however small; sums are
    f32 (2^-19 of the sum of magnitudes for the lengths here); a bf16 output is off by half a step, 2^-8."""
    s = scale * (q @ k.T)
    w = torch.softmax(s, -1)
    want, mag = w @ v, w @ v.abs()
    sens = abs(scale) * q.abs().amax(-1, keepdim=True) * k.abs().sum(-1).max()
    ds = sens * (2.0 ** -19 + (q.shape[-1] + 32) * 2.0 ** -24)
    digits = 2.0 ** -26 if dtype == "f32" else 2.0 ** -17
    tol = mag * (2.2 * ds + digits + 2.0 ** -21 + 2.0 ** -19) + 1e-37
    return want, tol + (want.abs() * 2.0 ** -8 if dtype == "bf16" else 0)


def check(c, q, n, g, dtype, B, kv, hd, rows, kd, vd):
    out = torch.empty_like(q)
    S = q.shape[1]
    c.attend(q, i32([n] * B), out, c.workspace(g, B, S), stream=stream())
    for b in rows:
        for i in range(S):
            end = n - S + i + 1
            for j in range(kv):
                want, tol = want_and_bound(q[b, i, j * g:(j + 1) * g].double(), kd[b, :end, j].double(), vd[b, :end, j].double(),
                                           hd ** -0.5, dtype)
                err = (out[b, i, j * g:(j + 1) * g].double() - want).abs()
                assert (err <= tol).all(), f"row {b} token {i} head {j}: {float((err / tol).max()):.3g} of the bound"


@pytest.mark.parametrize("below", [15.0, 19.5, 20.05, 24.0, 30.0, 45.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,g,S", [(64, 4, 1), (128, 4, 1), (128, 8, 1), (128, 1, 1), (128, 4, 8), (64, 4, 4), (32, 2, 1)])
def test_a_heavy_position_of_value_zero(hd, g, S, dtype, below):
    # position 0 outweighs every other by 2^below and has the value 0: the others, spread over two binades of
    # weights, are the result.  320 (row, kv head) pairs of 32 tiles keep a CTA on one of them.
    B, kv, n = 40, 8, 4096
    gen = torch.Generator(device="cuda").manual_seed(861)
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)  # noqa: E731
    c = pkg.QCache.empty(B, kv, n, hd)
    k = torch.zeros(B, n, kv, hd, device="cuda")
    k[..., 1] = torch.floor(rand(B, n, kv) * 3)          # 0, 1, 2: exact codes, a binade of weight each
    k[:, 0, :, 0] = 1.0
    v = 0.5 + 0.5 * rand(B, n, kv, hd)
    v[:, 0] = 0.0
    c.write(k, v, i32([0] * B), stream=stream())
    c.read(i32([0] * B), k, v, stream=stream())
    assert (v[:, 0] == 0).all()
    q = torch.zeros(B, S, kv * g, hd, device="cuda")
    q[..., 0] = (below + rand(B, S, kv * g)) * LN2 * hd ** 0.5
    q[..., 1] = LN2 * hd ** 0.5
    check(c, q.to(DT[dtype]), n, g, dtype, B, kv, hd, (0, 17, 39), k, v)


@pytest.mark.parametrize("up", [12, 16, 20, 24, 40])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,g,S", [(64, 4, 1), (128, 4, 1), (128, 8, 1), (128, 4, 8), (32, 2, 1)])
def test_values_of_other_sizes_at_negligible_weights(hd, g, S, dtype, up):
    # a block whose values are 2^up larger, at a weight of 2^-(up + 30): nothing of the result, and none of the
    # others' digits
    B, kv, n = 40, 8, 2048
    gen = torch.Generator(device="cuda").manual_seed(862)
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)  # noqa: E731
    c = pkg.QCache.empty(B, kv, n, hd)
    k = torch.zeros(B, n, kv, hd, device="cuda")
    k[..., 1] = torch.floor(rand(B, n, kv) * 3)
    v = 0.5 + 0.5 * rand(B, n, kv, hd)
    for blk in (16, 640, 1600):
        k[:, blk:blk + 16, :, 0] = -1.0
        v[:, blk:blk + 16] *= 2.0 ** up
    c.write(k, v, i32([0] * B), stream=stream())
    c.read(i32([0] * B), k, v, stream=stream())
    q = torch.zeros(B, S, kv * g, hd, device="cuda")
    q[..., 0] = (up + 30) * LN2 * hd ** 0.5
    q[..., 1] = LN2 * hd ** 0.5
    check(c, q.to(DT[dtype]), n, g, dtype, B, kv, hd, (0, 23), k, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,g,S", [(64, 4, 1), (128, 4, 1), (128, 8, 1), (128, 4, 8)])
def test_scores_that_climb_and_fall_far(hd, g, S, dtype):
    # weights that rise by 2^90 along a row, and fall again: references follow, and what was added before them
    # keeps its share
    B, kv, n = 4, 2, 2048
    gen = torch.Generator(device="cuda").manual_seed(863)
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)  # noqa: E731
    c = pkg.QCache.empty(B, kv, n, hd)
    k = torch.zeros(B, n, kv, hd, device="cuda")
    ramp = torch.arange(n, device="cuda") // 64
    k[..., 0] = torch.minimum(ramp, 31 - ramp)[None, :, None].float()     # 0 .. 15 .. 0
    k[..., 1] = torch.floor(rand(B, n, kv) * 3)
    v = 0.5 + 0.5 * rand(B, n, kv, hd)
    v[:, 900:1150] = 0.0                                                  # the heaviest count for nothing
    c.write(k, v, i32([0] * B), stream=stream())
    c.read(i32([0] * B), k, v, stream=stream())
    q = torch.zeros(B, S, kv * g, hd, device="cuda")
    q[..., 0] = (2.0 + 4.0 * rand(B, S, kv * g)) * LN2 * hd ** 0.5
    q[..., 1] = LN2 * hd ** 0.5
    check(c, q.to(DT[dtype]), n, g, dtype, B, kv, hd, range(B), k, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,g,S", [(64, 4, 1), (128, 4, 1), (128, 8, 1), (128, 4, 8), (64, 1, 1), (32, 2, 1)])
def test_every_code_counts_at_its_value(hd, g, S, dtype):
    # all finite codes, subnormal ones among them, along the positions and dimensions: each output element
    # sees codes of one binade in all its positions, and one position of a large value elsewhere
    B, kv, n = 2, 2, 640
    c = pkg.QCache.empty(B, kv, n, hd)
    mags = torch.arange(127, device="cuda", dtype=torch.int32)
    d = torch.arange(hd, device="cuda")
    t = torch.arange(n, device="cuda")
    code = ((d * 8) % 128)[None, :] + (t % 8)[:, None]
    code = torch.where(code == 127, 126, code)
    sign = ((t[:, None] // 8 + d[None, :]) % 3 == 0)
    code = (code | torch.where(sign & (code > 0), 128, 0)).to(torch.uint8)
    assert set((code & 127).flatten().tolist()) == set(mags.tolist()) or hd < 128
    c.tensors[1].copy_(code[None, None].expand(B, kv, n, hd))
    c.tensors[3].fill_(0.25)
    c.tensors[2].fill_(1.0)
    k, v = torch.zeros(B, n, kv, hd, device="cuda"), torch.zeros(B, n, kv, hd, device="cuda")
    c.read(i32([0] * B), k, v, stream=stream())
    gen = torch.Generator(device="cuda").manual_seed(864)
    q = torch.randn(B, S, kv * g, hd, device="cuda", generator=gen)
    check(c, q.to(DT[dtype]), n, g, dtype, B, kv, hd, range(B), k, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hd,kv,g,S,B,n", [(64, 8, 4, 1, 40, 65536), (128, 8, 8, 1, 24, 8192),
                                           (128, 2, 4, 5, 16, 16384), (64, 2, 1, 8, 16, 16384)])
def test_long_sums_of_one_sign(hd, kv, g, S, B, n, dtype):
    # values of one sign and of many sizes: what the additions along a run of tiles lose adds up.  Scores are
    # products of two numbers that are held exactly, so weights are off by 2^-20 at most; a sum of products by up
    # to 2^-23 in each of the 32 additions (f32; bf16 256) between two that are rounded to nearest; those, one for
    # 8 tiles of 128 positions, and the sum of weights, one addition for two tiles and 16 at the end, by 2^-24 each.
    c = pkg.QCache.empty(B, kv, n, hd)
    gen = torch.Generator(device="cuda").manual_seed(865)
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)  # noqa: E731
    k = torch.zeros(B, n, kv, hd, device="cuda")
    k[..., 0] = torch.floor(rand(B, n, kv) * 9) - 4
    v = torch.exp2(-6 * rand(B, n, kv, hd))
    c.write(k, v, i32([0] * B), stream=stream())
    c.read(i32([0] * B), k, v, stream=stream())
    q = torch.zeros(B, S, kv * g, hd, device="cuda")
    q[..., 0] = torch.floor(1 + 3 * rand(B, S, kv * g)) / 4
    q = q.to(DT[dtype])
    out = torch.empty_like(q)
    c.attend(q, i32([n] * B), out, c.workspace(g, B, S), stream=stream())
    cuts = 32 if dtype == "f32" else 256
    worst = 0.0
    for b in range(0, B, 5):
        for i in range(S):
            end = n - S + i + 1
            x, kd, vd = q[b, i].double().reshape(kv, g, hd), k[b, :end].double().transpose(0, 1), v[b, :end].double().transpose(0, 1)
            want = torch.softmax(hd ** -0.5 * x @ kd.transpose(1, 2), -1) @ vd
            err = (out[b, i].double().reshape(kv, g, hd) - want).abs() / want
            worst = max(worst, float(err.max()))
    assert worst <= 2.0 ** -20 + cuts * 2.0 ** -23 + (n / 1024 + n / 256 + 16) * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0), worst
