"""Attention over shared positions where a few positions outweigh, or outscale, all the others, whichever way a call goes:
the shared positions read once, for many columns or for few, or row by row.  What is lost of a small weight has to be small
beside that weight, not beside the largest."""
import math

import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
from tests.test_gpu_qcache import i32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LN2 = math.log(2.0)
# rows and tokens: 128 columns and 132, in tables with room for more; 16 and 24; and in tables with no more room than positions
WAYS = [("many", 128, 4, 32, 1), ("many", 64, 4, 33, 1), ("many", 64, 2, 8, 8), ("few", 128, 4, 4, 1), ("few", 64, 4, 2, 3),
        ("rows", 128, 4, 3, 1), ("rows", 64, 1, 2, 5)]


class Case:
    """All rows name the same n positions k, v [n, kv, hd]; the first `shared` of them count as shared."""

    def __init__(self, way, hd, B, n, kv=2):
        self.hd, self.B, self.n, self.kv, pages = hd, B, n, kv, -(-n // 64)
        self.c = pkg.QCache.empty(1, kv, pages * 64, hd)
        table = np.full((B, pages if way == "rows" else max(4096, pages)), -1)
        table[:, :pages] = np.random.default_rng(n).permutation(pages)
        self.table = i32(table)

    def put(self, k, v):
        self.c.write(k[None], v[None], i32([0]), table=self.table[:1])
        self.read(k, v)

    def read(self, k, v):
        self.c.read(i32([0]), k[None], v[None], table=self.table[:1])
        self.k, self.v = k.double(), v.double()

    def run(self, q, g, shared):
        out = torch.empty_like(q)
        self.c.attend_shared(q, i32([self.n] * self.B), i32([0, self.B]), i32([shared]), out,
                             self.c.workspace_shared(g, self.B, q.shape[1], 1), table=self.table)
        return out

    def check(self, q, g, dtype, shared):
        """A query enters with each element off by 2^-16 of itself and 2^-27 of the largest (f32: four pieces of five bits,
        the last in steps of 2^-10 / 2^10 where the largest is 128 or more), or is exact but for elements below 2^-9 of the largest,
        off by 2^-17 of that (bf16: two pieces).  hd products of pieces are summed in f32 and a few more roundings of a score
        follow: (hd + 32) 2^-24 of the sum of magnitudes.  A score off by ds moves a weight and the sum by exp(ds) - 1 each
        (2.2 ds); the exponential itself is off by 2^-21; a weight enters as bf16 pieces, off by 2^-26 (f32: three) or
        2^-17 (bf16: two) of itself; sums are f32: 2^-19 of the sum of magnitudes; a bf16 output is off by half a step, 2^-8."""
        out, scale = self.run(q, g, shared), self.hd ** -0.5
        for i in range(q.shape[1]):
            end = self.n - q.shape[1] + i + 1
            for j in range(self.kv):
                x = q[:, i, j * g:(j + 1) * g].double().flatten(0, 1)
                k, v = self.k[:end, j], self.v[:end, j]
                w = torch.softmax(scale * (x @ k.T), -1)
                want, mag, top = w @ v, w @ v.abs(), x.abs().amax(-1, keepdim=True)
                dq = 2.0 ** -16 * x.abs() + 2.0 ** -27 * top if dtype == "f32" else torch.where(x.abs() < 2.0 ** -9 * top, 2.0 ** -17 * top, 0 * top)
                sums = x.abs() @ k.abs().T
                ds = scale * (dq @ k.abs().T + (self.hd + 32) * 2.0 ** -24 * sums).amax(-1, keepdim=True)
                tol = mag * (2.2 * ds + (2.0 ** -26 if dtype == "f32" else 2.0 ** -17) + 2.0 ** -21 + 2.0 ** -19) + 1e-37
                tol = tol + (want.abs() * 2.0 ** -8 if dtype == "bf16" else 0)
                err = (out[:, i, j * g:(j + 1) * g].double().flatten(0, 1) - want).abs()
                assert (err <= tol).all(), f"token {i} head {j}: {float((err / tol).max()):.3g} of the bound"


def rand(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.rand(*s, device="cuda", generator=gen)


@pytest.mark.parametrize("below", [15.0, 20.05, 24.0, 30.0, 45.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("way,hd,g,B,S", WAYS)
def test_a_heavy_position_of_value_zero(way, hd, g, B, S, dtype, below):
    # one position outweighs every other by 2^below and has the value 0: the others, spread over two binades of
    # weights, are the result.  It is the first, one in the middle of the shared positions, or one of the rows' own.
    r, n = rand(861), 4200
    for heavy in (0, 2345, 4150):
        c = Case(way, hd, B, n)
        k, v = torch.zeros(n, c.kv, hd, device="cuda"), 0.5 + 0.5 * r(n, c.kv, hd)
        k[..., 1] = torch.floor(r(n, c.kv) * 3)          # 0, 1, 2: exact codes, a binade of weight each
        k[heavy, :, 0], k[heavy, :, 1], v[heavy] = 1.0, 0.0, 0.0
        c.put(k, v)
        assert (c.v[heavy] == 0).all()
        q = torch.zeros(B, S, c.kv * g, hd, device="cuda")
        q[..., 0] = (below + r(B, S, c.kv * g)) * LN2 * hd ** 0.5
        q[..., 1] = LN2 * hd ** 0.5
        c.check(q.to(DT[dtype]), g, dtype, 4099)


@pytest.mark.parametrize("up", [12, 16, 24, 40])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("way,hd,g,B,S", WAYS)
def test_values_of_other_sizes_at_negligible_weights(way, hd, g, B, S, dtype, up):
    # blocks whose values are 2^up larger, at a weight of 2^-(up + 30): nothing of the result, and none of the others' digits
    r, n = rand(862), 2100
    c = Case(way, hd, B, n)
    k, v = torch.zeros(n, c.kv, hd, device="cuda"), 0.5 + 0.5 * r(n, c.kv, hd)
    k[..., 1] = torch.floor(r(n, c.kv) * 3)
    for blk in (16, 640, 1600, 2080):
        k[blk:blk + 16, :, 0] = -1.0
        v[blk:blk + 16] *= 2.0 ** up
    c.put(k, v)
    q = torch.zeros(B, S, c.kv * g, hd, device="cuda")
    q[..., 0] = (up + 30) * LN2 * hd ** 0.5
    q[..., 1] = LN2 * hd ** 0.5
    c.check(q.to(DT[dtype]), g, dtype, 2000)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("way,hd,g,B,S", WAYS)
def test_scores_that_climb_and_fall_far(way, hd, g, B, S, dtype):
    # weights that rise by 2^90 along the positions, and fall again: references follow, and what was added before them
    # keeps its share; in steps of 64 positions, and all within the first tile
    r, n = rand(863), 2100
    for step in (64, 4):
        c = Case(way, hd, B, n)
        k, v = torch.zeros(n, c.kv, hd, device="cuda"), 0.5 + 0.5 * r(n, c.kv, hd)
        ramp = torch.arange(n, device="cuda") // step
        k[..., 0] = torch.minimum(ramp, (31 - ramp).clamp(min=0))[:, None].float()     # 0 .. 15 .. 0
        k[..., 1] = torch.floor(r(n, c.kv) * 3)
        v[900 * step // 64:1150 * step // 64] = 0.0                                    # the heaviest count for nothing
        c.put(k, v)
        q = torch.zeros(B, S, c.kv * g, hd, device="cuda")
        q[..., 0] = (2.0 + 4.0 * r(B, S, c.kv * g)) * LN2 * hd ** 0.5
        q[..., 1] = LN2 * hd ** 0.5
        c.check(q.to(DT[dtype]), g, dtype, 2050)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("way,hd,g,B,S", WAYS)
def test_references_that_move_within_a_tile(way, hd, g, B, S, dtype):
    # weights that rise by 2^26 with every block of 16 positions, eight times over, and start again: what was weighed a step before
    # is rescaled before its product, and as the heaviest 32 positions of 128 are 0 it is the result; the same bits every time
    r, n = rand(867), 1500
    c = Case(way, hd, B, n)
    k, v = torch.zeros(n, c.kv, hd, device="cuda"), 0.5 + 0.5 * r(n, c.kv, hd)
    block = torch.arange(n, device="cuda") // 16 % 8
    k[..., 0] = block[:, None].float()
    k[..., 1] = torch.floor(r(n, c.kv) * 3)
    v[block >= 6] = 0.0
    c.put(k, v)
    q = torch.zeros(B, S, c.kv * g, hd, device="cuda")
    q[..., 0] = (26.0 + r(B, S, c.kv * g)) * LN2 * hd ** 0.5
    q[..., 1] = LN2 * hd ** 0.5
    q = q.to(DT[dtype])
    c.check(q, g, dtype, 1400)
    first = c.run(q, g, 1400)
    assert all(torch.equal(c.run(q, g, 1400), first) for _ in range(8))


@pytest.mark.parametrize("dtype,up", [("f32", 12), ("f32", 16), ("f32", 20), ("bf16", 8), ("bf16", 10), ("bf16", 12)])
@pytest.mark.parametrize("way,hd,g,B,S", WAYS)
def test_an_element_far_above_the_others(way, hd, g, B, S, dtype, up):
    # a query's first element is 2^up times the others, and the keys are 0 there: the others decide the scores.  An element is
    # held to 2^-19 of itself (bf16: exactly) or, where pieces end, to a share of the largest, f << 1: f32 2^-27 with the shared
    # positions read once for many columns, else 2^-32; bf16 2^-17 of elements below 2^-9 of it, else 2^-22 of those below 2^-14.
    # Products are summed in f32: (hd + 32) 2^-24 of the sum of magnitudes.  Scores off by ds move a weight and the sum of weights by
    # exp(ds) - 1 each, together exp(2 ds) - 1; the rest as in Case.check.
    r, n = rand(868), 700
    c = Case(way, hd, B, n)
    k, v = 2.0 * r(n, c.kv, hd) - 1.0, 2.0 * r(n, c.kv, hd) - 1.0
    k[..., 0] = 0.0
    c.put(k, v)
    q = 2.0 * r(B, S, c.kv * g, hd) - 1.0
    q[..., 0] = 2.0 ** up * (1.0 + r(B, S, c.kv * g))
    q = q.to(DT[dtype])
    out, scale = c.run(q, g, 600), hd ** -0.5
    many = way == "many"
    for i in range(S):
        end = n - S + i + 1
        for j in range(c.kv):
            x = q[:, i, j * g:(j + 1) * g].double().flatten(0, 1)
            top = x.abs().amax(-1, keepdim=True)
            if dtype == "f32":
                dq = torch.maximum(2.0 ** -19 * x.abs(), (2.0 ** -27 if many else 2.0 ** -32) * top)
            else:
                dq = torch.where(x.abs() < (2.0 ** -9 if many else 2.0 ** -14) * top, (2.0 ** -17 if many else 2.0 ** -22) * top, 0 * top)
            kk, vv = c.k[:end, j], c.v[:end, j]
            w = torch.softmax(scale * (x @ kk.T), -1)
            want, mag = w @ vv, w @ vv.abs()
            ds = scale * (dq @ kk.abs().T + (hd + 32) * 2.0 ** -24 * (x.abs() @ kk.abs().T)).amax(-1, keepdim=True)
            tol = mag * (torch.expm1(2 * ds) + (2.0 ** -26 if dtype == "f32" else 2.0 ** -17) + 2.0 ** -21 + 2.0 ** -19)
            tol = tol + (want.abs() * 2.0 ** -8 if dtype == "bf16" else 0)
            err = (out[:, i, j * g:(j + 1) * g].double().flatten(0, 1) - want).abs()
            assert (err <= tol).all(), f"token {i} head {j}: {float((err / tol).max()):.3g} of the bound"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("way,hd,g,B,S", WAYS)
def test_every_code_counts_at_its_value(way, hd, g, B, S, dtype):
    # all finite codes, subnormal ones among them, along the positions and dimensions
    n = 640
    c = Case(way, hd, B, n)
    d, t = torch.arange(hd, device="cuda"), torch.arange(n, device="cuda")
    code = ((d * 8) % 128)[None, :] + (t % 8)[:, None]
    code = torch.where(code == 127, 126, code)
    sign = ((t[:, None] // 8 + d[None, :]) % 3 == 0)
    code = (code | torch.where(sign & (code > 0), 128, 0)).to(torch.uint8)
    c.c.tensors[1].copy_(code[None, None].expand(1, c.kv, n, hd))
    c.c.tensors[3].fill_(0.25)
    c.c.tensors[2].fill_(1.0)
    c.read(torch.zeros(n, c.kv, hd, device="cuda"), torch.zeros(n, c.kv, hd, device="cuda"))
    gen = torch.Generator(device="cuda").manual_seed(864)
    q = torch.randn(B, S, c.kv * g, hd, device="cuda", generator=gen)
    c.check(q.to(DT[dtype]), g, dtype, 600)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("way,hd,g,B,S,n", [("many", 64, 4, 32, 1, 65536), ("many", 128, 8, 24, 1, 16384), ("many", 128, 4, 7, 5, 16384),
                                            ("few", 128, 4, 4, 1, 65536), ("few", 64, 1, 3, 5, 16384), ("rows", 64, 1, 2, 3, 16384)])
def test_long_sums_of_one_sign(way, hd, g, B, S, n, dtype):
    # values of one sign and of many sizes: what the additions along a run of tiles lose adds up.  Scores are products of two
    # numbers that are held exactly, so weights are off by 2^-20 at most; a sum of products by up to 2^-23 in each of the additions
    # between two that are rounded to nearest: 16 positions and a weight's pieces each, 512 positions long (f32: 96) or 4096 (512);
    # those, one for 512 positions, and the sum of weights, one addition for 128 positions and 16 at the end, by 2^-24 each.
    c = Case(way, hd, B, n)
    r = rand(865)
    k, v = torch.zeros(n, c.kv, hd, device="cuda"), torch.exp2(-6 * r(n, c.kv, hd))
    k[..., 0] = torch.floor(r(n, c.kv) * 9) - 4
    c.put(k, v)
    q = torch.zeros(B, S, c.kv * g, hd, device="cuda")
    q[..., 0] = torch.floor(1 + 3 * r(B, S, c.kv * g)) / 4
    q = q.to(DT[dtype])
    out, worst = c.run(q, g, n - 100), 0.0
    cuts = 96 if dtype == "f32" else 512
    for b in range(0, B, 5):
        for i in range(S):
            end = n - S + i + 1
            x, kd, vd = q[b, i].double().reshape(c.kv, g, hd), c.k[:end].transpose(0, 1), c.v[:end].transpose(0, 1)
            want = torch.softmax(hd ** -0.5 * x @ kd.transpose(1, 2), -1) @ vd
            worst = max(worst, float(((out[b, i].double().reshape(c.kv, g, hd) - want).abs() / want).max()))
    assert worst <= 2.0 ** -20 + cuts * 2.0 ** -23 + (n / 512 + n / 128 + 16) * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0), worst


def test_places_behind_4_gb():
    # 2^32 bytes of codes in a cache, and pages at its end: offsets of 33 bits, for each way a call can go
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("24 GB of device memory")
    kv, hd, cap, rows, g, n = 8, 128, 64 * 1024, 72, 4, 1500          # 72 x 8 x 65536 x 128 = 4.8e9 bytes of keys
    c = pkg.QCache.empty(rows, kv, cap, hd)
    small = pkg.QCache.empty(1, kv, 1536, hd)
    r = rand(866)
    k, v = r(1, n, kv, hd) - 0.5, r(1, n, kv, hd) - 0.5
    last = rows * (cap // 64) - 1
    near, far = np.arange(24), last - np.arange(24)
    c.write(k, v, i32([0]), table=i32(far[None]))
    small.write(k, v, i32([0]), table=i32(near[None]))
    for B, wide in ((3, 24), (3, 8192), (40, 8192)):
        q = r(B, 1, kv * g, hd) - 0.5
        out = []
        for x, pages in ((c, far), (small, near)):
            table = np.full((B, wide), -1)
            table[:, :24] = pages
            o = torch.empty_like(q)
            x.attend_shared(q, i32([n] * B), i32([0, B]), i32([1111]), o, x.workspace_shared(g, B, 1, 1), table=i32(table))
            out.append(o)
        assert torch.equal(*out)
    del c
    torch.cuda.empty_cache()
