"""The torch wrappers without a stream argument: calls follow torch's current stream, so that they are ordered
with the work on their tensors, and captured where that is."""
import numpy as np
import pytest

import llama_architecture_kv_gb300 as pkg
from tests import qcache_ref as ref
from tests.test_gpu_qcache import attend_tolerance, i32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

B, KV, G, HD, N = 2, 2, 4, 64, 48


def operands(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    p, q = torch.softmax(f(B, 3, 999), -1), torch.softmax(f(B, 2, 999), -1)
    return dict(k=f(B, N, KV, HD), v=f(B, N, KV, HD), q=f(B, 1, KV * G, HD), p=p, r=q,
                u=torch.rand(B, 3, device="cuda", generator=gen),
                drafts=torch.randint(0, 999, (B, 2), device="cuda", generator=gen, dtype=torch.int32))


class Calls:
    """Buffers that the calls read and write, and one run of every call on them."""

    def __init__(self):
        self.c = pkg.QCache.empty(B, KV, 64, HD)
        self.x = {k: torch.zeros_like(t) for k, t in operands(0).items()}
        self.out = torch.zeros(B, 1, KV * G, HD, device="cuda")
        self.back = [torch.zeros(B, N, KV, HD, device="cuda") for _ in range(2)]
        self.ids = torch.zeros(B, 3, dtype=torch.int32, device="cuda")
        self.acc = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.pos, self.length, self.ws = i32([0] * B), i32([N] * B), self.c.workspace(G, B, 1)

    def run(self):
        x = self.x
        self.c.write(x["k"], x["v"], self.pos)
        self.c.attend(x["q"], self.length, self.out, self.ws)
        self.c.read(self.pos, *self.back)
        pkg.llm_verify(x["p"], x["r"], x["drafts"], x["u"], self.ids, self.acc)

    def check(self, given):
        n = {k: t.cpu().numpy() for k, t in given.items()}
        r = ref.RefCache(B, KV, 64, HD)
        r.write(n["k"].astype(np.float64), n["v"].astype(np.float64), [0] * B)
        want, mag, sens, flat = r.attend(n["q"].astype(np.float64), [N] * B)
        assert (np.abs(self.out.double().cpu().numpy() - want) <= attend_tolerance("f32", HD, want, mag, sens, flat)).all()
        for b in range(B):
            for got, w in zip(self.back, r.values(None, b, N)):
                assert np.array_equal(got[b].double().cpu().numpy(), w.swapaxes(0, 1))
            assert (self.ids[b].tolist(), int(self.acc[b])) == ref.verify(n["p"][b], n["r"][b], n["drafts"][b], None, n["u"][b])


def test_calls_follow_the_current_stream():
    one, given = Calls(), operands(1)
    one.run()                                  # (the kernels' first launches wait for the device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)         # about 50 ms, after which the operands are there
        for k, t in given.items():
            one.x[k].copy_(t)
        one.run()
        for t in one.x.values():
            t.zero_()                          # (behind the calls)
    side.synchronize()
    one.check(given)


def test_calls_inside_a_capture_are_captured():
    one = Calls()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        one.run()
    for seed in (2, 3):
        given = operands(seed)
        for k, t in given.items():
            one.x[k].copy_(t)
        gr.replay()
        torch.cuda.synchronize()
        one.check(given)


def test_a_given_stream_is_the_one_used():
    one, given = Calls(), operands(4)
    one.run()
    for k, t in given.items():
        one.x[k].copy_(t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(100_000_000)             # on the current stream: calls on another one need not wait for it
    begun = torch.cuda.Event()
    begun.record()
    s = side.cuda_stream
    one.c.write(one.x["k"], one.x["v"], one.pos, stream=s)
    one.c.attend(one.x["q"], one.length, one.out, one.ws, stream=s)
    one.c.read(one.pos, *one.back, stream=s)
    pkg.llm_verify(one.x["p"], one.x["r"], one.x["drafts"], one.x["u"], one.ids, one.acc, stream=s)
    side.synchronize()
    assert not begun.query()
    torch.cuda.synchronize()
    one.check(given)
