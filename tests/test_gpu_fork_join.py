"""Kernels that may start early, behind an event of another stream, a copy or a
memset: they wait for that too, run as they are and captured into a graph."""
import pytest
import torch

from long_context_05_b200 import dsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()
    yield
    torch.cuda.synchronize()


class Layer:
    """A decode step from raw rows: each input of a kernel comes from the side stream."""

    def __init__(self):
        g = torch.Generator(device="cuda")
        g.manual_seed(7)
        self.B, self.S, self.H = 4, 256, 64
        B, S, H = self.B, self.S, self.H
        rnd = lambda *a: torch.randn(*a, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.shape = dsa.make_shape(None, mode=dsa.DSA_DECODE, B=B, T=1, S=S, H_I=4, D_I=32, H=H, d_k=576, d_v=512, k=200,
                                    q_block=1)
        fill = dsa.make_shape(None, B=B, T=S, S=S, H_I=4, D_I=32, H=H, d_k=576, d_v=512, k=200, q_block=1)
        self.freq = (10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)).float()
        self.nr = dsa.make_norm_rope(Hq=H, Hk=1, D=576, norm_cols=512, rope_cols=64, inv_freq=self.freq)
        self.x, self.r = [rnd(B, 1, H, 576) for _ in range(3)], [rnd(B, 1, 1, 576) for _ in range(3)]
        self.sel = [torch.randint(0, S, (B, 1, 200), generator=g, device="cuda").int() for _ in range(3)]
        self.src = [torch.empty_like(t[0]) for t in (self.x, self.r, self.sel)]
        self.q, self.row, self.idx = (torch.zeros_like(t) for t in self.src)
        self.big = torch.randn(3000, 3000, generator=g, device="cuda")
        self.kv8 = torch.zeros(B, S, 576, dtype=torch.uint8, device="cuda")
        self.scale = torch.ones(B, S, device="cuda")
        dsa.cache_write(fill, kv=rnd(B, S, 576), kv8=self.kv8, kv_scale=self.scale)
        self.back = torch.zeros(B, S, 576, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros(B, 1, H, 512, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros(B, 1, H, device="cuda")
        self.tmp = torch.empty_like(self.big)
        self.ws = dsa.alloc_workspace8(self.shape)
        self.side = torch.cuda.Stream()

    def late(self, dst, src, wait):
        """dst = src from the side stream, behind a while of other work."""
        main = torch.cuda.current_stream()
        self.side.wait_stream(main)
        with torch.cuda.stream(self.side):
            torch.mm(self.big, self.big, out=self.tmp)
            dst.copy_(src)
        if wait:
            torch.cuda.synchronize()
        main.wait_stream(self.side)

    def __call__(self, wait=False):
        self.late(self.q, self.src[0], wait)
        dsa.norm_rope(self.shape, self.nr, self.q, self.row, self.q, self.row)   # (the old row: replaced below)
        self.late(self.row, self.src[1], wait)
        dsa.cache_write(self.shape, kv=self.row, kv8=self.kv8, kv_scale=self.scale)
        self.back.zero_()
        dsa.cache_read(self.shape, 0, self.S, kv8=self.kv8, kv_scale=self.scale, kv=self.back)
        self.late(self.idx, self.src[2], wait)
        dsa.sparse_attn8(self.shape, self.q, self.kv8, self.scale, self.idx, self.out, self.lse, self.ws)
        if wait:
            torch.cuda.synchronize()

    def set(self, i):
        for s, t in zip(self.src, (self.x, self.r, self.sel)):
            s.copy_(t[i])

    def result(self):
        return [t.clone() for t in (self.out, self.lse, self.back, self.q)]


@pytest.mark.parametrize("graph", [False, True])
def test_inputs_of_another_stream(graph):
    c = Layer()
    want = []
    for i in range(3):
        c.set(i)
        c(wait=True)
        want.append(c.result())
    run = c
    if graph:
        c.set(0)
        c()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c()
        run = g.replay
    for n in range(9):
        i = (2 * n + 1) % 3
        c.set(i)
        run()
        got = c.result()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b), (n, i)
    assert dsa.device_error()[0] == 0
