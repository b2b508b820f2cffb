"""A step's kernels one behind the other on a stream, where each may start while
the one before it still runs: the same bits as with a wait between them."""
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


class Step:
    """Queries (normed and rotated), a selection and a BF16 cache, decode."""

    def __init__(self, B, k, write, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        S, H = 600, 128
        self.lens = torch.randint(300, S, (B,), generator=g, device="cuda").int()
        self.shape = dsa.make_shape(None, mode=dsa.DSA_DECODE, B=B, T=1, S=S, H_I=4, D_I=32, H=H, d_k=576, d_v=512, k=k,
                                    q_block=1, seqlens=self.lens)
        self.x = [torch.randn(B, 1, H, 576, generator=g, device="cuda").bfloat16() for _ in range(4)]
        self.q_in = torch.empty_like(self.x[0])
        self.q = torch.zeros_like(self.q_in)
        self.freq = (10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)).float()
        self.nr = dsa.make_norm_rope(Hq=H, Hk=0, D=576, norm_cols=512, rope_cols=64, inv_freq=self.freq)
        self.kv = torch.randn(B, S, 576, generator=g, device="cuda").bfloat16()
        self.idx = torch.randint(0, 300, (B, 1, k), generator=g, device="cuda").int()
        self.out = torch.zeros(B, 1, H, 512, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros(B, 1, H, device="cuda")
        self.ws = dsa.alloc_workspace(self.shape)
        self.write = write
        self.row = torch.randn(B, 1, 576, generator=g, device="cuda").bfloat16()
        self.kv8 = torch.zeros(B, S, 576, dtype=torch.uint8, device="cuda")
        self.scale = torch.ones(B, S, device="cuda")

    def __call__(self, wait=lambda: None):
        wait()
        dsa.norm_rope(self.shape, self.nr, self.q_in, None, self.q, None)
        wait()
        if self.write:
            dsa.cache_write(self.shape, kv=self.row, kv8=self.kv8, kv_scale=self.scale)
            wait()
        dsa.sparse_attn(self.shape, self.q, self.kv, self.idx, self.out, self.lse, self.ws)
        wait()


@pytest.mark.parametrize("B,k", [(32, 100), (8, 256), (64, 128), (1, 300)])
@pytest.mark.parametrize("write", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_decode_attention_sees_the_rotated_queries(B, k, write, graph):
    s = Step(B, k, write)
    want = []
    for x in s.x:
        s.q_in.copy_(x)
        s(torch.cuda.synchronize)
        want.append((s.out.clone(), s.lse.clone()))
    run = s
    if graph:
        g = torch.cuda.CUDAGraph()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=st):
            s()
        run = g.replay
    got = []
    for i in range(24):
        s.q_in.copy_(s.x[i % 4])
        s.out.zero_()
        run()
        got.append((s.out.clone(), s.lse.clone()))
    torch.cuda.synchronize()
    assert dsa.device_error()[0] == 0
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 4][0]) and torch.equal(l, want[i % 4][1]), i


def test_decode_attention_sees_new_lengths():
    """The lengths are written by the kernel in front of the rotation."""
    s = Step(16, 128, True)
    a, b = s.lens.clone(), (s.lens // 2 + 150).int()
    want = {}
    for n, l in (("a", a), ("b", b)):
        s.lens.copy_(l)
        s.q_in.copy_(s.x[0])
        s(torch.cuda.synchronize)
        want[n] = (s.out.clone(), s.q.clone())
    assert not torch.equal(want["a"][1], want["b"][1])
    for i in range(20):
        n, l = (("a", a), ("b", b))[i % 2]
        s.lens.copy_(l)
        s()
        o, q = s.out.clone(), s.q.clone()
        torch.cuda.synchronize()
        assert torch.equal(o, want[n][0]) and torch.equal(q, want[n][1]), i
    assert dsa.device_error()[0] == 0
