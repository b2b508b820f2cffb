"""GPU parity of dsa_norm_rope and its backward pass against the FP64 oracle.

Tolerances, per element: the one rounding to BF16 is off by at most 2^-8 of
the value; before it the arithmetic is FP32 (a square root, a sine and a few
products and sums of numbers no larger than m = the row's largest |z| times
sqrt 2, each good to a few 2^-24, the sine and cosine to 2^-22): 2^-19 m
covers it.  Backward the same with the terms of dx.  Weight gradients are sums
of n FP32 products in a fixed tree: 2^-18 of the sum of the terms' sizes.
"""
import numpy as np
import pytest
import torch

from long_context_05_b200 import dsa
from oracle import dsa_oracle as O
from oracle import rows_oracle as R
from tests.parity import u16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()
    yield
    torch.cuda.synchronize()


def f64(t):
    return O.bf16_decode(u16(t))


class Case:
    def __init__(self, B, T, S, Hq, Hk, D, norm, rope, inter=False, lens=None, weights=True, eps=1e-6, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + D + T)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.B, self.T, self.S, self.D, self.norm, self.rope, self.inter, self.eps = B, T, S, D, norm, rope, inter, eps
        self.H = {"q": Hq, "k": Hk}
        self.lens = [S] * B if lens is None else lens
        self.x = {n: rnd(B, T, h, D).bfloat16() for n, h in self.H.items()}
        self.dy = {n: rnd(B, T, h, D).bfloat16() for n, h in self.H.items()}
        self.w = {n: 1 + 0.5 * rnd(norm) if weights and norm else None for n in self.H}
        self.freq = 10000.0 ** (-torch.arange(rope // 2, device="cuda", dtype=torch.float64) * 2 / max(rope, 1))
        self.freq = self.freq.float()
        sl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.shape = dsa.make_shape(None, B=B, T=T, S=S, H_I=4, D_I=32, H=8, d_k=80, d_v=64, k=4, q_block=T,
                                    seqlens=sl)
        self.desc = dsa.make_norm_rope(Hq=Hq, Hk=Hk, D=D, norm_cols=norm, rope_cols=rope, interleaved=inter, eps=eps,
                                       q_weight=self.w["q"], k_weight=self.w["k"],
                                       inv_freq=self.freq if rope else None)

    def forward(self, out=None):
        y = {n: torch.full_like(x, 77.0) for n, x in self.x.items()} if out is None else out
        a = {n: (self.x[n] if h else None, y[n] if h else None) for n, h in self.H.items()}
        dsa.norm_rope(self.shape, self.desc, a["q"][0], a["k"][0], a["q"][1], a["k"][1])
        return y

    def backward(self, dx=None, want=True):
        dx = {n: torch.full_like(x, 77.0) for n, x in self.x.items()} if dx is None else dx
        dw = {n: torch.full((self.norm,), 77.0, device="cuda") if want and self.norm and h else None
              for n, h in self.H.items()}
        o = lambda d, n: d[n] if self.H[n] else None  # noqa: E731
        dsa.norm_rope_backward(self.shape, self.desc, o(self.x, "q"), o(self.x, "k"), o(self.dy, "q"), o(self.dy, "k"),
                               o(dx, "q"), o(dx, "k"), dw["q"], dw["k"],
                               dsa.alloc_norm_rope_workspace(self.shape, self.desc))
        return dx, dw

    def rows(self):
        for n, h in self.H.items():
            for b in range(self.B):
                for t in range(self.T):
                    for i in range(h):
                        yield n, b, t, i, self.lens[b] - self.T + t

    def args(self, n):
        w = None if self.w[n] is None else self.w[n].double().cpu().numpy()
        return dict(weight=w, norm=self.norm, rope=self.rope, inv_freq=self.freq.double().cpu().numpy(), eps=self.eps,
                    interleaved=self.inter)


def check(c: Case):
    y = c.forward()
    dx, dw = c.backward()
    assert dsa.device_error()[0] == 0
    x, dy = {n: f64(v) for n, v in c.x.items()}, {n: f64(v) for n, v in c.dy.items()}
    y, dx = {n: f64(v) for n, v in y.items()}, {n: f64(v) for n, v in dx.items()}
    acc = {n: np.zeros(c.norm) for n in c.H}
    size = {n: np.zeros(c.norm) for n in c.H}
    for n, b, t, i, pos in c.rows():
        at, a = (b, t, i), c.args(n)
        want = R.norm_rope_row(x[n][at], pos, **a)
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * np.abs(want).max() * 2 ** 0.5
        assert (np.abs(y[n][at] - want) <= tol).all(), (n, at, np.abs(y[n][at] - want).max())
        gx, gw = R.norm_rope_grad_row(x[n][at], dy[n][at], pos, **a)
        # dx is a difference of two terms; the second's size enters the FP32 error
        rho = 1.0 / np.sqrt(np.mean(x[n][at][:c.norm] ** 2) + c.eps) if c.norm else 1.0
        w = np.ones(c.norm) if a["weight"] is None else a["weight"]
        m = max(np.abs(dy[n][at]).max() * 2 ** 0.5 * max(1.0, rho * np.abs(w).max(initial=1.0)) * 4, np.abs(gx).max())
        tol = 2.0 ** -8 * np.abs(gx) + 2.0 ** -19 * m
        assert (np.abs(dx[n][at] - gx) <= tol).all(), (n, at, np.abs(dx[n][at] - gx).max())
        acc[n] += gw
        size[n] += np.abs(gw)
    for n, h in c.H.items():
        if c.norm and h:
            err = np.abs(dw[n].double().cpu().numpy() - acc[n])
            # a rotated gradient is a sum of two products: its size is that of the pair
            assert (err <= 2.0 ** -18 * (size[n] + size[n].max())).all(), (n, err.max())


@pytest.mark.parametrize("D,norm,rope,inter", [
    (576, 512, 64, False), (576, 576, 64, False), (576, 512, 64, True), (80, 64, 16, False), (80, 80, 80, True),
    (128, 128, 64, False), (128, 128, 128, False), (128, 0, 64, True), (64, 64, 0, False), (32, 32, 32, False),
    (8, 8, 0, False), (16, 8, 16, False), (192, 128, 64, False), (248, 248, 16, True), (256, 256, 256, False),
    (584, 512, 64, False), (1024, 1024, 256, False), (1024, 512, 128, True)])
def test_rows(D, norm, rope, inter):
    check(Case(2, 3, 50, 5, 1, D, norm, rope, inter))


@pytest.mark.parametrize("B,T,S,Hq,Hk", [(1, 1, 1, 1, 1), (3, 1, 131072, 128, 1), (1, 37, 40, 1, 3), (5, 7, 9, 17, 0),
                                         (4, 19, 19, 0, 2), (1, 700, 700, 2, 1)])
def test_layouts(B, T, S, Hq, Hk):
    check(Case(B, T, S, Hq, Hk, 80, 64, 16, lens=None))


def test_ragged_lengths_and_far_positions():
    check(Case(4, 3, 200_000_000, 2, 1, 128, 128, 64, lens=[3, 131071, 16_777_217, 200_000_000]))


def test_no_weights_and_zero_rows():
    c = Case(1, 4, 9, 3, 1, 80, 64, 16, weights=False, eps=1e-3)
    c.x["q"][0, 1] = 0
    c.x["k"][:] = 0
    check(c)


def test_large_and_small_rows():
    c = Case(1, 4, 9, 3, 1, 80, 64, 16)
    c.x["q"][0, 0] *= 2.0 ** 60           # squares stay finite in FP32
    c.x["q"][0, 1] *= 2.0 ** -40          # eps dominates
    check(c)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,norm,rope", [(576, 512, 64), (128, 128, 128), (64, 0, 64)])
def test_in_place(D, norm, rope, inter):
    c = Case(2, 5, 9, 33, 1, D, norm, rope, inter)
    want, (dwant, wwant) = c.forward(), c.backward()
    y = {n: x.clone() for n, x in c.x.items()}
    keep = c.x
    c.x = y
    c.forward(out=y)
    assert all(torch.equal(y[n], want[n]) for n in y)
    c.x = keep
    d = {n: v.clone() for n, v in c.dy.items()}
    c.dy = d
    dx, dw = c.backward(dx=d)
    assert all(torch.equal(dx[n], dwant[n]) for n in dx)
    assert norm == 0 or all(torch.equal(dw[n], wwant[n]) for n in dw)


def test_backward_needs_no_inputs_without_a_norm_and_no_workspace_without_weights():
    c = Case(1, 5, 9, 3, 1, 64, 0, 64)
    want, _ = c.backward()
    dx = {n: torch.empty_like(v) for n, v in c.x.items()}
    dsa.norm_rope_backward(c.shape, c.desc, None, None, c.dy["q"], c.dy["k"], dx["q"], dx["k"])
    assert all(torch.equal(dx[n], want[n]) for n in dx)
    c = Case(1, 5, 9, 3, 1, 64, 64, 64)
    want, _ = c.backward()
    dx = {n: torch.empty_like(v) for n, v in c.x.items()}
    dsa.norm_rope_backward(c.shape, c.desc, c.x["q"], c.x["k"], c.dy["q"], c.dy["k"], dx["q"], dx["k"])
    assert all(torch.equal(dx[n], want[n]) for n in dx)
    dw = torch.empty(64, device="cuda")
    with pytest.raises(dsa.DsaError) as e:
        dsa.norm_rope_backward(c.shape, c.desc, c.x["q"], c.x["k"], c.dy["q"], c.dy["k"], dx["q"], dx["k"], dw)
    assert e.value.code == 3


def test_same_bits_again_on_another_stream_and_from_a_graph():
    c = Case(2, 130, 200, 40, 1, 128, 128, 64)
    y, (dx, dw) = c.forward(), c.backward()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, (dx2, dw2) = c.forward(), c.backward()
    s.synchronize()
    for a, b in ((y, y2), (dx, dx2), (dw, dw2)):
        assert all(torch.equal(a[n], b[n]) for n in a)
    # captured once, replayed on other inputs
    out = {n: torch.empty_like(v) for n, v in c.x.items()}
    ws = dsa.alloc_norm_rope_workspace(c.shape, c.desc)
    gx = {n: torch.empty_like(v) for n, v in c.x.items()}
    gw = {n: torch.empty(128, device="cuda") for n in c.x}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.norm_rope(c.shape, c.desc, c.x["q"], c.x["k"], out["q"], out["k"])
        dsa.norm_rope_backward(c.shape, c.desc, c.x["q"], c.x["k"], c.dy["q"], c.dy["k"], gx["q"], gx["k"], gw["q"],
                               gw["k"], ws)
    for n in c.x:
        c.x[n].copy_(torch.randn_like(c.x[n].float()))
    g.replay()
    torch.cuda.synchronize()
    y, (dx, dw) = c.forward(), c.backward()
    for a, b in ((y, out), (dx, gx), (dw, gw)):
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_weight_gradient_of_a_side_without_heads_is_zero():
    c = Case(1, 5, 9, 2, 0, 64, 64, 32)
    dx, dw = torch.empty_like(c.x["q"]), {n: torch.full((64,), 77.0, device="cuda") for n in "qk"}
    dsa.norm_rope_backward(c.shape, c.desc, c.x["q"], None, c.dy["q"], None, dx, None, dw["q"], dw["k"],
                           dsa.alloc_norm_rope_workspace(c.shape, c.desc))
    assert torch.equal(dw["q"], c.backward()[1]["q"])
    assert bool((dw["k"] == 0).all()) and dsa.device_error()[0] == 0


def test_lengths_out_of_range_are_reported():
    c = Case(2, 3, 50, 2, 1, 80, 64, 16, lens=[50, 51])
    c.forward()
    st, det = dsa.device_error()
    assert st == 6 and det & 0xFF == 0x50
