"""Attention over an 8-bit cache where one key outweighs a long tail, on the GPU.

Per head row, with w the softmax weights, s the keys' scales, A = sum_k w_k
|V_k| and every chunk of 128 keys c holding its largest w s at m_c:
* the output's rounding to BF16: 2^-8 |out|;
* P in an e4m3 and an e5m2 term, behind a rounding to FP16: (2^-8 + 2^-11) A,
  and below P = 2^-6 a step of 2^-13, off by 2^-14, in units in which the
  largest P of the row is 2^6 or more (parts of up to 2048 keys) or the
  largest of each chunk is 2^2 or more (longer ones; or 2^-24 of the row's):
  2048 * 2^-14 / 2^6 = 128 * 2^-14 / 2^2 = 2^-9 of the largest w s, times a
  byte's 448 at most:  448 * 2^-9 * sum_c m_c covers both, and a split row;
* the exponential and FP32 sums: 2^-18 A.
Nothing grows with the number of keys beside the row's own sum.  The queries
are exact (two columns of few bits); a logit is off by 2^-20 of itself, which
moves the output by twice that times A.
"""
import numpy as np
import pytest
import torch

from long_context_05_b200 import dsa

pytestmark = pytest.mark.gpu

DK, DV = 576, 512


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()
    yield
    torch.cuda.synchronize()


class Tail:
    """Keys with values of a common mean, and logits set by two columns: query
    head h sees  gap_h * a_k + z_k,  a_k = column 512, z_k = column 513."""

    def __init__(self, B, T, S, H=128, k=64, page=0, gaps=(6.0, 13.0), seed=0, unit=2.0 ** -8, decode=False):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + S)
        self.g, self.B, self.T, self.S, self.H, self.k, self.page, self.unit = g, B, T, S, H, k, page, unit
        kw, self.table, self.rows = {}, None, B * S
        if page:
            per = (S + page - 1) // page
            self.table = torch.randperm(B * per + 1, generator=g, device="cuda")[:B * per].view(B, per).int()
            self.rows = (B * per + 1) * page
            kw = dict(page_size=page, num_pages=B * per + 1, block_table=self.table)
        self.tau = 2.0 ** -4
        self.shape = dsa.make_shape(None, mode=dsa.DSA_DECODE if decode else dsa.DSA_PREFILL, B=B, T=T, S=S, H_I=4,
                                    D_I=32, H=H, d_k=DK, d_v=DV, k=k, q_block=T, softmax_scale=self.tau, **kw)
        # logit = tau q s k8; columns are held in bytes of value / unit
        self.gap = torch.linspace(*gaps, H, device="cuda").mul(2 ** 4).bfloat16()     # gap / tau
        self.q = torch.zeros(B, T, H, DK, dtype=torch.bfloat16, device="cuda")
        f = 2.0 ** -8 / unit
        self.q[..., 512] = self.gap * f
        self.q[..., 513] = 16.0 * f
        self.x = torch.zeros(B, S, DK, device="cuda")                # in units of `unit`
        self.x[..., :DV] = 128 * (1 + torch.randn(B, S, DV, generator=g, device="cuda"))
        self.scale = torch.full((B, S), unit, device="cuda")
        self.idx = None

    def logits(self, b, at, a=None, z=None):
        if a is not None:
            self.x[b, at, 512] = 256 * torch.as_tensor(a, device="cuda", dtype=torch.float32)
        if z is not None:
            self.x[b, at, 513] = 256 * torch.as_tensor(z, device="cuda", dtype=torch.float32)
        return self

    def build(self):
        self.k8 = self.x.clamp(-448, 448).to(torch.float8_e4m3fn)
        if self.table is None:
            self.pool8, self.pool_scale = self.k8.view(torch.uint8).contiguous(), self.scale.clone()
        else:
            s = torch.arange(self.S, device="cuda")
            at = (self.table.long()[:, s // self.page] * self.page + s % self.page).flatten()
            self.pool8 = torch.zeros(self.rows, DK, dtype=torch.uint8, device="cuda")
            self.pool_scale = torch.ones(self.rows, device="cuda")
            self.pool8[at] = self.k8.view(torch.uint8).flatten(0, 1)
            self.pool_scale[at] = self.scale.flatten()
        return self

    def run(self):
        self.build()
        out = torch.full((self.B, self.T, self.H, DV), 77.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.B, self.T, self.H), 77.0, device="cuda")
        ws = dsa.alloc_workspace8(self.shape)
        if self.idx is None:
            dsa.dense_attn8(self.shape, self.q, self.pool8, self.pool_scale, out, lse, ws)
        else:
            dsa.sparse_attn8(self.shape, self.q, self.pool8, self.pool_scale, self.idx, out, lse, ws)
        assert dsa.device_error()[0] == 0
        return out, lse

    def check(self, out, lse, queries):
        for b in range(self.B):
            for t in queries:
                if self.idx is None:
                    sel = torch.arange(self.S - self.T + t + 1, device="cuda")
                else:
                    sel = self.idx[b, t].long()
                    sel = sel[sel >= 0]
                sc = self.scale[b, sel].double()
                kv = self.k8[b, sel].double()
                x = (self.q[b, t].double() @ kv.T) * sc * self.tau
                want_l = torch.logsumexp(x, -1)
                w = torch.exp(x - want_l[:, None])
                v = kv[:, :DV] * sc[:, None]
                want, A = w @ v, w @ v.abs()
                n = sel.numel()
                ws = torch.nn.functional.pad(w * sc, (0, -n % 128)).view(self.H, -1, 128)
                tol = (2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) * A
                       + 448 * 2.0 ** -9 * ws.amax(-1).sum(-1, keepdim=True)
                       + 2.0 ** -19 * x.abs().amax(-1, keepdim=True) * A)
                err = (out[b, t].double() - want).abs()
                assert bool((err <= tol).all()), (b, t, float((err / tol).max()))
                lt = 2.0 ** -19 * (1 + want_l.abs() + x.abs().amax(-1))
                le = (lse[b, t].double() - want_l).abs()
                assert bool((le <= lt).all()), (b, t, float((le / lt).max()))
                rel = float(err.norm() / want.norm())
                assert rel <= 4e-3, (b, t, rel)
        return self


def _z(c, n, spread):
    return spread * torch.randn(n, generator=c.g, device="cuda") if spread else 0.0


@pytest.mark.parametrize("spread", [0.0, 0.25, 0.5])
@pytest.mark.parametrize("B,T,page,decode", [(1, 80, 0, False),          # one part of 2048 keys
                                             (32, 1, 64, True),          # two parts
                                             (1, 1, 0, True)])           # a chunk to a part
def test_one_key_above_a_selection(B, T, page, decode, spread):
    c = Tail(B, T, 2048, k=2048, page=page, decode=decode)
    c.idx = torch.empty(B, T, 2048, dtype=torch.int32, device="cuda")
    place = [0, 5, 127, 128, 1031, 2047]
    for b in range(B):
        c.logits(b, slice(None), z=_z(c, 2048, spread)).logits(b, 0, a=1.0, z=0.0)
        for t in range(T):
            n = 2048 - T + t + 1
            r = torch.full((2048,), -1, dtype=torch.int32, device="cuda")
            r[:n] = torch.randperm(n, generator=c.g, device="cuda").int()
            p = place[(b + t) % len(place)]
            i = int((r == 0).nonzero())
            r[i], r[p] = r[p].clone(), r[i].clone()
            c.idx[b, t] = r
    c.check(*c.run(), queries=range(0, T, 1 + T // 8))


@pytest.mark.parametrize("spread", [0.0, 0.25, 0.5])
@pytest.mark.parametrize("T,S,at", [(80, 8192, 0), (80, 8192, 4103), (80, 65536, 5), (80, 2300, 127), (1, 65536, 0),
                                    (3, 8191, 17)])
def test_one_key_above_every_other_dense(T, S, at, spread):
    c = Tail(1, T, S, decode=T == 1)
    c.logits(0, slice(None), z=_z(c, S, spread)).logits(0, at, a=1.0, z=0.0)
    c.check(*c.run(), queries=sorted({0, T // 2, T - 1}))


@pytest.mark.parametrize("T,S", [(80, 65536), (80, 8192), (1, 40000)])
@pytest.mark.parametrize("order", ["falling", "rising", "islands", "steps"])
def test_references_that_rise_and_fall(T, S, order):
    """Chunks whose largest weights differ by many octaves, up and down."""
    c = Tail(1, T, S, gaps=(1.0, 12.0), decode=T == 1)
    s = torch.arange(S, device="cuda", dtype=torch.float32)
    a = {"falling": 1.5 - 1.5 * s / S, "rising": 1.5 * s / S,
         "islands": (s % 701 == 3).float() * (1 + (s // 701) % 3 / 4),           # some chunks hold a peak, of three heights
         "steps": ((s // 300) % 5) / 4}[order]
    c.logits(0, slice(None), a=a, z=_z(c, S, 0.25))
    c.check(*c.run(), queries=sorted({0, T - 1}))


def test_a_key_far_above_everything():
    """A gap past the depth that the reference follows, and past FP32's exponents."""
    for gap in (30.0, 110.0):
        c = Tail(1, 80, 8192, gaps=(gap * 0.5, gap))
        c.logits(0, 0, a=1.0)
        c.check(*c.run(), queries=[0, 79])


@pytest.mark.parametrize("unit", [2.0 ** -100, 2.0 ** -30, 2.0 ** 60])
def test_long_tails_at_any_scale(unit):
    c = Tail(1, 80, 8192, unit=unit)
    c.logits(0, slice(None), z=_z(c, 8192, 0.25)).logits(0, 5, a=1.0, z=0.0)
    c.check(*c.run(), queries=[0, 79])


def test_repeats_and_graph():
    c = Tail(1, 80, 8192)
    c.logits(0, slice(None), z=_z(c, 8192, 0.5)).logits(0, 5, a=1.0, z=0.0)
    out, lse = c.run()
    for _ in range(2):
        o, l = c.run()
        assert torch.equal(o, out) and torch.equal(l, lse)
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    ws = dsa.alloc_workspace8(c.shape)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dsa.dense_attn8(c.shape, c.q, c.pool8, c.pool_scale, o, l, ws)
    for _ in range(2):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert np.isfinite(lse.cpu().numpy()).all()
