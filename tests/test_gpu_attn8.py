"""GPU parity of the attention over an 8-bit cache against the FP64 oracle.

Per element, with w the softmax weights and A = sum_k w_k |V_k|:
* the output's rounding to BF16: 2^-8 |out|;
* P in two e4m3 terms: off by 2^-8 of itself at most, which moves the output
  by 2^-8 A, and by e4m3's subnormal half step, 2^-10 where the largest P of
  the row is 2^6 or more: 2^-16 w_max sum_k |V_k| / s_k' with s' the keys'
  scales over the largest: 2^-16 w_max n max|V|;
* logits: q's two terms are off by 2^-19 of the row's largest |q|, FP32 sums
  by less; a logit off by d moves the output by at most 2 d A and lse by d;
  d = tau (2^-18 max|q| max_k sum|k_c| + 2^-20 max_k sum|q_c k_c|);
* the exponential and FP32 sums: 2^-18 A, and 2^-20 (1 + |lse|) for lse.
"""
import numpy as np
import pytest
import torch

from long_context_05_b200 import dsa
from long_context_05_b200.inputs import Workload, make_inputs
from oracle import dsa_oracle as O
from oracle import rows_oracle as R
from tests import parity as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()
    yield
    torch.cuda.synchronize()


class Case:
    def __init__(self, B, T, S, H, d_k=576, k=64, page=0, lens=None, decode=False, seed=0, tau=0.0, spread=0.5,
                 exps=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + S * 7 + T)
        self.g = g
        self.B, self.T, self.S, self.H, self.d_k, self.k, self.page = B, T, S, H, d_k, k, page
        self.d_v = 512 if d_k == 576 else 64
        self.lens = [S] * B if lens is None else lens
        self.tau = tau or 1.0 / np.sqrt(d_k)
        self.rows, self.table, kw = B * S, None, {}
        if page:
            per = (S + page - 1) // page
            pages = B * per + 2
            self.table = torch.randperm(pages, generator=g, device="cuda")[:B * per].view(B, per).int()
            for b in range(B):
                self.table[b, (self.lens[b] + page - 1) // page:] = -5
            self.rows = pages * page
            kw = dict(page_size=page, num_pages=pages, block_table=self.table)
        sl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.shape = dsa.make_shape(None, mode=dsa.DSA_DECODE if decode else dsa.DSA_PREFILL, B=B, T=T, S=S, H_I=4,
                                    D_I=32, H=H, d_k=d_k, d_v=self.d_v, k=k, q_block=T, seqlens=sl, softmax_scale=tau,
                                    **kw)
        self.q = torch.randn(B, T, H, d_k, generator=g, device="cuda").bfloat16()
        x = torch.randn(self.rows, d_k, generator=g, device="cuda")
        x *= torch.exp(spread * torch.randn(self.rows, 1, generator=g, device="cuda"))
        self.kv8 = torch.zeros(self.rows, d_k, dtype=torch.uint8, device="cuda")
        self.scale = torch.ones(self.rows, device="cuda")
        amax = x.abs().amax(-1)
        self.scale = amax / 448 if exps is None else torch.exp2(
            exps[torch.randint(0, len(exps), (self.rows,), generator=g, device="cuda")])
        y = x / (amax / 448).unsqueeze(-1) if exps is not None else x / self.scale.unsqueeze(-1)
        self.kv8 = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.idx = None

    def row(self, b, s):
        if self.table is None:
            return b * self.S + s
        return int(self.table[b, s // self.page]) * self.page + s % self.page

    def select(self, empty=0.0):
        """Random selections without repeats, empty slots scattered among them."""
        idx = np.full((self.B, self.T, self.k), -1, np.int32)
        rng = np.random.default_rng(self.S + self.k)
        for b in range(self.B):
            for t in range(self.T):
                n = self.lens[b] - self.T + t + 1
                m = min(self.k, n)
                r = np.full(self.k, -1)
                r[:m] = rng.permutation(n)[:m]
                r[rng.random(self.k) < empty] = -1
                idx[b, t] = rng.permutation(r) if empty else r
        self.idx = torch.from_numpy(idx).cuda()
        return self

    def run(self, dense=False, ws=None, lse=True):
        out = torch.full((self.B, self.T, self.H, self.d_v), 77.0, dtype=torch.bfloat16, device="cuda")
        l = torch.full((self.B, self.T, self.H), 77.0, device="cuda") if lse else None
        ws = dsa.alloc_workspace8(self.shape) if ws is None else ws
        if dense:
            dsa.dense_attn8(self.shape, self.q, self.kv8, self.scale, out, l, ws)
        else:
            dsa.sparse_attn8(self.shape, self.q, self.kv8, self.scale, self.idx, out, l, ws)
        return out, l

    def check(self, out, lse, dense=False, rows=None):
        assert dsa.device_error()[0] == 0
        o, l = O.bf16_decode(P.u16(out)), lse.double().cpu().numpy()
        q = O.bf16_decode(P.u16(self.q))
        idx = None if dense else self.idx.cpu().numpy()
        for b in range(self.B):
            at = [self.row(b, s) for s in range(self.lens[b])]
            kv = R.dequantise(self.kv8[at].cpu().numpy(), self.scale[at].cpu().numpy())
            for t in range(self.T) if rows is None else rows:
                sel = np.arange(self.lens[b] - self.T + t + 1) if dense else idx[b, t]
                want, wl, A, wm = R.attention_row(q[b, t], kv, sel, self.d_v, self.tau)
                sel = sel[sel >= 0]
                if sel.size == 0:
                    assert (o[b, t] == 0).all() and np.isneginf(l[b, t]).all(), (b, t)
                    continue
                K = np.abs(kv[sel])
                qa = np.abs(q[b, t])
                d = self.tau * (2.0 ** -18 * qa.max(1) * K.sum(1).max() + 2.0 ** -20 * (qa @ K.T).max(1))
                tol = (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -18 + 2 * d[:, None]) * A
                       + 2.0 ** -16 * wm[:, None] * sel.size * K[:, :self.d_v].max())
                err = np.abs(o[b, t] - want)
                assert (err <= tol).all(), (b, t, err.max(), (err / tol).max())
                lt = d + 2.0 ** -20 * (1 + np.abs(wl))
                assert (np.abs(l[b, t] - wl) <= lt).all(), (b, t, np.abs(l[b, t] - wl).max(), lt.min())
                # the typical element is far inside those worst cases
                assert np.linalg.norm(err) <= 4e-3 * np.linalg.norm(want), (b, t)


@pytest.mark.parametrize("B,T,S,H,d_k,k,page,lens,decode", [
    (1, 1, 1, 8, 576, 1, 0, None, True),
    (1, 1, 5, 128, 576, 3, 0, None, True),
    (2, 1, 300, 128, 576, 130, 0, [140, 300], True),
    (3, 1, 700, 16, 576, 513, 64, [1, 64, 700], True),
    (2, 3, 200, 40, 576, 64, 0, None, False),
    (2, 5, 130, 128, 576, 65, 48, [63, 130], False),
    (1, 90, 400, 128, 576, 200, 0, None, False),       # more CTAs than SMs: no key splits
    (1, 1, 3, 8, 80, 2, 0, None, True),
    (2, 4, 300, 56, 80, 190, 16, [17, 290], False),
    (1, 160, 260, 128, 80, 129, 0, None, False),
    (4, 1, 2100, 128, 80, 2048, 0, None, True),
])
def test_selected(B, T, S, H, d_k, k, page, lens, decode):
    c = Case(B, T, S, H, d_k, k, page, lens, decode).select()
    c.check(*c.run(), rows=range(0, T, 1 + T // 12))


@pytest.mark.parametrize("B,T,S,H,d_k,page,lens,decode", [
    (1, 1, 1, 128, 576, 0, None, True),
    (2, 1, 1000, 128, 576, 64, [65, 1000], True),
    (1, 1, 9000, 24, 576, 0, None, True),
    (2, 7, 70, 128, 576, 0, [7, 70], False),
    (1, 100, 130, 128, 576, 0, None, False),
    (3, 1, 129, 8, 80, 16, [1, 64, 129], True),
    (2, 33, 190, 48, 80, 0, None, False),
])
def test_dense(B, T, S, H, d_k, page, lens, decode):
    c = Case(B, T, S, H, d_k, 8, page, lens, decode)
    c.check(*c.run(dense=True), dense=True, rows=range(0, T, 1 + T // 12))


@pytest.mark.parametrize("decode,T", [(True, 1), (False, 80)])
def test_empty_slots_anywhere_and_empty_rows(decode, T):
    c = Case(2, T, 300, 128, 576, 257, 0, None, decode).select(empty=0.6)
    c.idx[0, 0] = -1                                   # nothing selected
    c.idx[1, T - 1, :256] = -1                         # a single key, in the last chunk
    c.idx[1, T - 1, 256] = 7
    c.check(*c.run(), rows=sorted({0, 1 % T, T // 2, T - 1}))


@pytest.mark.parametrize("T", [1, 80])
def test_duplicates_count_twice(T):
    c = Case(1, T, 200, 64, 576, 128).select()
    c.idx[..., 64:] = c.idx[..., :64]
    c.check(*c.run(), rows=[0, T - 1])


@pytest.mark.parametrize("T", [1, 80])
def test_unread_rows_may_hold_anything(T):
    """NaN bytes, NaN and infinite scales in rows that no query selects."""
    c = Case(1, T, 400, 128, 576, 100, 16).select()
    used = torch.zeros(c.rows, dtype=torch.bool)
    for s in np.unique(c.idx.cpu().numpy()):
        if s >= 0 and s < 400:
            used[c.row(0, int(s))] = True
    if T == 80:                                        # keep some rows unread
        c.idx[c.idx >= 390] = -1
        used = torch.zeros(c.rows, dtype=torch.bool)
        for s in np.unique(c.idx.cpu().numpy()):
            if s >= 0:
                used[c.row(0, int(s))] = True
    assert not bool(used.all())
    c.kv8[~used.cuda()] = 0x7F
    c.scale[~used.cuda()] = float("nan")
    c.check(*c.run(), rows=[0, T - 1])


@pytest.mark.parametrize("B,T,S,H,d_k,page,lens", [
    (1, 9, 140, 8, 576, 0, None),                      # eight queries' rows to a CTA, split keys
    (2, 50, 333, 24, 576, 16, [51, 333]),              # queries that start inside a CTA's rows
    (1, 300, 300, 72, 80, 0, None),                    # from the first position on
    (3, 37, 200, 96, 80, 32, [37, 128, 200]),
    (1, 200, 1000, 40, 576, 0, None),                  # one split a CTA
])
def test_dense_rows_of_several_queries(B, T, S, H, d_k, page, lens):
    c = Case(B, T, S, H, d_k, 8, page, lens)
    c.check(*c.run(dense=True), dense=True, rows=sorted({0, 1, 7, 8, T // 2, T - 2, T - 1}))


def test_dense_agrees_with_every_key_selected():
    """The same keys in the same chunks, in a CTA of one query and of several."""
    c = Case(1, 160, 160, 40, 576, 160)
    pos = torch.arange(160, device="cuda", dtype=torch.int32)
    c.idx = torch.where(pos[None] <= pos[:, None], pos[None], torch.full_like(pos[None], -1))[None].contiguous()
    (o1, l1), (o2, l2) = c.run(), c.run(dense=True)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


def test_dense_does_not_read_past_the_query():
    c = Case(1, 40, 100, 64, 576, 8)
    c.kv8[90:] = 0x7F
    c.scale[90:] = float("inf")
    out, lse = c.run(dense=True)
    c.check(out[:, :30].contiguous(), lse[:, :30].contiguous(), dense=True, rows=[])
    o, l = out.float(), lse
    assert bool(torch.isfinite(o[:, :30]).all()) and bool(torch.isfinite(l[:, :30]).all())


@pytest.mark.parametrize("T", [1, 80])
@pytest.mark.parametrize("exps", [[-40.0, -39.0], [30.0, 31.0], [-20.0, 0.0, 10.0]])
def test_scales_far_from_one(T, exps):
    """Tokens whose scales differ by many octaves, tiny and huge caches."""
    c = Case(1, T, 300, 32, 576, 200, exps=torch.tensor(exps, device="cuda"), tau=2.0 ** -(max(exps) + 10)).select()
    c.check(*c.run(), rows=[0, T - 1])


@pytest.mark.parametrize("T", [1, 80])
def test_sharp_and_growing_logits(T):
    """Large logits, in an order that moves the running reference all the time."""
    c = Case(1, T, 600, 128, 576, 600, tau=0.5).select()
    q = O.bf16_decode(P.u16(c.q))
    kv = R.dequantise(c.kv8.cpu().numpy(), c.scale.cpu().numpy())
    for t in range(T):
        sel = c.idx[0, t].cpu().numpy()
        ok = sel[sel >= 0]
        order = np.argsort(q[0, t, 0] @ kv[ok].T)
        sel[:ok.size] = ok[order]
        c.idx[0, t] = torch.from_numpy(sel).cuda()
    c.check(*c.run(), rows=[0, T // 2, T - 1])


def test_queries_of_many_sizes():
    c = Case(1, 4, 200, 128, 576, 150).select()
    c.q[0, 0] *= 2.0 ** -30
    c.q[0, 1] = 0
    c.q[0, 2, :, :570] *= 2.0 ** -12                   # small beside the row's last columns
    c.q[0, 3, :64] *= 30.0
    c.check(*c.run())


def test_modes_agree_and_runs_repeat():
    c = Case(2, 1, 500, 128, 576, 300, decode=True).select()
    out, lse = c.run()
    for _ in range(3):
        o2, l2 = c.run()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    c.shape.mode = dsa.DSA_PREFILL
    o2, l2 = c.run()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    o2, _ = c.run(lse=False)
    assert torch.equal(out, o2)


def test_bad_indices_and_pages_are_reported_and_skipped():
    c = Case(1, 2, 100, 64, 576, 70, 16).select()
    good = c.idx.clone()
    c.idx[0, 0, 3], c.idx[0, 1, 69] = 100, 1 << 30
    out, lse = c.run()
    st, det = dsa.device_error()
    assert st == 6 and det & 0xFF == 0x70
    c.idx[0, 0, 3] = c.idx[0, 1, 69] = -1
    c.check(out, lse)
    c.idx = good
    c.table[0, 2] = 10 ** 6
    out, lse = c.run()
    assert dsa.device_error()[0] == 6
    c.idx[(c.idx >= 32) & (c.idx < 48)] = -1
    c.table[0, 2] = 0                                  # never used below
    c.check(out, lse)


def test_workspace_is_checked():
    c = Case(1, 1, 500, 128, 576, 300, decode=True).select()
    for ws in (None, torch.empty(64, dtype=torch.uint8, device="cuda")):
        with pytest.raises(dsa.DsaError) as e:
            o = torch.empty(1, 1, 128, 512, dtype=torch.bfloat16, device="cuda")
            dsa.sparse_attn8(c.shape, c.q, c.kv8, c.scale, c.idx, o, None, ws)
        assert e.value.code == 3


def test_cache_past_two_gigabytes():
    S = (1 << 31) // 576 + 5000
    c = Case.__new__(Case)
    c.B, c.T, c.S, c.H, c.d_k, c.k, c.page, c.d_v = 1, 1, S, 128, 576, 300, 0, 512
    c.lens, c.tau, c.table, c.rows = [S], 1 / 24.0, None, S
    c.shape = dsa.make_shape(None, mode=dsa.DSA_DECODE, B=1, T=1, S=S, H_I=4, D_I=32, H=128, d_k=576, d_v=512, k=300,
                             q_block=1)
    c.q = torch.randn(1, 1, 128, 576, device="cuda").bfloat16()
    c.kv8 = torch.zeros(S, 576, dtype=torch.uint8, device="cuda")
    c.kv8[-5000:] = torch.randint(0, 120, (5000, 576), device="cuda").byte()
    c.scale = torch.full((S,), 2.0 ** -8, device="cuda")
    c.idx = (S - 1 - torch.randperm(5000, device="cuda")[:300]).int().view(1, 1, 300)
    ws = torch.empty(dsa.workspace8_size(c.shape), dtype=torch.uint8, device="cuda")
    out, lse = c.run(ws=ws)
    assert dsa.device_error()[0] == 0
    sel = c.idx[0, 0].long()
    kv = R.dequantise(c.kv8[sel].cpu().numpy(), c.scale[sel].cpu().numpy())
    want, wl, _, _ = R.attention_row(O.bf16_decode(P.u16(c.q))[0, 0], kv, np.arange(300), 512, c.tau)
    assert np.linalg.norm(O.bf16_decode(P.u16(out))[0, 0] - want) <= 4e-3 * np.linalg.norm(want)
    assert np.abs(lse[0, 0].cpu().numpy() - wl).max() <= 1e-4


def test_two_graphs_share_a_workspace_and_another_stream():
    a = Case(2, 1, 500, 128, 576, 300, decode=True, seed=1).select()
    b = Case(2, 1, 500, 128, 576, 300, decode=True, seed=2).select()
    ws = dsa.alloc_workspace8(a.shape)
    want = [c.run() for c in (a, b)]
    outs = [(torch.zeros_like(w[0]), torch.zeros_like(w[1])) for w in want]
    graphs = []
    for c, (o, l) in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dsa.sparse_attn8(c.shape, c.q, c.kv8, c.scale, c.idx, o, l, ws)
        graphs.append(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            for g in graphs:
                g.replay()
    s.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])


# ------------------------------------------------------------- the path together

def _prepare(wl, seed):
    """Raw rows of a sequence, before the norm, the rotation and the quantising."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return dict(q=r(wl.B, wl.S, wl.H, wl.d_k), kv=r(wl.B, wl.S, 1, wl.d_k), q_I=r(wl.B, wl.S, wl.H_I, wl.D_I),
                k_I=r(wl.B, wl.S, 1, wl.D_I), w=torch.randn(wl.B, wl.S, wl.H_I, generator=g, device="cuda") / 8)


def _step(wl, raw, cache, s0, s1, page, table, nw, freq, fused_ws=False):
    """Tokens [s0, s1) of every sequence through norm and rotation, the cache
    write and the whole path."""
    T = s1 - s0
    B = wl.B
    sl = torch.full((B,), s1, dtype=torch.int32, device="cuda")
    paged = dict(page_size=page, num_pages=cache["pages"], block_table=table) if page else {}
    sh = dsa.make_shape(None, mode=dsa.DSA_DECODE if T == 1 else dsa.DSA_PREFILL, B=B, T=T, S=wl.S, H_I=wl.H_I,
                        D_I=wl.D_I, H=wl.H, d_k=wl.d_k, d_v=wl.d_v, k=wl.k, q_block=wl.q_block, seqlens=sl, **paged)
    part = {n: raw[n][:, s0:s1].contiguous() for n in raw}
    dv = wl.d_v
    nr = dsa.make_norm_rope(Hq=wl.H, Hk=1, D=wl.d_k, norm_cols=dv, rope_cols=wl.d_k - dv, q_weight=nw, k_weight=nw,
                            inv_freq=freq[0])
    ni = dsa.make_norm_rope(Hq=wl.H_I, Hk=1, D=wl.D_I, norm_cols=wl.D_I, rope_cols=wl.D_I // 2, interleaved=True,
                            inv_freq=freq[1])
    dsa.norm_rope(sh, nr, part["q"], part["kv"], part["q"], part["kv"])
    dsa.norm_rope(sh, ni, part["q_I"], part["k_I"], part["q_I"], part["k_I"])
    qI8 = torch.empty(B, T, wl.H_I, wl.D_I, dtype=torch.uint8, device="cuda")
    qs = torch.empty(B, T, wl.H_I, device="cuda")
    dsa.cache_write(sh, kv=part["kv"], kv8=cache["kv8"], kv_scale=cache["kv_scale"], k_I=part["k_I"],
                    kI8=cache["kI8"], kI_scale=cache["kI_scale"], q_I=part["q_I"], qI8=qI8, qI_scale=qs)
    out = torch.empty(B, T, wl.H, dv, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, T, wl.H, device="cuda")
    idx = torch.full((B, T, wl.k), -9, dtype=torch.int32, device="cuda")
    dsa.forward8(sh, dict(q_I=qI8, q_scale=qs, w=part["w"], k_I=cache["kI8"], k_scale=cache["kI_scale"], q=part["q"],
                          kv8=cache["kv8"], kv_scale=cache["kv_scale"]), out, lse, idx, dsa.alloc_workspace8(sh))
    return sh, part, (qI8, qs), out, lse, idx


def test_calls_at_once_on_two_streams():
    """Split and unsplit, selected and dense calls side by side, each with a workspace of its own."""
    cases = [(Case(2, 1, 1500, 128, 576, 700, 16, [900, 1500], True).select(), False),
             (Case(1, 90, 400, 64, 576, 128).select(), False),
             (Case(1, 70, 300, 24, 576, 8, seed=1), True), (Case(2, 1, 2000, 16, 576, 8, 0, None, True), True)]
    want = [c.run(dense=d) for c, d in cases]
    ws = [dsa.alloc_workspace8(c.shape) for c, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases[:2]]
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        c, d = cases[i % 4]
        with torch.cuda.stream(streams[i % 4 // 2]):
            got.append((i % 4, c.run(dense=d, ws=ws[i % 4])))
    torch.cuda.synchronize()
    assert dsa.device_error()[0] == 0
    for i, (o, l) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1]), i


@pytest.mark.parametrize("page", [0, 32])
def test_prefill_then_decode_through_every_operator(page):
    """A prefill of 70 tokens, then three decode steps, each from raw rows;
    every selection and output against the oracle on the values that the
    caches hold, and the caches against the oracle's rows."""
    wl = Workload("chain", B=2, T=70, S=96, H_I=16, D_I=128, H=64, d_k=576, d_v=512, k=24, q_block=32, seed=0)
    raw = _prepare(wl, 11)
    rows = wl.B * wl.S
    table = None
    cache = {}
    if page:
        cache["pages"] = wl.B * 3 + 1
        rows = cache["pages"] * page
        table = torch.tensor([[5, 0, 3], [1, 6, 2]], dtype=torch.int32, device="cuda")
    cache |= dict(kv8=torch.zeros(rows, 576, dtype=torch.uint8, device="cuda"),
                  kv_scale=torch.zeros(rows, device="cuda"),
                  kI8=torch.zeros(rows, 128, dtype=torch.uint8, device="cuda"),
                  kI_scale=torch.zeros(rows, device="cuda"))
    nw = 1 + 0.1 * torch.randn(512, device="cuda")
    freq = ((10000.0 ** (-torch.arange(32, device="cuda") / 32)).float(),
            (10000.0 ** (-torch.arange(32, device="cuda") / 32)).float())

    def at(b, s):
        return b * wl.S + s if not page else int(table[b, s // page]) * page + s % page

    tau = 1 / 24.0
    for s0, s1 in ((0, 70), (70, 71), (71, 72), (72, 73)):
        sh, part, (qI8, qs), out, lse, idx = _step(wl, raw, cache, s0, s1, page, table, nw, freq)
        assert dsa.device_error()[0] == 0
        T = s1 - s0
        x = O.bf16_decode(P.u16(raw["kv"]))
        for b in range(wl.B):
            rr = [at(b, s) for s in range(s1)]
            kd = R.dequantise(cache["kI8"][rr].cpu().numpy(), cache["kI_scale"][rr].cpu().numpy())
            kv = R.dequantise(cache["kv8"][rr].cpu().numpy(), cache["kv_scale"][rr].cpu().numpy())
            for t in sorted({0, T // 2, T - 1}):
                # the cached row is the token's normed and rotated row: e4m3's half step and BF16's
                want = R.norm_rope_row(x[b, s0 + t, 0], s0 + t, nw.double().cpu().numpy(), 512, 64,
                                       freq[0].double().cpu().numpy(), 1e-6, False)
                step = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * float(cache["kv_scale"][rr[s0 + t]])
                assert (np.abs(kv[s0 + t] - want) <= step + 2.0 ** -7 * np.abs(want)).all()
                qd = R.dequantise(qI8[b, t].cpu().numpy(), qs[b, t].cpu().numpy())
                sc = O.indexer_row(qd, part["w"][b, t].double().cpu().numpy(), kd, s0 + t)
                P.check_selection(idx[b, t].cpu().numpy(), O.topk_row(sc, wl.k), sc, False, f"{s0} {b} {t}")
                q = O.bf16_decode(P.u16(part["q"][b, t]))
                o, l, A, wm = R.attention_row(q, kv, idx[b, t].cpu().numpy(), 512, tau)
                got = O.bf16_decode(P.u16(out[b, t]))
                tol = 2.0 ** -8 * np.abs(o) + 2.0 ** -7 * A + 2.0 ** -16 * wm[:, None] * 24 * np.abs(kv).max()
                assert (np.abs(got - o) <= tol).all()
                assert np.abs(lse[b, t].cpu().numpy() - l).max() <= 1e-4
    # reading the caches back gives the values they stand for
    kvr = torch.zeros(wl.B, 73, 576, dtype=torch.bfloat16, device="cuda")
    dsa.cache_read(sh, 0, 73, kv8=cache["kv8"], kv_scale=cache["kv_scale"], kv=kvr)
    got = O.bf16_decode(P.u16(kvr))
    for b in range(wl.B):
        rr = [at(b, s) for s in range(73)]
        assert np.array_equal(got[b], R.dequantise(cache["kv8"][rr].cpu().numpy(), cache["kv_scale"][rr].cpu().numpy()))


@pytest.mark.parametrize("fused", [False, True])
def test_forward8_selects_as_forward_does(fused):
    """Same indexer inputs: the same selection, and the attention over it."""
    wl = Workload("f8", B=1, T=300, S=32768, H_I=32, D_I=128, H=16, d_k=576, d_v=512, k=256, q_block=150, seed=3)
    inp = make_inputs(wl, "cuda")
    inp.pop("needle_pos", None)
    sh = dsa.make_shape(wl)
    outs = dsa.alloc_outputs(wl)
    dsa.forward(sh, inp, outs.out, outs.lse, outs.idx, dsa.alloc_workspace(sh))
    kv8 = torch.empty(wl.S, 576, dtype=torch.uint8, device="cuda")
    sc = torch.empty(wl.S, device="cuda")
    whole = dsa.make_shape(None, B=1, T=wl.S, S=wl.S, H_I=32, D_I=128, H=16, d_k=576, d_v=512, k=256, q_block=1)
    dsa.cache_write(whole, kv=inp["kv"], kv8=kv8, kv_scale=sc)
    n = dsa.workspace8_size(sh)
    if fused:
        n -= dsa.workspace_size(sh) - dsa.select_workspace_size(sh)
        small = torch.empty(n - 512, dtype=torch.uint8, device="cuda")
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty(1, 300, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 300, 16, device="cuda")
    idx = torch.empty(1, 300, 256, dtype=torch.int32, device="cuda")
    i8 = {m: inp[m] for m in ("q_I", "q_scale", "w", "k_I", "k_scale", "q")} | dict(kv8=kv8, kv_scale=sc)
    dsa.forward8(sh, i8, out, lse, idx, ws)
    assert dsa.device_error()[0] == 0
    assert torch.equal(idx.sort(-1).values, outs.idx.sort(-1).values)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    dsa.sparse_attn8(sh, inp["q"], kv8, sc, idx, o2, l2, dsa.alloc_workspace8(sh))
    # forward8 takes rows that keep every key densely: none here
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    if fused:
        with pytest.raises(dsa.DsaError) as e:
            dsa.forward8(sh, i8, out, lse, idx, small)
        assert e.value.code == 3


def test_forward8_short_prefill_is_dense():
    """k covers every key: the selection is all visible keys, the output the dense form's."""
    wl = Workload("f8d", B=2, T=40, S=60, H_I=16, D_I=128, H=64, d_k=576, d_v=512, k=64, q_block=40, seed=3)
    inp = make_inputs(wl, "cuda")
    inp.pop("needle_pos", None)
    c = Case(2, 40, 60, 64, 576, 64)
    out = torch.empty(2, 40, 64, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 40, 64, device="cuda")
    idx = torch.empty(2, 40, 64, dtype=torch.int32, device="cuda")
    sh = dsa.make_shape(wl)
    i8 = {m: inp[m] for m in ("q_I", "q_scale", "w", "k_I", "k_scale")} | dict(q=c.q, kv8=c.kv8, kv_scale=c.scale)
    dsa.forward8(sh, i8, out, lse, idx, dsa.alloc_workspace8(sh))
    c.check(out, lse, dense=True, rows=[0, 17, 39])
    for t in (0, 39):
        assert sorted(idx[1, t].tolist()) == sorted(list(range(21 + t)) + [-1] * (43 - t))
