"""GPU parity of dsa_cache_write and dsa_cache_read: bytes, scales and BF16
rows equal the oracle's exactly (one rounding each way, to nearest even)."""
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


class Pool:
    """Caches of a batch, filled with marks, and where a token lies."""

    def __init__(self, B, T, S, d_k, D_I, H_I, page=0, lens=None, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + S)
        self.B, self.T, self.S, self.d_k, self.D_I, self.H_I, self.page = B, T, S, d_k, D_I, H_I, page
        self.lens = [S] * B if lens is None else lens
        kw = {}
        self.rows = B * S
        self.table = None
        if page:
            per = (S + page - 1) // page
            pages = B * per + 2
            self.table = torch.randperm(pages, generator=g, device="cuda")[:B * per].view(B, per).int()
            for b in range(B):                     # entries of pages past the length may be anything
                self.table[b, (self.lens[b] + page - 1) // page:] = 1 << 30
            self.rows = pages * page
            kw = dict(page_size=page, num_pages=pages, block_table=self.table)
        sl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.shape = dsa.make_shape(None, B=B, T=T, S=S, H_I=H_I, D_I=D_I, H=8, d_k=d_k, d_v=512 if d_k == 576 else 64,
                                    k=4, q_block=T, seqlens=sl, **kw)
        self.kv8 = torch.full((self.rows, d_k), 0x55, dtype=torch.uint8, device="cuda")
        self.kI8 = torch.full((self.rows, D_I), 0x55, dtype=torch.uint8, device="cuda")
        self.kv_scale = torch.full((self.rows,), 77.0, device="cuda")
        self.kI_scale = torch.full((self.rows,), 77.0, device="cuda")
        self.qI8 = torch.full((B, T, H_I, D_I), 0x55, dtype=torch.uint8, device="cuda")
        self.qI_scale = torch.full((B, T, H_I), 77.0, device="cuda")

    def row(self, b, s):
        if self.table is None:
            return b * self.S + s
        return int(self.table[b, s // self.page]) * self.page + s % self.page

    def write(self, kv, k_I, q_I):
        dsa.cache_write(self.shape, kv=kv, kv8=self.kv8, kv_scale=self.kv_scale, k_I=k_I, kI8=self.kI8,
                        kI_scale=self.kI_scale, q_I=q_I, qI8=self.qI8, qI_scale=self.qI_scale)

    def read(self, begin, count, kv, k_I):
        dsa.cache_read(self.shape, begin, count, kv8=self.kv8, kv_scale=self.kv_scale, kv=kv, kI8=self.kI8,
                       kI_scale=self.kI_scale, k_I=k_I)


def rows_of(g, *shape):
    """Rows of many sizes: spread norms, a zero row, ties of the rounding, the
    largest and the smallest numbers."""
    x = torch.randn(*shape, generator=g, device="cuda")
    flat = x.view(-1, shape[-1])
    n = flat.shape[0]
    flat *= torch.exp2(torch.randint(-20, 20, (n, 1), generator=g, device="cuda").float())
    x = x.bfloat16()
    flat = x.view(-1, shape[-1])
    special = [torch.zeros(shape[-1]), torch.full((shape[-1],), 448.0), torch.full((shape[-1],), -450.0),
               torch.arange(shape[-1]).float() * 0.0625 + 16, torch.full((shape[-1],), 3.3e38),
               torch.full((shape[-1],), 1e-38), torch.full((shape[-1],), 2.0 ** -45)]
    for i, s in enumerate(special):
        if i < n // 2:
            flat[2 * i] = s.bfloat16().cuda()
    return x


@pytest.mark.parametrize("B,T,S,d_k,D_I,H_I,page,lens", [
    (1, 1, 1, 576, 128, 4, 0, None),
    (2, 5, 40, 576, 128, 64, 0, [17, 40]),
    (3, 7, 40, 80, 32, 4, 16, [7, 23, 40]),
    (2, 33, 33, 80, 64, 8, 0, None),
    (5, 1, 100, 576, 64, 16, 48, [1, 16, 17, 99, 100]),
    (2, 40, 90, 576, 32, 32, 64, [64, 90]),
])
def test_write_then_read(B, T, S, d_k, D_I, H_I, page, lens):
    p = Pool(B, T, S, d_k, D_I, H_I, page, lens)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    kv, k_I, q_I = rows_of(g, B, T, d_k), rows_of(g, B, T, D_I), rows_of(g, B, T, H_I, D_I)
    p.write(kv, k_I, q_I)
    assert dsa.device_error()[0] == 0
    written = set()
    for src, dst, sc in ((kv, p.kv8, p.kv_scale), (k_I, p.kI8, p.kI_scale)):
        x, b8, s32 = O.bf16_decode(u16(src)), dst.cpu().numpy(), sc.cpu().numpy()
        for b in range(B):
            for t in range(T):
                r = p.row(b, p.lens[b] - T + t)
                written.add(r)
                want, scale = R.quantise_row(x[b, t])
                assert s32[r] == scale and np.array_equal(b8[r], want), (b, t)
        rest = sorted(set(range(p.rows)) - written)
        assert (b8[rest] == 0x55).all() and (s32[rest] == 77.0).all()
    x, b8, s32 = O.bf16_decode(u16(q_I)), p.qI8.cpu().numpy(), p.qI_scale.cpu().numpy()
    for at in np.ndindex(B, T, H_I):
        want, scale = R.quantise_row(x[at])
        assert s32[at] == scale and np.array_equal(b8[at], want), at
    # read the new tokens back, with a margin on both sides
    begin = max(0, min(p.lens) - T - 2)
    count = S - begin
    o_kv = torch.full((B, count, d_k), 77.0, dtype=torch.bfloat16, device="cuda")
    o_kI = torch.full((B, count, D_I), 77.0, dtype=torch.bfloat16, device="cuda")
    p.read(begin, count, o_kv, o_kI)
    assert dsa.device_error()[0] == 0
    for dst, sc, out in ((p.kv8, p.kv_scale, o_kv), (p.kI8, p.kI_scale, o_kI)):
        b8, s32, got = dst.cpu().numpy(), sc.cpu().numpy(), O.bf16_decode(u16(out))
        for b in range(B):
            for i in range(count):
                if begin + i >= p.lens[b]:
                    assert (got[b, i] == 77.0).all()
                    continue
                r = p.row(b, begin + i)
                want = R.dequantise(b8[r], s32[r])
                # 77 * e4m3 needs more bits than BF16 has; the written rows do not
                bf = torch.from_numpy(want).bfloat16().double().numpy()
                assert np.array_equal(got[b, i], bf)
                if r in written:
                    assert np.array_equal(got[b, i], want)


def test_parts_alone_and_an_empty_read():
    p = Pool(2, 3, 20, 80, 32, 4)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    kv, k_I, q_I = rows_of(g, 2, 3, 80), rows_of(g, 2, 3, 32), rows_of(g, 2, 3, 4, 32)
    q = Pool(2, 3, 20, 80, 32, 4)
    q.write(kv, k_I, q_I)
    dsa.cache_write(p.shape, kv=kv, kv8=p.kv8, kv_scale=p.kv_scale)
    assert torch.equal(p.kv8, q.kv8) and torch.equal(p.kv_scale, q.kv_scale) and bool((p.kI8 == 0x55).all())
    dsa.cache_write(p.shape, k_I=k_I, kI8=p.kI8, kI_scale=p.kI_scale)
    assert torch.equal(p.kI8, q.kI8) and bool((p.qI8 == 0x55).all())
    dsa.cache_write(p.shape, q_I=q_I, qI8=p.qI8, qI_scale=p.qI_scale)
    assert torch.equal(p.qI8, q.qI8) and torch.equal(p.qI_scale, q.qI_scale)
    out = torch.zeros(2, 4, 32, dtype=torch.bfloat16, device="cuda")
    dsa.cache_read(p.shape, 16, 4, kI8=p.kI8, kI_scale=p.kI_scale, k_I=out)
    assert bool((out[:, 1:] != 0).any())
    dsa.cache_read(p.shape, 20, 0, kI8=p.kI8, kI_scale=p.kI_scale,
                   k_I=out[:, :0].contiguous())
    assert dsa.device_error()[0] == 0


def test_steps_append_to_one_cache():
    """Token by token, in chunks of three, and at once: the same cache."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    S = 9
    kv, k_I, q_I = rows_of(g, 1, S, 576), rows_of(g, 1, S, 128), rows_of(g, 1, S, 4, 128)
    caches = []
    for step in (1, 3, 9):
        p = Pool(1, step, S, 576, 128, 4, 16, [S])
        table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
        for e in range(step, S + 1, step):
            sl = torch.tensor([e], dtype=torch.int32, device="cuda")
            sh = dsa.make_shape(None, B=1, T=step, S=S, H_I=4, D_I=128, H=8, d_k=576, d_v=512, k=4, q_block=1,
                                seqlens=sl, page_size=16, num_pages=3, block_table=table)
            part = slice(e - step, e)
            dsa.cache_write(sh, kv=kv[:, part].contiguous(), kv8=p.kv8, kv_scale=p.kv_scale,
                            k_I=k_I[:, part].contiguous(), kI8=p.kI8, kI_scale=p.kI_scale)
        caches.append(p)
    for p in caches[1:]:
        for n in ("kv8", "kv_scale", "kI8", "kI_scale"):
            assert torch.equal(getattr(p, n), getattr(caches[0], n))


def test_bad_pages_and_lengths_are_reported_and_nothing_else_is_touched():
    p = Pool(2, 2, 32, 80, 32, 4, 16, [32, 32])
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    kv, k_I, q_I = rows_of(g, 2, 2, 80), rows_of(g, 2, 2, 32), rows_of(g, 2, 2, 4, 32)
    good = p.table.clone()
    for bad in (-1, 1 << 30, 6):
        p.table.copy_(good)
        p.table[1, 1] = bad
        p.kv8.fill_(0x55)
        p.write(kv, k_I, q_I)
        st, det = dsa.device_error()
        assert st == 6 and det & 0xFF == 0x60
        r0 = int(good[0, 1]) * 16 + 14
        assert int((p.kv8 != 0x55).any(1).sum()) == 2 and bool((p.kv8[r0:r0 + 2] != 0x55).any(1).all())
        out = torch.full((2, 3, 80), 77.0, dtype=torch.bfloat16, device="cuda")
        dsa.cache_read(p.shape, 15, 3, kv8=p.kv8, kv_scale=p.kv_scale, kv=out)
        st, det = dsa.device_error()
        assert st == 6 and det & 0xFF == 0x60
        assert bool((out[1, 1:] == 0).all()) and bool((out[1, 0] != 0).all()) and bool((out[0] != 77.0).any())
    q = Pool(1, 2, 32, 80, 32, 4, 0, [33])
    q.write(kv[:1], k_I[:1], q_I[:1])
    assert dsa.device_error()[0] == 6
    assert bool((q.kv8[30:] != 0x55).any()) and bool((q.kv8[:30] == 0x55).all())


def test_rows_past_two_gigabytes():
    """A cache whose bytes pass 2^31: the last rows, written and read back."""
    S = (1 << 31) // 576 + 1000
    free, _ = torch.cuda.mem_get_info()
    assert free > 8 << 30
    kv8 = torch.zeros(S, 576, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(S, device="cuda")
    sh = dsa.make_shape(None, B=1, T=3, S=S, H_I=4, D_I=128, H=8, d_k=576, d_v=512, k=4, q_block=3)
    kv = torch.randn(1, 3, 576, device="cuda").bfloat16()
    dsa.cache_write(sh, kv=kv, kv8=kv8, kv_scale=sc)
    out = torch.zeros(1, 3, 576, dtype=torch.bfloat16, device="cuda")
    dsa.cache_read(sh, S - 3, 3, kv8=kv8, kv_scale=sc, kv=out)
    assert dsa.device_error()[0] == 0
    assert bool((sc[:-3] == 0).all())
    x = O.bf16_decode(u16(kv[0]))
    for t in range(3):
        b, s = R.quantise_row(x[t])
        assert np.array_equal(kv8[S - 3 + t].cpu().numpy(), b) and float(sc[S - 3 + t]) == s
        assert np.array_equal(O.bf16_decode(u16(out[0, t])), R.dequantise(b, s))


def test_written_indexer_operands_score_as_their_values():
    """The bytes and scales feed dsa_indexer_scores as they are."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    p = Pool(1, 50, 50, 576, 128, 16)
    kv = torch.randn(1, 50, 576, generator=g, device="cuda").bfloat16()
    k_I = torch.randn(1, 50, 128, generator=g, device="cuda").bfloat16()
    q_I = torch.randn(1, 50, 16, 128, generator=g, device="cuda").bfloat16()
    w = torch.randn(1, 50, 16, generator=g, device="cuda")
    p.write(kv, k_I, q_I)
    sc = torch.zeros(50, 64, device="cuda")
    dsa.indexer_scores(p.shape, p.qI8, p.qI_scale, w, p.kI8, p.kI_scale, 0, 50, sc)
    qd = R.dequantise(p.qI8[0].cpu().numpy(), p.qI_scale[0].cpu().numpy())
    kd = R.dequantise(p.kI8.cpu().numpy(), p.kI_scale.cpu().numpy())
    wn = w[0].double().cpu().numpy()
    got = sc.cpu().numpy()
    for t in range(50):
        want = O.indexer_row(qd[t], wn[t], kd, t)
        size = np.abs(wn[t]) @ np.abs(qd[t] @ kd[:t + 1].T)
        assert (np.abs(got[t, :t + 1] - want) <= 1e-5 * size).all()


def test_two_graphs_and_a_stream():
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    p = Pool(2, 4, 20, 80, 32, 4)
    kv, k_I, q_I = rows_of(g, 2, 4, 80), rows_of(g, 2, 4, 32), rows_of(g, 2, 4, 4, 32)
    out = torch.zeros(2, 4, 80, dtype=torch.bfloat16, device="cuda")
    w, r = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(w):
        p.write(kv, k_I, q_I)
    with torch.cuda.graph(r):
        dsa.cache_read(p.shape, 16, 4, kv8=p.kv8, kv_scale=p.kv_scale, kv=out)
    s = torch.cuda.Stream()
    for _ in range(2):
        kv.copy_(torch.randn_like(kv.float()))
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            w.replay()
            r.replay()
        torch.cuda.current_stream().wait_stream(s)
        x = O.bf16_decode(u16(kv))
        for b, t in np.ndindex(2, 4):
            assert np.array_equal(O.bf16_decode(u16(out[b, t])), R.dequantise(*R.quantise_row(x[b, t])))
