"""Attention over an 8-bit cache at the ends of its inputs' ranges, on the GPU."""
import pytest
import torch

from long_context_05_b200 import dsa
from tests.test_gpu_attn8 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("B,T,H,d_k,k,dense,page", [
    (1, 1, 128, 576, 600, False, 0),                   # a chunk to a part
    (20, 1, 128, 576, 600, False, 16),                 # two chunks to a part
    (1, 80, 128, 576, 600, False, 0),                  # one part
    (1, 1, 24, 576, 8, True, 0),
    (1, 100, 40, 576, 8, True, 0),                     # several queries to a CTA
    (1, 1, 16, 80, 300, False, 0),
    (1, 160, 128, 80, 300, False, 0),
])
def test_queries_that_are_no_numbers(bad, B, T, H, d_k, k, dense, page):
    """NaN out and lse in the rows that hold one, split or not; the other rows as without them."""
    c = Case(B, T, 700, H, d_k, k, page, seed=3)
    if not dense:
        c.select()
    want = c.run(dense=dense)
    rows = [(0, 0, 0), (B - 1, T - 1, H - 1), (0, T // 2, H // 2)]
    for i, (b, t, h) in enumerate(rows):
        c.q[b, t, h, (0, d_k - 1, 65)[i]] = bad
    out, lse = c.run(dense=dense)
    assert dsa.device_error()[0] == 0
    hit = torch.zeros(B, T, H, dtype=torch.bool, device="cuda")
    for r in rows:
        hit[r] = True
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])


@pytest.mark.parametrize("exps", [[-30.0, 34.0], [-100.0, -36.0], [36.0, 60.0, 100.0], [-64.0, 0.0]])
@pytest.mark.parametrize("T,S,dense", [(1, 900, False), (80, 900, False), (3, 900, True), (80, 2900, True)])
def test_scales_two_to_the_64_apart(T, S, dense, exps):
    """Keys of about the same weight, whose scales are as far apart as they may be."""
    c = Case(1, T, S, 128, 576, 700, exps=torch.tensor(exps, device="cuda"), tau=2.0 ** -(max(exps) + 10))
    if not dense:
        c.select()
    c.check(*c.run(dense=dense), dense=dense, rows=sorted({0, T // 2, T - 1}))


@pytest.mark.parametrize("T", [1, 80])
@pytest.mark.parametrize("size,exps,tau", [(118, [-100.0, -99.0], 2.0 ** -30), (-108, [99.0, 100.0], 2.0 ** -4),
                                           (-116, [99.0, 100.0], 2.0 ** 4)])
def test_queries_near_the_ends_of_bf16(T, size, exps, tau):
    """Queries far from one beside scales that bring their logits back."""
    c = Case(1, T, 300, 128, 576, 200, exps=torch.tensor(exps, device="cuda"), tau=tau).select()
    c.q *= 2.0 ** size
    c.check(*c.run(), rows=[0, T - 1])


def test_dense_rows_in_front_of_unfinished_ones():
    """Keys past a query's own position are not read where a CTA holds one query: its results are those of its keys."""
    c = Case(1, 40, 100, 64, 576, 8)
    c.kv8[90:] = 0x7F
    c.scale[90:] = float("inf")
    out, lse = c.run(dense=True)
    c.check(out[:, :30].contiguous(), lse[:, :30].contiguous(), dense=True, rows=[0, 1, 15, 28, 29])


@pytest.mark.parametrize("B,T,H,dense", [(1, 160, 8, False), (2, 100, 24, False), (3, 80, 64, True)])
def test_calls_of_many_rows_need_no_workspace(B, T, H, dense):
    """Enough rows for every SM in this call, few in the other kind's: nothing is split, so nothing is asked for."""
    c = Case(B, T, 300, H, 576, 100)
    if not dense:
        c.select()
    want = c.run(dense=dense)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    if dense:
        dsa.dense_attn8(c.shape, c.q, c.kv8, c.scale, out, lse, None)
    else:
        dsa.sparse_attn8(c.shape, c.q, c.kv8, c.scale, c.idx, out, lse, None)
    assert dsa.device_error()[0] == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
