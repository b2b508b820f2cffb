"""Writes of the 8-bit caches that have no place to go, on the GPU."""
import pytest
import torch

from long_context_05_b200 import dsa
from tests.test_gpu_cache8 import Pool, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("T,short", [(1, 0), (1, -3), (3, 2), (3, 0)])
def test_a_sequence_shorter_than_its_new_rows_writes_nothing(page, T, short):
    """An empty slot of a padded batch: reported, and its rows and pages are left as they were."""
    p = Pool(3, T, 32, 80, 32, 4, page, [20, 32, 9])
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    kv, k_I, q_I = rows_of(g, 3, T, 80), rows_of(g, 3, T, 32), rows_of(g, 3, T, 4, 32)
    p.write(kv, k_I, q_I)
    assert dsa.device_error()[0] == 0
    want = {n: getattr(p, n).clone() for n in ("kv8", "kv_scale", "kI8", "kI_scale", "qI8", "qI_scale")}
    lens = torch.tensor([20, short, 9], dtype=torch.int32, device="cuda")
    kw = dict(page_size=page, num_pages=p.kv8.shape[0] // page, block_table=p.table) if page else {}
    sh = dsa.make_shape(None, B=3, T=T, S=32, H_I=4, D_I=32, H=8, d_k=80, d_v=64, k=4, q_block=T, seqlens=lens, **kw)
    other = torch.randn(3, T, 80, generator=g, device="cuda").bfloat16()
    other[0], other[2] = kv[0], kv[2]
    dsa.cache_write(sh, kv=other, kv8=p.kv8, kv_scale=p.kv_scale, k_I=k_I, kI8=p.kI8, kI_scale=p.kI_scale,
                    q_I=q_I, qI8=p.qI8, qI_scale=p.qI_scale)
    st, det = dsa.device_error()
    assert st == 6 and det & 0xFF == 0x60
    for n, w in want.items():
        assert torch.equal(getattr(p, n), w), n
