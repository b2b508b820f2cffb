"""Norm and rotation of rows of very different sizes without an eps, on the GPU:
forward and backward against the FP64 oracle, at the tolerances of
test_gpu_norm_rope.py (relative to each row's own size)."""
import pytest
import torch

from long_context_05_b200 import dsa
from tests.test_gpu_norm_rope import Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    dsa.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("D,norm,rope,inter", [(576, 512, 64, False), (128, 128, 64, True), (64, 64, 0, False),
                                               (1024, 1024, 128, False)])
@pytest.mark.parametrize("exps", [(-58, -44, -30), (-10, 0, 10), (25, 40, 55)])
def test_rows_of_any_size_without_eps(D, norm, rope, inter, exps):
    c = Case(2, 3, 50, 4, 1, D, norm, rope, inter, eps=0.0)
    for t, e in enumerate(exps):
        for n in c.x:
            c.x[n][:, t, :, :norm] *= 2.0 ** e
    check(c)
