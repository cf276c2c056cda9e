"""The decode-layer calls at the edges of what they allow."""
import pytest
import torch

from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

if cuda_ok():
    from tiered_weight_gemv_b200 import spax
    from test_paged_attention_gpu import Case


@pytest.mark.parametrize("window", [2 ** 31 - 65, 2 ** 31 - 64, 2 ** 31 - 1])
@pytest.mark.parametrize("dtype", [0, 1])
def test_the_largest_windows_are_none(window, dtype):
    case = Case([0, 1, 700, 3000, 64], 8, 2, 128, dtype, 16, seed=1)
    want = case.run()
    out, lse = case.run(window)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and case.status.item() == 0
    case.check(out, lse)
