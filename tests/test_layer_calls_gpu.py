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


def test_empty_batches_through_the_binding():
    def none(*shape, t=torch.float32):
        return torch.empty(0, *shape, dtype=t, device="cuda")

    c = spax.alloc_kv_cache(2, 16, 2, 64)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = spax.alloc_attention_workspace(c, 4)
    i32 = torch.int32
    for table in (none(3, t=i32), torch.zeros(2, 3, dtype=i32, device="cuda")):
        for kw in (dict(), dict(q_out=none(4, 64)), dict(seq=none(t=i32))):
            spax.spax_kv_append(c, none(4, 64), none(2, 64), none(2, 64), none(t=i32), table, st, **kw)
        spax.spax_kv_append(c, None, none(2, 64), none(2, 64), none(t=i32), table, st)
        spax.spax_paged_attention(c, none(4, 64), table, none(t=i32), none(4, 64), st, ws, scale=1.0, lse=none(4))
    spax.spax_residual_norm(none(64), none(64), none(64), none(64), pre=spax.Norm(), gate=none(64))
    torch.cuda.synchronize()
    assert st.item() == 0 and not c.k.any() and not c.v.any()
