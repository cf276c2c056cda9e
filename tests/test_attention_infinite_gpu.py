"""spax_paged_attention over a bf16 cache that holds many infinities: what a formula of fp32 gives, where
queries and probabilities enter the products in parts of either sign."""
import pytest
import torch

from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

if cuda_ok():
    from test_paged_attention_gpu import Case

SHAPES = [(8, 8, 64), (8, 8, 128), (32, 2, 128), (24, 2, 64), (4, 4, 256)]


@pytest.mark.parametrize("H,K,D", SHAPES)
def test_an_infinite_channel_of_the_values(H, K, D):
    """+-inf at one entry of every position is +-inf there, and nothing else changes. The scores rise by
    about 2^7.5 from one tile of a warp to its next, so probabilities are held up to 2^8, where their
    lower parts are up to 1/2 of either sign."""
    L, n = 1408, 128 // K
    case = Case([L] * n, H, K, D, 0, 16, seed=D)
    t = torch.arange(L, device="cuda")
    at = [(case.table[i].long()[t // 16], t % 16) for i in range(n)]
    case.q.zero_()
    case.q[..., 0] = 1.0
    case.scale = 1.0
    for pg, rw in at:
        case.c.k[pg, rw, :, 0] = (t * 0.0406).to(torch.bfloat16)[:, None]
    ref = case.run()
    assert torch.isfinite(ref[0]).all()
    for pg, rw in at:
        case.c.v[pg, rw, :, 3] = float("inf")
        case.c.v[pg, rw, :, 9] = -float("inf")
    out, lse = case.run()
    assert torch.isposinf(out[..., 3]).all() and torch.isneginf(out[..., 9]).all()
    out[..., 3], out[..., 9] = ref[0][..., 3], ref[0][..., 9]
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("H,K,D", SHAPES)
def test_several_infinite_entries_of_a_key(H, K, D):
    """Eight entries of -inf under queries of 259, which is 260 - 1 in parts: the score is -inf and the
    position left out."""
    case = Case([50, 300], H, K, D, 0, 16, seed=3)
    case.q[..., :8] = 259.0
    for i, n in enumerate(case.lens_l):
        t = torch.arange(n, device="cuda")
        case.c.k[case.table[i].long()[t // 16], t % 16, :, :8] = 0.0
    case.c.k[int(case.table[1, 2]), 5, :, :8] = -float("inf")
    case.check(*case.run())
