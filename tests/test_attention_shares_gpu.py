"""spax_paged_attention where rows fill more than half the wave, so that all units are dealt in equal
shares: a CTA ends a row, takes whole ones and begins another, and long rows spread over many CTAs.
Against the fp64 oracle with the bounds of test_paged_attention_gpu."""
import numpy as np
import pytest
import torch

from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

if cuda_ok():
    from tiered_weight_gemv_b200 import spax
    from test_paged_attention_gpu import Case


def lengths(n, seed):
    """Up to 400, some empty, and a long one among them."""
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(0, 400, n)]
    for i in (0, n // 3, n // 3 + 1, n - 1):
        lens[i] = 0
    lens[n // 2] = 5003
    return lens


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("window", [0, 90, 1000])
@pytest.mark.parametrize("H,K,D,page", [(8, 8, 64, 16), (32, 8, 128, 16), (16, 8, 256, 21), (96, 8, 64, 64),
                                        (80, 8, 128, 16), (16, 8, 80, 8), (72, 8, 256, 16)])
def test_equal_shares(H, K, D, page, window, dtype):
    case = Case(lengths(60, H + D), H, K, D, dtype, page, seed=D)
    first = case.run(window)
    assert case.status.item() == 0
    case.check(*first, window)
    for _ in range(10):
        again = case.run(window)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("n", [127, 128, 129, 300])
def test_equal_shares_around_128_sequences(n, dtype):
    case = Case(lengths(n, n), 16, 4, 64, dtype, 16, seed=n)
    first = case.run()
    case.check(*first)
    for _ in range(10):
        again = case.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    out, lse = case.run(200, 30.0)
    assert case.status.item() == 0
    case.check(out, lse, 200, 30.0)


@pytest.mark.parametrize("H,K,D", [(32, 8, 128), (96, 8, 64)])
def test_equal_shares_of_bad_lengths_and_pages(H, K, D):
    """A length past the table and a page outside the pool in the middle of the shares."""
    lens = lengths(60, 7)
    case = Case(lens, H, K, D, 0, 16, seed=7)
    long = 30
    case.table[long, 100] = case.c.n_pages
    case.lens[10] = case.table.shape[1] * 16 + 1
    case.lens_l = lens[:10] + [0] + lens[11:]
    out, lse = case.run()
    assert case.status.item() == spax.ERR_INDEX
    case.check(out, lse)
