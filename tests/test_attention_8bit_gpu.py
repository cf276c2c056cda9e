"""spax_paged_attention beside an 8-bit cache where a head's queries or probabilities span many powers
of two, against the fp64 oracle.

Tolerances, with u = 2^-24 and the names of test_paged_attention_gpu. Two fp16 parts (11 bits, and 11 of
the remainder, which has up to 12) leave at most 2 u of a value; a query entry, in units that bring the
head's largest Q below 2^15, is held in steps of 2^-24 * 2^-12 at least, so off by up to 2^-37 there,
which is 2^-51 Q; a probability, lifted so that the largest is 2^12 at least, likewise by 2^-49 of the
largest. So a score is off by 2 u A from its entries, D u A from its D / 2 steps of addition, a few u A
from its factors and 2^-51 Q sum_i |scale k_i|, together within dS = 2 D u A + 2^-51 Q sum_i |scale k_i|;
x follows from it as there; and the outputs carry 2^-49 sum_j |v_j| more than there, the sum of
probabilities being at least the largest.
"""
import numpy as np
import pytest
import torch

from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

if cuda_ok():
    from oracle import layer
    from test_paged_attention_gpu import U, Case

SHAPES = [(8, 1, 128), (4, 2, 64), (16, 1, 128), (16, 1, 64), (8, 2, 256), (3, 1, 80)]


def check(case, out, lse):
    keys = case.c.k.float().double().cpu().numpy() * np.float64(np.float32(case.c.k_scale))
    vals = case.c.v.float().double().cpu().numpy() * np.float64(np.float32(case.c.v_scale))
    scale = np.float64(np.float32(case.scale))
    table, lens, q = case.table.cpu().numpy(), case.lens.cpu().numpy(), case.q.double().cpu().numpy()
    o, ls, A, spread = layer.attention(q, keys, vals, table, lens, scale)
    keys_sum = layer.attention(np.ones_like(q), keys, vals, table, lens, scale)[2]
    mean = layer.attention(np.zeros_like(q), keys, vals, table, lens, scale)[3]  # of |v_j|
    dS = 2 * case.D * U * A + 2.0 ** -51 * np.abs(q).max(-1) * keys_sum
    x = 2 * dS + 8 * U * A + 8 * U
    L = np.array(case.lens_l)[:, None]
    steps = (L / 64 + 160) * U
    tol = (2 * x + 4 * steps)[:, :, None] * spread + 2.0 ** -49 * L[:, :, None] * mean
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= tol)
    assert np.all(np.abs(lse.double().cpu().numpy() - ls) <= x + 2 * steps + 2 * U * np.abs(ls))
    assert case.status.item() == 0


@pytest.mark.parametrize("H,K,D", SHAPES)
@pytest.mark.parametrize("big", [1e4, 1e6, 1e9])
def test_a_large_query_entry_takes_nothing_from_the_others(H, K, D, big):
    """One entry far above the others of its head, on a channel where every key is zero."""
    case = Case([1, 33, 700], H, K, D, 1, 16, seed=D)
    raw = case.c.k.view(torch.uint8)
    raw[..., 5] = torch.where(raw[..., 5] == 0x7F, raw[..., 5], torch.zeros_like(raw[..., 5]))
    case.q[..., 5] = big / case.c.k_scale
    check(case, *case.run())


@pytest.mark.parametrize("H,K,D", SHAPES)
@pytest.mark.parametrize("gap", [12.0, 18.0, 24.0])
def test_small_probabilities_beside_a_position_of_zero_values(H, K, D, gap):
    """The first position takes nearly all of the sum and has values of zero: the output is what the
    others, e^-gap each, make of theirs."""
    case = Case([9, 40, 300], H, K, D, 1, 16, seed=D)
    case.q.zero_()
    case.q[..., 0] = gap / 16 / case.c.k_scale
    case.scale = 1.0
    k, v = case.c.k.view(torch.uint8), case.c.v.view(torch.uint8)
    sixteen = torch.tensor(16.0, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    for i, n in enumerate(case.lens_l):
        t = torch.arange(n, device="cuda")
        pg = case.table[i].long()[t // 16]
        k[pg, t % 16, :, 0] = 0
        k[pg[0], 0, :, 0] = sixteen
        v[pg[0], 0] = 0
    check(case, *case.run())
