"""The decode-layer calls at the edges of what they allow, without a GPU (nothing here launches a
kernel)."""
import ctypes

import pytest

from test_layer_host import A, append, attention, cache, residual
from tiered_weight_gemv_b200 import spax

SMS = 148
NO_WINDOW = 2 ** 31 - 1


@pytest.mark.parametrize("H,K,D", [(4, 4, 64), (32, 8, 128), (16, 1, 128), (71, 1, 64), (16, 2, 256), (40, 1, 80)])
@pytest.mark.parametrize("dtype", [spax.KV_BF16, spax.KV_E4M3])
def test_attention_never_takes_more_ctas_than_its_workspace_has_slots(H, K, D, dtype):
    """A CTA owns two slots (two counters, a part of 8 or 16 heads, their maxima and sums twice), whatever
    the window: the largest ones are no window at all."""
    width = 64 if D <= 64 else 128 if D <= 128 else 256
    heads = 16 if H // K > 8 and D <= 128 else 8
    for n_seq in (1, 25, 64, 128, 65535):
        for most in (1, 63, 64, 65, 8192, 131072, 1 << 30):
            plans = {}
            for window in (0, 1, 64, 4096, 2 ** 31 - 66, 2 ** 31 - 65, 2 ** 31 - 64, 2 ** 31 - 63, NO_WINDOW):
                ctas, ws = spax.spax_attention_plan_sms(n_seq, H, K, D, dtype, most, window, SMS)
                assert 1 <= ctas <= 4 * SMS
                assert 2 * ctas * (2 * 4 + heads * (width * 4 + 16)) <= ws
                plans[window] = ctas
            assert len({plans[w] for w in plans if w == 0 or w >= most}) == 1
            assert plans[1] <= plans[64] <= plans[4096] <= plans[0]


def test_attention_plans_refuse():
    ok = dict(n_seq=3, n_heads=8, n_kv_heads=2, head_dim=64, kv_dtype=0, max_positions=64, window=0, sm_count=SMS)
    assert spax.spax_attention_plan_sms(**ok)[0] == 6  # a row of one unit each
    for change in (dict(n_seq=0), dict(n_seq=65536), dict(n_heads=0), dict(n_heads=7), dict(n_kv_heads=0),
                   dict(head_dim=72), dict(head_dim=512), dict(kv_dtype=2), dict(max_positions=0),
                   dict(max_positions=(1 << 30) + 1), dict(window=-1), dict(sm_count=0),
                   dict(sm_count=65537), dict(sm_count=2 ** 31 - 1, max_positions=1 << 30, n_seq=65535)):
        with pytest.raises(spax.SpaxError):
            spax.spax_attention_plan_sms(**{**ok, **change})


def test_empty_tensors_have_null_pointers():
    assert append(n=0, q=None, k=None, v=None, q_out=None, seq=None, pos=None, H=4) == spax.OK
    assert append(n=0, q=None, k=None, v=None, q_out=None, seq=None, pos=None, table=None, n_seq=0) == spax.OK
    assert attention(n=0, q=None, out=None, lens=None, table=None) == spax.OK
    assert residual(n=0, h=None, y=None, r=None, x=None) == spax.OK


def test_rows_of_eight_ctas_fit_a_grid():
    """2^28 rows of a cluster of 8 would be 2^31 CTAs, one more than a grid holds."""
    assert residual(n=1 << 28, d=32768) == spax.ERR_SHAPE
    assert residual(n=1 << 28, d=64) == spax.ERR_SHAPE
    assert 8 * ((1 << 28) - 1) <= 2 ** 31 - 1


@pytest.mark.parametrize("off", [1, 2, 3])
def test_pointers_off_their_elements_are_refused(off):
    for name in ("seq", "pos", "table"):
        assert append(**{name: A + off}) == spax.ERR_ARG
    for name in ("table", "lens"):
        assert attention(**{name: A + off}) == spax.ERR_ARG
    for name, at in (("h", 1), ("y", 2), ("r", 3), ("x", 4), ("gate", 8)):
        assert residual(**{name: at * A + off}) == spax.ERR_ARG
    # the calls' outputs that the helpers leave out: lse and the status word
    c, prm = ctypes.byref(cache()), ctypes.byref(spax.spax_attn_params(0.1, 0.0, 0))
    for lse, status in ((A + off, None), (None, A + off)):
        assert spax._lib.spax_paged_attention(c, A, 256, 3, 4, A, 4, A, prm, 4 * A, lse, status, A, 1 << 30,
                                              None) == spax.ERR_ARG
    assert spax._lib.spax_kv_append(c, A, 256, A, 128, A, 128, 3, 4, A, A, A, 3, 4, None, A, 256, A + off,
                                    None) == spax.ERR_ARG
