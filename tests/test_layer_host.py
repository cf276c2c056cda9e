"""The decode-layer calls without a GPU: their argument checks (nothing here launches a kernel),
and the oracle's forms of them against closed forms."""
import ctypes
import math

import numpy as np
import pytest

from oracle import layer
from tiered_weight_gemv_b200 import spax

A = 1 << 20  # an aligned address that is never dereferenced


def cache(**kw):
    c = dict(n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, dtype=spax.KV_BF16, k_scale=1.0,
             v_scale=1.0, reserved=0, page_stride=16 * 128, token_stride=128, head_stride=64, d_k=A,
             d_v=2 * A)
    c.update(kw)
    return spax.spax_kv_cache(*[c[f] for f, _ in spax.spax_kv_cache._fields_])


BAD_CACHES = [
    (dict(d_k=None), spax.ERR_ARG), (dict(d_v=None), spax.ERR_ARG), (dict(dtype=2), spax.ERR_ARG),
    (dict(n_pages=0), spax.ERR_SHAPE), (dict(page_size=0), spax.ERR_SHAPE),
    (dict(n_kv_heads=0), spax.ERR_SHAPE), (dict(head_dim=0), spax.ERR_SHAPE),
    (dict(head_dim=72), spax.ERR_SHAPE), (dict(head_dim=272), spax.ERR_SHAPE),
    (dict(k_scale=0.5), spax.ERR_ARG),  # a bf16 cache holds the values themselves
    (dict(dtype=spax.KV_E4M3, k_scale=0.0), spax.ERR_ARG),
    (dict(dtype=spax.KV_E4M3, v_scale=math.inf), spax.ERR_ARG),
    (dict(dtype=spax.KV_E4M3, v_scale=math.nan), spax.ERR_ARG),
    (dict(d_k=A + 8), spax.ERR_ARG), (dict(d_v=A + 2), spax.ERR_ARG),
    (dict(head_stride=68), spax.ERR_ARG), (dict(token_stride=32), spax.ERR_ARG),
    (dict(page_stride=-2048), spax.ERR_ARG), (dict(page_stride=0), spax.ERR_ARG),
    (dict(page_stride=1 << 62), spax.ERR_SHAPE),
    (dict(dtype=spax.KV_E4M3, token_stride=136), spax.ERR_ARG),  # 8 bytes off a 16-byte step
]


def append(c=None, rope=None, **kw):
    a = dict(q=A, qs=256, k=A, ks=128, v=A, vs=128, n=3, H=4, seq=A, pos=A, table=A, n_seq=3,
             max_pages=4, q_out=A, qos=256)
    a.update(kw)
    c = cache() if c is None else c
    return spax._lib.spax_kv_append(
        ctypes.byref(c), a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["n"], a["H"],
        a["seq"], a["pos"], a["table"], a["n_seq"], a["max_pages"],
        None if rope is None else ctypes.byref(spax.spax_rope(*rope)), a["q_out"], a["qos"], None,
        None)


def attention(c=None, prm=(0.1, 0.0, 0), **kw):
    a = dict(q=A, qs=256, n=3, H=4, table=A, max_pages=4, lens=A, out=4 * A, ws=A, ws_bytes=1 << 30)
    a.update(kw)
    c = cache() if c is None else c
    return spax._lib.spax_paged_attention(
        ctypes.byref(c), a["q"], a["qs"], a["n"], a["H"], a["table"], a["max_pages"], a["lens"],
        None if prm is None else ctypes.byref(spax.spax_attn_params(*prm)), a["out"], None, None,
        a["ws"], a["ws_bytes"], None)


def residual(post=None, pre=None, **kw):
    a = dict(h=A, y=2 * A, n=2, d=64, gate=None, gs=0, rs=1.0, os=1.0, r=3 * A, x=4 * A)
    a.update(kw)
    ref = [None if p is None else ctypes.byref(spax.spax_norm(*p)) for p in (post, pre)]
    return spax._lib.spax_residual_norm(a["h"], a["y"], a["n"], a["d"], ref[0], a["gate"], a["gs"],
                                        a["rs"], a["os"], ref[1], a["r"], a["x"], None)


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_cache_descriptions_are_checked(change, want):
    assert append(cache(**change)) == want
    assert attention(cache(**change)) == want


def test_a_null_cache_is_refused():
    assert spax._lib.spax_kv_append(None, A, 256, A, 128, A, 128, 1, 4, A, A, A, 1, 1, None, A, 256,
                                    None, None) == spax.ERR_ARG
    prm = spax.spax_attn_params(1.0, 0.0, 0)
    assert spax._lib.spax_paged_attention(None, A, 256, 1, 4, A, 1, A, ctypes.byref(prm), 4 * A,
                                          None, None, A, 1 << 30, None) == spax.ERR_ARG


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), spax.ERR_SHAPE), (dict(H=-1), spax.ERR_SHAPE), (dict(n_seq=-1), spax.ERR_SHAPE),
    (dict(q=None), spax.ERR_ARG), (dict(H=0), spax.ERR_ARG), (dict(k=None), spax.ERR_ARG),
    (dict(v=None), spax.ERR_ARG), (dict(q_out=None), spax.ERR_ARG), (dict(pos=None), spax.ERR_ARG),
    (dict(table=None), spax.ERR_ARG), (dict(n_seq=0), spax.ERR_ARG),
    (dict(seq=None, n=4), spax.ERR_ARG),  # more tokens than sequences
    (dict(max_pages=0), spax.ERR_SHAPE), (dict(max_pages=1 << 27), spax.ERR_SHAPE),
    (dict(q=A + 4), spax.ERR_ARG), (dict(k=A + 8), spax.ERR_ARG), (dict(v=A + 12), spax.ERR_ARG),
    (dict(q_out=A + 4), spax.ERR_ARG), (dict(qs=252), spax.ERR_ARG), (dict(ks=130), spax.ERR_ARG),
    (dict(vs=0), spax.ERR_ARG), (dict(qos=258), spax.ERR_ARG), (dict(qos=512), spax.ERR_ARG),
    (dict(ks=(1 << 32) + 4), spax.ERR_ARG), (dict(vs=-128), spax.ERR_ARG),
    (dict(rope=(60, 0, A)), spax.ERR_SHAPE), (dict(rope=(72, 0, A)), spax.ERR_SHAPE),
    (dict(rope=(-8, 0, A)), spax.ERR_SHAPE), (dict(rope=(64, 2, A)), spax.ERR_ARG),
    (dict(rope=(64, 0, None)), spax.ERR_ARG), (dict(rope=(64, 0, A + 4)), spax.ERR_ARG),
])
def test_append_refuses(kw, want):
    assert append(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(prm=None), spax.ERR_ARG), (dict(prm=(math.nan, 0.0, 0)), spax.ERR_ARG),
    (dict(prm=(math.inf, 0.0, 0)), spax.ERR_ARG), (dict(prm=(1.0, -1.0, 0)), spax.ERR_ARG),
    (dict(prm=(1.0, math.inf, 0)), spax.ERR_ARG), (dict(prm=(1.0, 0.0, -1)), spax.ERR_ARG),
    (dict(prm=(1.0, 1e-30, 0)), spax.ERR_ARG), (dict(prm=(1.0, 1e30, 0)), spax.ERR_ARG),
    (dict(n=65535, max_pages=1 << 20, out=1 << 40), spax.ERR_SHAPE), (dict(n=65536), spax.ERR_SHAPE),
    (dict(n=-1), spax.ERR_SHAPE), (dict(H=0), spax.ERR_SHAPE), (dict(H=5), spax.ERR_SHAPE),
    (dict(table=None), spax.ERR_ARG), (dict(lens=None), spax.ERR_ARG), (dict(out=None), spax.ERR_ARG),
    (dict(q=None), spax.ERR_ARG), (dict(q=A + 4), spax.ERR_ARG), (dict(out=4 * A + 8), spax.ERR_ARG),
    (dict(qs=200), spax.ERR_ARG), (dict(qs=258), spax.ERR_ARG), (dict(qs=1 << 62), spax.ERR_ARG), (dict(max_pages=0), spax.ERR_SHAPE),
    (dict(max_pages=1 << 27), spax.ERR_SHAPE), (dict(out=A), spax.ERR_ARG),
    (dict(out=A + 2048), spax.ERR_ARG),
])
def test_attention_refuses(kw, want):
    assert attention(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), spax.ERR_SHAPE), (dict(d=0), spax.ERR_SHAPE), (dict(d=32769), spax.ERR_SHAPE),
    (dict(h=None), spax.ERR_ARG), (dict(r=None, x=None), spax.ERR_ARG),
    (dict(y=None, post=(0, 0, A, None, 1e-5)), spax.ERR_ARG), (dict(y=None, gate=A), spax.ERR_ARG),
    (dict(rs=math.nan), spax.ERR_ARG), (dict(os=math.inf), spax.ERR_ARG),
    (dict(gate=A, gs=63), spax.ERR_ARG), (dict(gate=A, gs=-64), spax.ERR_ARG),
    (dict(gate=A, gs=1 << 62), spax.ERR_ARG),
    (dict(pre=(2, 0, A, None, 1e-5)), spax.ERR_ARG), (dict(pre=(0, 2, A, None, 1e-5)), spax.ERR_ARG),
    (dict(pre=(0, 0, A, None, -1e-5)), spax.ERR_ARG), (dict(pre=(0, 0, A, None, math.nan)), spax.ERR_ARG),
    (dict(post=(0, 0, A + 2, None, 1e-5)), spax.ERR_ARG), (dict(post=(1, 1, A, A + 1, 1e-5)), spax.ERR_ARG),
    (dict(r=4 * A), spax.ERR_ARG), (dict(r=A + 16), spax.ERR_ARG), (dict(x=2 * A + 256), spax.ERR_ARG),
    (dict(gate=3 * A), spax.ERR_ARG),
])
def test_residual_norm_refuses(kw, want):
    assert residual(**kw) == want


def test_nothing_to_do_is_no_error():
    assert append(n=0) == spax.OK
    assert attention(n=0) == spax.OK
    assert residual(n=0) == spax.OK


def test_workspace_sizes_refuse_unsupported_layouts():
    for H, K, D in [(0, 1, 64), (4, 0, 64), (5, 2, 64), (4, 2, 8), (4, 2, 72), (4, 2, 512)]:
        assert spax.spax_attention_workspace_bytes(H, K, D) == 0


# ---- the oracle's forms against closed forms

def test_oracle_rotation_keeps_relative_angles():
    rng = np.random.default_rng(1)
    f = 10000.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        a, b = rng.normal(size=(2, 1, 1, 24))
        dots = [np.sum(layer.rotate(a, [p], f, inter) * layer.rotate(b, [p + 5], f, inter))
                for p in (0, 3, 1000)]
        assert np.ptp(dots) <= 1e-9
        assert np.allclose(layer.rotate(a, [0], f, inter), a)
        assert np.array_equal(layer.rotate(a, [9], f, inter)[..., 16:], a[..., 16:])
        quarter = layer.rotate(a, [1], [np.pi / 2], inter)  # a quarter turn of the first pair
        assert np.allclose(quarter[0, 0, :2], [-a[0, 0, 1], a[0, 0, 0]])


def test_oracle_attention_of_equal_keys_is_the_mean():
    rng = np.random.default_rng(2)
    k = np.ones((3, 4, 1, 16))
    v = rng.normal(size=(3, 4, 1, 16))
    q = rng.normal(size=(2, 2, 16))
    table = np.array([[2, 0], [1, 7]])
    out, lse, _, _ = layer.attention(q, k, v, table, [6, 0], 0.5)
    rows = np.concatenate([v[2, :, 0], v[0, :2, 0]])
    assert np.allclose(out[0], rows.mean(0)) and np.all(out[1] == 0) and np.all(lse[1] == -np.inf)
    assert np.allclose(lse[0], 0.5 * q[0].sum(-1) + np.log(6))
    out, _, _, _ = layer.attention(q, k, v, table, [6, 8], 0.5, window=1)
    assert np.allclose(out[0], v[0, 1, 0])
    assert np.all(out[1] == 0)  # its only position is on a page that is not there
    out, lse, _, _ = layer.attention(q, k, v, table, [6, 9], 0.5, softcap=1e-9)
    assert np.allclose(out[0], rows.mean(0)) and np.allclose(lse[0], np.log(6)) and np.all(out[1] == 0)


def test_oracle_norms():
    z = np.array([[3.0, -4.0]])
    assert np.allclose(layer.norm(z, None, None, 0.0, False), z / np.sqrt(12.5))
    assert np.allclose(layer.norm(z, [2, 2], [1, 1], 0.0, True), [[3, -1]])
    r, x = layer.residual_norm(z, 2 * z, gate=[1, 0], res_scale=0.5, out_scale=3.0)
    assert np.allclose(r, [[19.5, -2.0]]) and np.array_equal(r, x)
