"""spax_residual_norm against the fp64 oracle.

Tolerances, with u = 2^-24. A sum over a row of d values is taken by at least 32 threads, at most
d / 32 + 1 values each (serially) and a tree of at most 12 levels: relative to the sum of the
absolute terms it is off by e = (d / 32 + 14) u. The mean square is then off by e + 2 u relative, its
root's reciprocal by (e + 2 u) / 2 + 3 u (sum with eps, root, division). A normed entry n_i w + b
carries that, the deviation's own error and three more roundings; a mean (LAYER) is off by
e * mean|z|, which moves every deviation by as much.
"""
import numpy as np
import pytest
import torch

from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

if cuda_ok():
    from oracle import layer
    from tiered_weight_gemv_b200 import spax

U = 2.0 ** -24


def norm_tol(z, dz, w, b, eps, is_layer):
    """Bound of the normed rows' error when the rows z carry errors up to dz."""
    d = z.shape[-1]
    e = (d / 32 + 14) * U
    w = np.ones(d) if w is None else np.abs(w)
    b = np.zeros(d) if b is None else np.abs(b)
    shift = np.zeros(z.shape[:-1] + (1,))
    if is_layer:
        shift = e * np.abs(z).mean(-1, keepdims=True) + dz.mean(-1, keepdims=True)
        z = z - z.mean(-1, keepdims=True)
    dev = dz + shift + np.abs(z) * U
    ms = (z * z).mean(-1, keepdims=True) + eps
    inv = 1 / np.sqrt(ms)
    # the mean square moves by 2 |z| dev + dev^2 on average
    rel = ((2 * np.abs(z) * dev + dev * dev).mean(-1, keepdims=True) / ms + e + 2 * U) / 2 + 3 * U
    n = np.abs(z) * inv
    return 1.01 * ((dev * inv + n * rel + 2 * n * U) * w + (n * w + b) * U) + 1e-37


def make(n, d, kind, wt, post, gate, seed=0):
    torch.manual_seed(seed)
    t = torch.float32 if wt == "fp32" else torch.bfloat16
    vec = lambda s, m: (torch.randn(d, device="cuda") * s + m).to(t)  # noqa: E731
    is_layer = kind == 1
    pre = spax.Norm(vec(0.3, 1.0), vec(0.3, 0.0) if is_layer else None, kind=kind)
    po = spax.Norm(vec(0.3, 1.0), vec(0.3, 0.0) if is_layer else None, eps=1e-6, kind=kind)
    g = {None: None, "row": torch.randn(d, device="cuda"),
         "token": torch.randn(n, d, device="cuda")}[gate]
    h, y = torch.randn(n, d, device="cuda") * 3 + 0.5, torch.randn(n, d, device="cuda") - 0.25
    return h, y, pre, po if post else None, g


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(h, y, pre, post, gate, rs, os_, r, x):
    hn, yn = f64(h), f64(y)
    dz = 0.0
    z = yn
    if y is not None and post is not None:
        w, b = f64(post.weight), f64(post.bias)
        eps = float(np.float32(post.eps))
        z = layer.norm(yn, w, b, eps, post.kind == 1)
        dz = norm_tol(yn, np.zeros_like(yn), w, b, eps, post.kind == 1)
    rs, os_ = float(np.float32(rs)), float(np.float32(os_))
    want = rs * hn
    dr = np.abs(want) * 2 * U
    if y is not None:
        g = np.ones(1) if gate is None else f64(gate)
        part = os_ * g * z
        want = want + part
        dr = dr + np.abs(os_ * g) * dz + 3 * U * np.abs(part) + U * np.abs(want)
    dr = 1.01 * dr + 1e-37
    if r is not None:
        assert np.all(np.abs(f64(r) - want) <= dr)
    if x is not None:
        if pre is None:
            assert np.all(np.abs(f64(x) - want) <= dr)
        else:
            w, b, eps = f64(pre.weight), f64(pre.bias), float(np.float32(pre.eps))
            wx = layer.norm(want, w, b, eps, pre.kind == 1)
            assert np.all(np.abs(f64(x) - wx) <= norm_tol(want, dr, w, b, eps, pre.kind == 1))


@pytest.mark.parametrize("n,d", [(1, 1), (1, 4096), (3, 5), (2, 33), (7, 1000), (5, 4097), (2, 8192),
                                 (150, 512), (331, 2049), (1, 32768), (3, 28672), (1, 32767),
                                 (700, 64), (160, 16384)])
@pytest.mark.parametrize("kind,wt,post,gate", [(0, "bf16", False, None), (1, "fp32", True, "token"),
                                               (0, "fp32", True, "row"), (1, "bf16", False, "row")])
def test_against_the_oracle(n, d, kind, wt, post, gate):
    h, y, pre, po, g = make(n, d, kind, wt, post, gate, n + d)
    r, x = torch.full_like(h, float("nan")), torch.full_like(h, float("nan"))
    spax.spax_residual_norm(h, y, r, x, pre=pre, post=po, gate=g, res_scale=0.75, out_scale=-1.5)
    check(h, y, pre, po, g, 0.75, -1.5, r, x)


@pytest.mark.parametrize("n,d", [(2, 260), (3, 4099), (200, 1024), (1, 16384)])
def test_optional_parts(n, d):
    h, y, pre, post, g = make(n, d, 0, "fp32", True, "row")
    for kw in [dict(y=None, r=False), dict(y=None, pre=None), dict(pre=None), dict(r=False, pre=None),
               dict(x=False), dict(x=False, pre=None, post=None), dict(gate=None, post=None)]:
        a = dict(y=y, pre=pre, post=post, gate=g, r=True, x=True)
        a.update(kw)
        if a["y"] is None:
            a.update(post=None, gate=None)
        r = torch.full_like(h, float("nan")) if a["r"] else None
        x = torch.full_like(h, float("nan")) if a["x"] else None
        spax.spax_residual_norm(h, a["y"], r, x, pre=a["pre"], post=a["post"], gate=a["gate"])
        check(h, a["y"], a["pre"], a["post"], a["gate"], 1.0, 1.0, r, x)
    for kind in (0, 1):  # no weights at all
        r, x = torch.empty_like(h), torch.empty_like(h)
        nn = spax.Norm(kind=kind)
        spax.spax_residual_norm(h, y, r, x, pre=nn, post=nn)
        check(h, y, nn, nn, None, 1.0, 1.0, r, x)


@pytest.mark.parametrize("n,d", [(1, 4096), (300, 1028), (2, 16384), (3, 257)])
def test_in_place_outputs(n, d):
    h, y, pre, post, g = make(n, d, 0, "bf16", True, "token")
    r, x = torch.empty_like(h), torch.empty_like(h)
    spax.spax_residual_norm(h, y, r, x, pre=pre, post=post, gate=g)
    for swap in (False, True):
        a, b = h.clone(), y.clone()
        spax.spax_residual_norm(a, b, *((b, a) if swap else (a, b)), pre=pre, post=post, gate=g)
        assert torch.equal(b if swap else a, r) and torch.equal(a if swap else b, x)


@pytest.mark.parametrize("d", [512, 515])
def test_unaligned_rows(d):
    """Rows whose addresses are 4 bytes off a 16-byte boundary."""
    h, y, pre, post, g = make(4, d, 1, "bf16", True, "token")
    big = torch.empty(5, 4 * d + 1, device="cuda")
    hs, ys, r, x, gs = (big[i, 1:].view(4, d) for i in range(5))
    hs.copy_(h), ys.copy_(y), gs.copy_(g)
    wide = torch.empty(4, d + 1, dtype=torch.bfloat16, device="cuda")
    un = [spax.Norm(wide[2 * i, 1:], wide[2 * i + 1, 1:], eps=m.eps, kind=1) for i, m in enumerate((pre, post))]
    for u, m in zip(un, (pre, post)):
        u.weight.copy_(m.weight), u.bias.copy_(m.bias)
    spax.spax_residual_norm(hs, ys, r, x, pre=un[0], post=un[1], gate=gs)
    check(h, y, pre, post, g, 1.0, 1.0, r, x)


def test_extreme_rows():
    """All zero rows, a constant row (its deviations are zero) and large and small magnitudes."""
    d = 2048
    for kind in (0, 1):
        n = spax.Norm(kind=kind)
        h = torch.zeros(4, d, device="cuda")
        h[1] = 3.5
        h[2] = torch.randn(d, device="cuda") * 1e15
        h[3] = torch.randn(d, device="cuda") * 1e-12
        x = torch.empty_like(h)
        spax.spax_residual_norm(h, None, None, x, pre=n)
        check(h, None, n, None, None, 1.0, 1.0, None, x)
        assert torch.all(x[0] == 0)
        bad = torch.randn(3, d, device="cuda")
        bad[1, 5] = float("nan")
        x = torch.empty_like(bad)
        spax.spax_residual_norm(bad, None, None, x, pre=n)
        assert torch.isnan(x[1]).all() and torch.isfinite(x[0]).all() and torch.isfinite(x[2]).all()


def test_captured_and_repeated_calls_give_the_same_bits():
    for n, d in [(1, 4096), (2, 16384), (190, 2048)]:
        h, y, pre, post, g = make(n, d, 0, "bf16", True, "row")
        r, x = torch.empty_like(h), torch.empty_like(h)
        spax.spax_residual_norm(h, y, r, x, pre=pre, post=post, gate=g)
        want = r.clone(), x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            spax.spax_residual_norm(h, y, r, x, pre=pre, post=post, gate=g)
        for _ in range(3):
            r.zero_(), x.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(r, want[0]) and torch.equal(x, want[1])


def test_the_binding_refuses():
    h, y, pre, post, g = make(3, 64, 0, "fp32", True, "token")
    r, x = torch.empty_like(h), torch.empty_like(h)
    for kw, err in [(dict(h=h.cpu()), TypeError), (dict(y=y.half()), TypeError),
                    (dict(r=r[:2]), ValueError), (dict(x=x.t()), ValueError),
                    (dict(gate=g[:2]), ValueError), (dict(h=h[:, ::2]), ValueError),
                    (dict(pre=spax.Norm(torch.ones(32, device="cuda"))), ValueError),
                    (dict(r=x), spax.SpaxError), (dict(y=None), spax.SpaxError)]:
        a = dict(h=h, y=y, r=r, x=x, pre=pre, post=post, gate=g)
        a.update(kw)
        with pytest.raises(err):
            spax.spax_residual_norm(**a)
    with pytest.raises(TypeError):
        spax.Norm(torch.ones(8, device="cuda"), torch.ones(8, device="cuda").half())
