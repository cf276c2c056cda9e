"""The decode-layer calls at the edges of what they allow."""
import pytest
import torch

from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

if cuda_ok():
    from oracle import layer
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


def test_what_a_descriptor_is_formed_from_is_fixed():
    """Setting an attribute that a call would not see is refused, and the object stays as it was."""
    c = spax.alloc_kv_cache(2, 16, 2, 64, spax.KV_E4M3, k_scale=0.5)
    rope = spax.Rope(torch.ones(8, dtype=torch.float64, device="cuda"))
    norm = spax.Norm(torch.ones(64, device="cuda"))
    for obj, names in ((c, ("k", "v", "k_scale", "v_scale", "n_pages", "page_size", "dtype")),
                       (rope, ("inv_freq", "interleaved")), (norm, ("weight", "bias", "eps", "kind"))):
        for name in names:
            before = getattr(obj, name)
            with pytest.raises(AttributeError, match="make a new"):
                setattr(obj, name, 3)
            with pytest.raises(AttributeError):
                delattr(obj, name)
            assert getattr(obj, name) is before
        obj.layer = 7  # a caller's own
        assert obj.layer == 7
        del obj.layer
        assert not hasattr(obj, "layer")


def test_replaced_storage_is_seen():
    """Tensors whose storage is replaced after the descriptor was formed: the calls read the new one, or
    refuse it."""
    d = 64
    h = torch.randn(3, d, device="cuda")
    w, b = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
    norm = spax.Norm(w, b, kind=spax.NORM_LAYER)
    got, want = torch.empty_like(h), torch.empty_like(h)
    for new in ((2 * w, w.clone()), (w.to(torch.bfloat16) * 3, b.to(torch.bfloat16) - 1)):
        w.data, b.data = new
        spax.spax_residual_norm(h, None, None, got, pre=norm)
        spax.spax_residual_norm(h, None, None, want, pre=spax.Norm(*new, kind=spax.NORM_LAYER))
        assert torch.equal(got, want)
    for bad, err in ((torch.ones(d), TypeError), (torch.ones(32, dtype=torch.bfloat16, device="cuda"), ValueError)):
        w.data = bad
        with pytest.raises(err):
            spax.spax_residual_norm(h, None, None, got, pre=norm)

    case = Case([40, 7], 4, 2, 64)
    first = case.run()
    k, v = case.c.k, case.c.v
    f = torch.rand(32, dtype=torch.float64, device="cuda")
    rope = spax.Rope(f)
    k.data, v.data, f.data = k.flip(-1).contiguous(), v.clone() * 2, f * 0.5
    out, lse = case.run()
    assert not torch.equal(out, first[0])
    case.check(out, lse)
    new, st = torch.randn(2, 2, 64, device="cuda"), case.status
    case.table[:, -1] = torch.tensor([case.c.n_pages - 1, case.c.n_pages - 2], device="cuda")
    pos = torch.full_like(case.lens, case.table.shape[1] * 16 - 1)
    spax.spax_kv_append(case.c, None, new, new, pos, case.table, st, rope=rope)
    at = case.table[:, -1].long()
    assert torch.equal(v[at, 15], new.to(torch.bfloat16)) and st.item() == 0
    want = layer.rotate(new.cpu().numpy(), pos.tolist(), f.cpu().numpy(), False)
    size = new.abs().double().cpu().numpy()
    turned = (size + size[..., list(range(32, 64)) + list(range(32))]) * 2.0 ** -21  # as in test_kv_append_gpu
    tol = turned + (abs(want) + turned) * 2.0 ** -8  # and half a step of bf16
    assert (abs(k[at, 15].double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 40, -2 ** 31, -2 ** 32 + 1])
def test_windows_past_32_bits_are_refused(window):
    """A structure's field keeps the low 32 bits of what it is given."""
    case = Case([20, 30], 4, 2, 64)
    with pytest.raises((ValueError, spax.SpaxError)):
        case.run(window)
    assert case.status.item() == 0


@pytest.mark.parametrize("n,d", [(1, 4096), (3, 515), (200, 1028), (2, 16384)])
def test_a_residual_sum_with_the_next_norm_is_the_two_calls(n, d):
    """A layer's last sum and the next layer's first norm in one call give the bits of two."""
    h, y = (torch.randn(n, d, device="cuda") for _ in range(2))
    for kind in (spax.NORM_RMS, spax.NORM_LAYER):
        norm = spax.Norm(torch.rand(d, device="cuda"), kind=kind)
        r, x, r2, x2 = (torch.empty_like(h) for _ in range(4))
        spax.spax_residual_norm(h, y, r, x, pre=norm)
        spax.spax_residual_norm(h, y, r2, None)
        spax.spax_residual_norm(r2, None, None, x2, pre=norm)
        assert torch.equal(r, r2) and torch.equal(x, x2)
