"""spax_kv_append against the fp64 oracle.

Tolerances: cos and sin each carry sincospif's error (at most 2 ulp, 2 * 2^-23 absolute) and the
fp64 angle's (pos * f * 2^-51 radians, below 2^-31 here); the products and their sum round three
times by 2^-24. A rotated entry is therefore within (|a| + |b|) * 7 * 2^-24 < (|a| + |b|) * 2^-21 of
the pair's exact value. What is then held in fewer bits is off by half a step more: 2^-8 of the
value in bf16; 2^-4 of the value in e4m3, or half its smallest step, 2^-10, below 2^-6.
Entries that are not turned are rounded from their exact value and must match bit for bit.
"""
import numpy as np
import pytest
import torch

from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

if cuda_ok():
    from oracle import layer
    from tiered_weight_gemv_b200 import spax

ROT = 2.0 ** -21


def poison(cache):
    """A recognisable finite pattern in every element, so that a stray write shows."""
    for t in (cache.k, cache.v):
        raw = t.view(torch.uint8) if cache.dtype == spax.KV_E4M3 else t.view(torch.int16)
        raw.copy_(torch.randint(0, 60, raw.shape, device="cuda").to(raw.dtype))


def stored(pool):
    return pool.float().double().cpu().numpy()


def setup(n_tok, H, K, D, dtype, page, hnd, n_seq, max_pages, seed=0, scales=(1.0, 1.0)):
    torch.manual_seed(seed)
    n_pages = n_seq * max_pages + 2
    c = spax.alloc_kv_cache(n_pages, page, K, D, dtype, heads_first=hnd, k_scale=scales[0],
                            v_scale=scales[1])
    poison(c)
    table = torch.randperm(n_pages, device="cuda")[: n_seq * max_pages].reshape(n_seq, max_pages)
    qkv = torch.randn(n_tok, (H + 2 * K) * D, device="cuda") * 3
    cut = qkv.split([H * D, K * D, K * D], 1)
    q, k, v = (t.unflatten(1, (-1, D)) for t in cut)
    return c, table.int().contiguous(), qkv, q, k, v


def check(c, table, q, k, v, q_out, before, q_before, pos, seq, f, inter):
    ks, vs = c.k_scale, c.v_scale
    pos, seq = pos.cpu().numpy(), seq.cpu().numpy()
    tab = table.cpu().numpy()
    places = [layer.place(tab, c.n_pages, c.page_size, s, p) for s, p in zip(seq, pos)]
    live = np.array([p is not None for p in places])
    rot = 2 * len(f)

    def bound(x):  # |a| + |b| of each entry's pair
        x = np.abs(x.double().cpu().numpy())
        out = np.zeros_like(x)
        for i in range(len(f)):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + len(f))
            out[..., a] = out[..., b] = x[..., a] + x[..., b]
        return out * ROT

    safe = np.where(live, pos, 0)
    if q is not None:
        want = layer.rotate(q.cpu().numpy(), safe, f, inter)
        got = q_out.double().cpu().numpy()
        assert np.all(np.abs(got - want)[live] <= bound(q)[live])
        assert np.array_equal(got[live][..., rot:], q.double().cpu().numpy()[live][..., rot:])
        assert np.array_equal(got[~live], q_before.double().cpu().numpy()[~live])
    exp_k, exp_v = before
    got_k, got_v = stored(c.k), stored(c.v)
    rk, bk = layer.rotate(k.cpu().numpy(), safe, f, inter), bound(k)
    half, low = (2.0 ** -8, 0.0) if c.dtype == spax.KV_BF16 else (2.0 ** -4, 2.0 ** -10)
    t = torch.bfloat16 if c.dtype == spax.KV_BF16 else torch.float8_e4m3fn

    def rounded(x, scale):
        x = x if c.dtype == spax.KV_BF16 else (x / scale).clamp(-448, 448)
        return x.to(t).double().cpu().numpy()

    plain_k, plain_v = rounded(k, ks), rounded(v, vs)
    for i, at in enumerate(places):
        if at is None:
            continue
        # the fp32 value is within bk / ks (and one rounding of the division) of the exact one,
        # and its clamp at 448 within as much of the clamped one
        x = rk[i] / ks
        x = x if c.dtype == spax.KV_BF16 else np.clip(x, -448, 448)
        slack = bk[i] / ks + np.abs(x) * 2.0 ** -24
        assert np.all(np.abs(got_k[at] - x)[:, :rot]
                      <= (np.maximum(half * (np.abs(x) + slack), low) + slack)[:, :rot])
        assert np.array_equal(got_k[at][:, rot:], plain_k[i][:, rot:])
        assert np.array_equal(got_v[at], plain_v[i])
        exp_k[at], exp_v[at] = got_k[at], got_v[at]
    assert np.array_equal(got_k, exp_k) and np.array_equal(got_v, exp_v)  # nothing else changed


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("n_seq,per,H,K,D,rot,inter,page,hnd,start", [
    (1, 1, 32, 32, 128, 128, False, 16, False, 0),
    (1, 1, 32, 32, 128, 128, False, 16, False, 1001),
    (9, 1, 64, 8, 128, 128, False, 64, True, 77),
    (3, 37, 12, 3, 80, 32, True, 21, False, 5),
    (2, 65, 4, 4, 64, 64, True, 1, True, 0),
    (2, 33, 7, 1, 256, 256, False, 256, False, 250),
    (4, 5, 6, 2, 96, 48, False, 8, True, 3),
    (2, 3, 5, 5, 16, 8, True, 5, False, 2),
    (2, 70, 16, 2, 192, 0, False, 32, False, 9),
    (1, 3, 3, 3, 112, 112, False, 16, True, 0),
])
def test_against_the_oracle(dtype, n_seq, per, H, K, D, rot, inter, page, hnd, start):
    max_pages = -(-(start + per) // page)
    n = n_seq * per
    scales = (0.02, 0.5) if dtype else (1.0, 1.0)  # 0.02: values up to 12 pass 448 steps
    c, table, qkv, q, k, v = setup(n, H, K, D, dtype, page, hnd, n_seq, max_pages, n, scales)
    f = 10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    rope = spax.Rope(torch.tensor(f, dtype=torch.float64, device="cuda"), inter) if rot else None
    order = torch.randperm(n, device="cuda")
    seq = torch.arange(n_seq, device="cuda").repeat_interleave(per)[order].int()
    pos = (torch.arange(per, device="cuda").repeat(n_seq) + start)[order].int()
    before = stored(c.k), stored(c.v)
    q_out = torch.full_like(q, 7.0).contiguous()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q0 = q_out.clone()
    spax.spax_kv_append(c, q, k, v, pos, table, st, rope=rope, seq=seq, q_out=q_out)
    assert st.item() == 0
    check(c, table, q, k, v, q_out, before, q0, pos, seq, f, inter)
    # in place gives the same rows, and leaves k and v as they were
    kv = k.clone(), v.clone()
    spax.spax_kv_append(c, q, k, v, pos, table, st, rope=rope, seq=seq)
    assert torch.equal(q, q_out) and torch.equal(k, kv[0]) and torch.equal(v, kv[1])


def test_padding_and_bad_places_write_nothing():
    c, table, qkv, q, k, v = setup(9, 4, 2, 64, 0, 8, False, 3, 4)
    table[1, 2] = c.n_pages  # a page past the pool
    table[1, 3] = -1
    before = stored(c.k), stored(c.v)
    f = 10000.0 ** (-np.arange(16) / 16)
    rope = spax.Rope(torch.tensor(f, dtype=torch.float64, device="cuda"))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 1, 2, 0, 1, 1, -1, 3, 2], dtype=torch.int32, device="cuda")
    pos = torch.tensor([31, -1, 0, 32, 16, 31, 4, 4, -2 ** 31], dtype=torch.int32, device="cuda")
    out = torch.full((9, 4, 64), -3.0, device="cuda")
    keep = out.clone()
    spax.spax_kv_append(c, q, k, v, pos, table, st, rope=rope, seq=seq, q_out=out)
    assert st.item() == spax.ERR_INDEX
    check(c, table, q, k, v, out, before, keep, pos, seq, f, False)
    st.zero_()  # padding alone is no error
    spax.spax_kv_append(c, q, k, v, torch.full_like(pos, -1), table, st, rope=rope, seq=seq, q_out=out)
    assert st.item() == 0


def test_without_queries_and_without_sequences():
    c, table, qkv, q, k, v = setup(3, 4, 2, 64, 0, 8, True, 3, 2)
    before = stored(c.k), stored(c.v)
    f = 10000.0 ** (-np.arange(32) / 32)
    rope = spax.Rope(torch.tensor(f, dtype=torch.float64, device="cuda"))
    pos = torch.tensor([3, 15, 8], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    spax.spax_kv_append(c, None, k, v, pos, table, st, rope=rope)
    assert st.item() == 0
    check(c, table, None, k, v, None, before, None, pos, torch.arange(3), f, False)


def test_values_of_the_8_bit_type():
    """Ties, subnormals, saturation, infinities, NaN and zero signs of the stored values."""
    c, table, qkv, q, k, v = setup(1, 1, 1, 16, 1, 4, False, 1, 1)
    x = torch.tensor([0.0, -0.0, 448.0, 449.0, 1e30, -float("inf"), float("inf"), float("nan"),
                      2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 1.0625, 1.1875, -464.0, 0.0175, 3e-4],
                     device="cuda").view(1, 1, 16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    spax.spax_kv_append(c, None, x, x, pos, table, st)
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).float().view(16)
    for pool in (c.k, c.v):
        got = pool[table[0, 0], 0, 0].float()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert torch.equal(got[fine], want[fine])
        assert torch.equal(torch.signbit(got[fine]), torch.signbit(want[fine]))


def test_far_positions_keep_their_angle():
    """At position p = 2^20 + 3 an fp32 angle would be off by up to 2^-4; the bound of this file's
    head (with the fp64 angle's p * 2^-51 = 2^-31) still holds."""
    c, table, qkv, q, k, v = setup(1, 2, 1, 128, 0, 64, False, 1, (1 << 14) + 1)
    p = (1 << 20) + 3
    f = 500000.0 ** (-np.arange(64) / 64)
    rope = spax.Rope(torch.tensor(f, dtype=torch.float64, device="cuda"))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.tensor([p], dtype=torch.int32, device="cuda")
    out = torch.zeros(1, 2, 128, device="cuda")
    spax.spax_kv_append(c, q, k, v, pos, table, st, rope=rope, q_out=out)
    want = layer.rotate(q.cpu().numpy(), [p], f, False)
    x = np.abs(q.double().cpu().numpy())
    b = (x + np.roll(x, 64, -1)) * ROT
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= b)


def test_more_tokens_than_a_grid_dimension_of_65535():
    n, per = 70001, 64
    n_seq = -(-n // per)
    c, table, qkv, q, k, v = setup(n, 2, 1, 16, 0, 16, False, n_seq, 4)
    i = torch.arange(n, device="cuda")
    seq, pos = (i // per).int(), (i % per).int()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(n, 2, 16, device="cuda")
    spax.spax_kv_append(c, q, k, v, pos, table, st, seq=seq, q_out=out)
    at = table[seq.long(), pos.long() // 16].long(), pos.long() % 16
    assert st.item() == 0 and torch.equal(out, q)
    assert torch.equal(c.k[at], k.to(torch.bfloat16)) and torch.equal(c.v[at], v.to(torch.bfloat16))


def test_another_stream_and_a_captured_call():
    c, table, qkv, q, k, v = setup(5, 8, 2, 128, 0, 16, False, 5, 3)
    rope = spax.Rope(torch.rand(64, dtype=torch.float64, device="cuda"))
    pos = torch.full((5,), 7, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(5, 8, 128, device="cuda")
    spax.spax_kv_append(c, q, k, v, pos, table, st, rope=rope, q_out=out)
    want, wk = out.clone(), c.k.clone()
    c.k.zero_(), out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    spax.spax_kv_append(c, q, k, v, pos, table, st, rope=rope, q_out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spax.spax_kv_append(c, q, k, v, pos, table, st, rope=rope, q_out=out)
    pos.add_(20)  # the replay reads the positions of its time
    g.replay()
    again = torch.zeros_like(out)
    spax.spax_kv_append(c, q, k, v, pos, table, st, rope=rope, q_out=again)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and not torch.equal(out, want) and st.item() == 0


def test_the_binding_refuses():
    c, table, qkv, q, k, v = setup(2, 4, 2, 64, 0, 8, False, 2, 2)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ok = dict(cache=c, q=q, k=k, v=v, pos=pos, page_table=table, status=st)
    for change, err in [(dict(q=q.cpu()), TypeError), (dict(k=k.double()), TypeError),
                        (dict(pos=pos.long()), TypeError), (dict(pos=pos[:1]), ValueError),
                        (dict(v=v[:1]), ValueError), (dict(k=k[:, :1]), ValueError),
                        (dict(k=k.transpose(1, 2)), ValueError), (dict(page_table=table[0]), ValueError),
                        (dict(page_table=table[:1]), ValueError), (dict(q=None, q_out=q), ValueError),
                        (dict(q_out=torch.empty(2, 4, 128, device="cuda")), ValueError)]:
        with pytest.raises(err):
            spax.spax_kv_append(**{**ok, **change})
    with pytest.raises(TypeError):
        spax.KvCache(c.k, c.v.half())
    with pytest.raises(ValueError):
        spax.KvCache(c.k, c.v.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(TypeError):
        spax.Rope(torch.rand(8, device="cuda"))
