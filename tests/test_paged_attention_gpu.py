"""spax_paged_attention against the fp64 oracle.

Tolerances, with u = 2^-24 and A the largest sum over the entries of |scale q_i k_i| among the
positions a head sees. A score is a sum of D products, exact or off by u each (a query entry in two
fp16 parts), taken in at most D / 2 steps of error 2 u each: it is off by (D + 1) u A, within dS =
2 D u A (+ 16 u softcap for the capped form, whose tanh and two products are each within a few ulp).
A probability's exponent carries the error of the score, of the maximum (also dS) and the rounding of
its argument (|s - m| <= 2 A, 4 u of it): relative to itself it is off by x = 2 dS + 8 u A + 8 u.
Numerator and denominator are sums of at most L terms in at most
L / 64 + 160 serial steps (tiles and joins), each 2 u. So

    |out - exact| <= (2 x + 4 (L / 64 + 160) u) * sum_j p_j |v_j|,
    |lse - exact| <= x + 2 (L / 64 + 160) u + 2 u |lse|.

Every element of the cache that no position of a test reaches is NaN.
"""
import math

import numpy as np
import pytest
import torch

from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

if cuda_ok():
    from oracle import layer
    from tiered_weight_gemv_b200 import spax

U = 2.0 ** -24


class Case:
    def __init__(self, lens, H, K, D, dtype=0, page=16, hnd=False, seed=0, sharp=1.0, max_pages=None):
        torch.manual_seed(seed)
        self.lens_l, self.H, self.K, self.D = lens, H, K, D
        n = len(lens)
        need = [-(-x // page) for x in lens]
        mp = max(1, max(need, default=1)) if max_pages is None else max_pages
        n_pages = sum(need) + 3
        ks, vs = (0.03, 0.25) if dtype else (1.0, 1.0)
        self.c = c = spax.alloc_kv_cache(n_pages, page, K, D, dtype, hnd, ks, vs)
        for t in (c.k, c.v):  # NaN everywhere
            (t.view(torch.uint8) if dtype else t.view(torch.int16)).fill_(0x7F if dtype else 0x7FC0)
        perm = torch.randperm(n_pages)
        table = torch.full((n, mp), -7, dtype=torch.int32)  # entries past a sequence: never read
        at = 0
        for i, x in enumerate(lens):
            table[i, : need[i]] = perm[at: at + need[i]].int()
            at += need[i]
            t = torch.arange(x)
            pg, rw = table[i].long()[t // page].cuda(), (t % page).cuda()
            for pool in (c.k, c.v):
                val = torch.randn(x, K, D, device="cuda").to(pool.dtype)
                if dtype:
                    pool.view(torch.uint8)[pg, rw] = val.view(torch.uint8)
                else:
                    pool[pg, rw] = val
        self.table = table.cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # a projection's row: q with k and v behind it, so the rows are strided
        self.q = (torch.randn(n, (H + 2 * K), D, device="cuda") * (sharp / ks))[:, :H]
        self.scale = 1 / math.sqrt(D)
        self.ws = spax.alloc_attention_workspace(c, H)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, window=0, softcap=0.0, **kw):
        out = torch.full((len(self.lens_l), self.H, self.D), float("nan"), device="cuda")
        lse = torch.full(out.shape[:2], float("nan"), device="cuda")
        spax.spax_paged_attention(self.c, self.q, self.table, self.lens, out, self.status, self.ws,
                                  scale=self.scale, window=window, softcap=softcap, lse=lse, **kw)
        return out, lse

    def check(self, out, lse, window=0, softcap=0.0):
        keys = self.c.k.float().double().cpu().numpy() * np.float64(np.float32(self.c.k_scale))
        vals = self.c.v.float().double().cpu().numpy() * np.float64(np.float32(self.c.v_scale))
        scale = np.float64(np.float32(self.scale))
        o, ls, A, spread = layer.attention(self.q.double().cpu().numpy(), keys, vals,
                                           self.table.cpu().numpy(), self.lens.cpu().numpy(), scale,
                                           window, softcap)
        L = np.array([min(x, window) if window else x for x in self.lens_l]).clip(0)[:, None]
        dS = 2 * self.D * U * A + 16 * U * softcap
        x = 2 * dS + 8 * U * A + 8 * U
        steps = (L / 64 + 160) * U
        tol = (2 * x + 4 * steps)[:, :, None] * spread
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.all(np.abs(got - o) <= tol), np.max(np.abs(got - o) / np.maximum(tol, 1e-300))
        empty = np.isneginf(ls)
        ls = np.where(empty, 0, ls)
        assert np.array_equal(np.isneginf(gl), empty)
        assert np.all(np.abs(np.where(empty, 0, gl) - ls)[~empty] <= (x + 2 * steps + 2 * U * np.abs(ls))[~empty])
        assert np.all(got[empty] == 0)


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 511, 700]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("H,K,D,page,hnd", [
    (4, 4, 128, 16, False), (8, 2, 128, 16, False), (8, 1, 128, 64, True), (16, 1, 128, 1, False),
    (5, 1, 64, 21, False), (6, 2, 80, 32, True), (14, 2, 96, 8, False), (3, 3, 192, 16, True),
    (16, 2, 256, 24, False), (32, 1, 64, 256, True), (9, 1, 256, 5, False), (20, 1, 16, 16, False),
    (34, 2, 128, 48, False), (2, 1, 112, 128, True), (6, 2, 48, 7, False), (4, 2, 176, 3, True)])
def test_against_the_oracle(dtype, H, K, D, page, hnd):
    case = Case(LENS, H, K, D, dtype, page, hnd, seed=H * D + page)
    out, lse = case.run()
    assert case.status.item() == 0
    case.check(out, lse)


@pytest.mark.parametrize("lens", [[1], [16], [517], [3000], [20011], [0], [0, 0, 0]])
@pytest.mark.parametrize("H,K,D,dtype", [(8, 8, 128, 0), (4, 1, 128, 1), (8, 1, 64, 0), (16, 1, 256, 0)])
def test_one_sequence_split_over_its_length(lens, H, K, D, dtype):
    case = Case(lens, H, K, D, dtype, 16, seed=lens[0])
    out, lse = case.run()
    assert case.status.item() == 0
    case.check(out, lse)
    again = case.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("H,K,D,dtype", [(8, 1, 80, 0), (8, 1, 112, 1), (5, 1, 48, 0), (16, 2, 96, 0),
                                         (6, 1, 176, 1), (12, 1, 16, 0), (16, 1, 112, 1)])
def test_heads_that_no_warp_holds_alone_are_joined(H, K, D, dtype):
    """Rows of many parts, joined in one or two steps by threads of several warps to a head, often enough
    that their order differs."""
    for n in (1100, 4000, 17 * 64, 60 * 64):
        case = Case([n, 5, n - 1], H, K, D, dtype, 32, seed=n)
        first = case.run()
        case.check(*first)
        for _ in range(20):
            again = case.run()
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 699, 700, 100000])
@pytest.mark.parametrize("dtype,softcap", [(0, 0.0), (1, 5.0)])
def test_windows_and_capped_scores(window, dtype, softcap):
    case = Case(LENS, 6, 2, 128, dtype, 21, seed=window, sharp=3.0)
    out, lse = case.run(window, softcap)
    assert case.status.item() == 0
    case.check(out, lse, window, softcap)


def test_many_sequences():
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    case = Case(lens, 4, 2, 64, 0, 16, seed=5)
    out, lse = case.run()
    case.check(out, lse)
    lens = [0] * 300 + [900] + [0] * 400 + [3] * 3 + [0] * 20
    case = Case(lens, 2, 2, 64, 1, 16, seed=6)
    out, lse = case.run()
    case.check(out, lse)
    assert case.status.item() == 0


@pytest.mark.parametrize("n", [31, 32, 33, 127, 128, 129])
@pytest.mark.parametrize("dtype,window", [(0, 0), (1, 90)])
def test_numbers_of_sequences(n, dtype, window):
    """Around the numbers at which the dealing of work changes its form, with empty and long rows."""
    lens = [(i * 37) % 211 if i % 5 else 0 for i in range(n)]
    lens[n // 2], lens[-1] = 1500, 0
    case = Case(lens, 8, 2, 64, dtype, 16, seed=n)
    out, lse = case.run(window)
    assert case.status.item() == 0
    case.check(out, lse, window)


@pytest.mark.parametrize("H,K,D", [(128, 1, 64), (96, 2, 128), (71, 1, 64), (40, 1, 256)])
def test_many_query_heads_to_a_key_head(H, K, D):
    for dtype in (0, 1):
        case = Case([700, 0, 33], H, K, D, dtype, 16, seed=H)
        out, lse = case.run()
        case.check(out, lse)


def test_keys_and_values_of_one_tensor():
    both = torch.randn(6, 2, 16, 2, 64, device="cuda").to(torch.bfloat16)
    case = Case([70, 20], 4, 2, 64)
    case.table = torch.tensor([[5, 0, 2, 3, 1], [4, 1, 0, 0, 0]], dtype=torch.int32, device="cuda")
    case.c = spax.KvCache(both[:, 0], both[:, 1])
    case.check(*case.run())


def test_large_scores_and_one_hot_rows():
    """Scores of some hundreds: the running maximum moves far, most probabilities vanish."""
    for dtype in (0, 1):
        case = Case([1, 40, 333, 2500], 8, 2, 128, dtype, 16, seed=9, sharp=100.0)
        out, lse = case.run()
        assert torch.isfinite(out).all()
        case.check(out, lse)


@pytest.mark.parametrize("dtype", [0, 1])
def test_queries_and_probabilities_keep_32_bits(dtype):
    """A score that is what remains of cancelling products, and an output that is what remains of
    cancelling values: both vanish if a query or a probability is held in fewer bits. Beside bf16 the
    parts hold a query exactly; beside an 8-bit cache two fp16 parts leave at most 2^-12 * 2^-12 of an
    entry, so the two entries of size 1 + 2^-21 and 1 (in steps of 1 / k_scale) put the score off by at
    most (2 + 2^-21) * 2^-24, where the remainder is 2^-21."""
    D = 64
    case = Case([1, 2], 1, 1, D, dtype, 16)
    raw = (lambda t: t.view(torch.uint8)) if dtype else (lambda t: t)  # noqa: E731
    one = torch.ones(1, D, device="cuda").to(case.c.k.dtype)
    for i, n in enumerate((1, 2)):
        pg = int(case.table[i, 0])
        raw(case.c.k)[pg, :n] = raw(one)
    raw(case.c.v)[int(case.table[1, 0]), 0] = raw(one)
    raw(case.c.v)[int(case.table[1, 0]), 1] = raw((-one.float()).to(one.dtype))
    big = float(case.c.k_scale)
    q = torch.zeros(2, 1, D, device="cuda")
    q[:, 0, 0], q[:, 0, 1] = (1 + 2.0 ** -21) / big, -1 / big
    case.q, case.scale = q, 1.0
    out, lse = case.run()
    exact = float(q[0, 0].double().sum()) * np.float64(np.float32(big))
    off = (2 + 2.0 ** -21) * 2.0 ** -24 + 4 * U * abs(exact) if dtype else 2.0 ** -3 * abs(exact)
    assert abs(lse[0, 0].item() - exact) <= off
    # one position's score lies 2^-18 over the other's: out = tanh(2^-19), the difference of two
    # probabilities, each of which is good to u of itself
    d = 2.0 ** -18
    q[1, 0].zero_()
    q[1, 0, 2] = d / big
    zero = torch.zeros(1, device="cuda").to(case.c.k.dtype)
    raw(case.c.k)[int(case.table[1, 0]), 1, 0, 2] = raw(zero)[0]
    out, lse = case.run()
    want = math.tanh(d / 2) * case.c.v_scale
    assert torch.all((out[1, 0].double() - want).abs() <= 4 * U * case.c.v_scale)


def test_bad_lengths_and_pages_are_reported_and_left_out():
    for dtype in (0, 1):
        case = Case([40, 40, 40, 40, 64], 4, 2, 64, dtype, 16, seed=3, max_pages=4)
        case.lens[1], case.lens[2] = -1, 65  # 65 is one past the table
        case.table[3, 1], case.table[4, 0] = case.c.n_pages, -1
        case.lens_l = [40, 0, 0, 40, 64]
        out, lse = case.run()
        assert case.status.item() == spax.ERR_INDEX
        case.check(out, lse)
        case.table[3, :] = -5  # no page at all: an empty row
        case.lens[1] = case.lens[2] = 0
        case.status.zero_()
        out, lse = case.run()
        assert case.status.item() == spax.ERR_INDEX
        case.check(out, lse)
        assert torch.all(out[3] == 0)


def test_non_finite_values_stay_in_their_rows():
    case = Case([50, 70, 90], 8, 2, 128, 0, 16, seed=8)
    ref = case.run()
    case.q[1, 3, 5] = float("nan")
    out, lse = case.run()
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3])
    out[1, 3], lse[1, 3] = ref[0][1, 3], ref[1][1, 3]
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    case.q[1, 3, 5] = 0.5
    ref = case.run()
    page = int(case.table[2, 1])
    case.c.v[page, 3, 1, 17] = float("inf")  # a seen value: its entry alone, for its four heads
    out, lse = case.run()
    assert torch.isposinf(out[2, 4:, 17]).all()
    out[2, 4:, 17] = ref[0][2, 4:, 17]
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("H,K,D", [(32, 2, 128), (4, 2, 64), (8, 2, 256)])
@pytest.mark.parametrize("entry", [float("inf"), -float("inf")])
def test_an_infinite_query_is_a_head_of_nan(entry, H, K, D, dtype):
    """Its head alone, and nothing where the sequence is empty."""
    case = Case([1, 300, 0], H, K, D, dtype, 16, seed=D + H)
    case.q[:, 2, 7] = entry
    out, lse = case.run()
    assert torch.isnan(out[:2, 2]).all() and torch.isnan(lse[:2, 2]).all()
    assert torch.all(out[2] == 0) and torch.isneginf(lse[2]).all()
    case.q[:, 2, 7] = 0.0  # the oracle's other heads do not read it
    other = case.run()
    out[:, 2], lse[:, 2] = other[0][:, 2], other[1][:, 2]
    case.check(out, lse)


@pytest.mark.parametrize("H,K,D", [(32, 2, 128), (4, 2, 64), (26, 2, 64), (8, 2, 256), (8, 2, 80)])
def test_an_infinite_value_is_an_infinite_entry(H, K, D):
    """In every shape: +-inf at a seen position is +-inf at its entry for the heads that see it, and
    changes nothing else; a key entry of -inf under positive queries leaves its position out."""
    case = Case([50, 300], H, K, D, 0, 16, seed=D + H)
    case.q = case.q.abs()
    ref = case.run()
    G = H // K
    page = int(case.table[1, 2])
    case.c.v[page, 5, 1, D - 1] = float("inf")
    case.c.v[page, 6, 0, 0] = -float("inf")
    out, lse = case.run()
    assert torch.isposinf(out[1, G:, D - 1]).all() and torch.isneginf(out[1, :G, 0]).all()
    out[1, G:, D - 1], out[1, :G, 0] = ref[0][1, G:, D - 1], ref[0][1, :G, 0]
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    case.c.k[page, 5, 1, 3] = case.c.k[page, 6, 0, 3] = -float("inf")
    case.c.v[page, 5, 1, D - 1] = case.c.v[page, 6, 0, 0] = 0.0
    out, lse = case.run()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    case.check(out, lse)


def test_scores_of_minus_infinity():
    """A key entry of -inf under a positive query entry: its score is -inf, its probability 0; a
    sequence with no other position gives 0 and -inf."""
    case = Case([1, 40], 2, 2, 64, 0, 16, seed=8)
    case.q[:, :, 0] = 1.0
    page = int(case.table[1, 0])
    case.c.k[int(case.table[0, 0]), 0, :, 0] = -float("inf")
    case.c.k[page, :16, :, 0] = -float("inf")  # the whole first tile
    out, lse = case.run()
    assert torch.all(out[0] == 0) and torch.isneginf(lse[0]).all()
    case.c.k[page, :16] = 0
    case.table[1, 0], first = case.c.n_pages, int(case.table[1, 0])  # the same rows, left out
    want = case.run()
    assert first == page
    assert torch.allclose(out[1], want[0][1], rtol=1e-5, atol=1e-6)
    assert torch.allclose(lse[1], want[1][1], rtol=1e-6)


def test_workspace_is_left_ready_and_calls_chain():
    """Calls of unlike shapes in a row on one workspace, eager and captured, without a wait between."""
    cases = [Case([n], 8, 1, 128, 0, 16, seed=n) for n in (9000, 100, 6000)]
    ws = cases[0].ws
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    for c in cases:
        c.ws = ws
    for _ in range(3):
        got = [c.run() for c in cases]
        for (a, b), (o, l) in zip(want, got):
            assert torch.equal(a, o) and torch.equal(b, l)
    outs = [(torch.zeros_like(a), torch.zeros_like(b)) for a, b in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c, (o, l) in zip(cases, outs):
            spax.spax_paged_attention(c.c, c.q, c.table, c.lens, o, c.status, ws, scale=c.scale, lse=l)
    for _ in range(2):
        for o, l in outs:
            o.zero_(), l.zero_()
        g.replay()
        torch.cuda.synchronize()
        for (a, b), (o, l) in zip(want, outs):
            assert torch.equal(a, o) and torch.equal(b, l)
    cases[0].lens.fill_(4321)  # a replay reads the lengths of its time
    cases[0].lens_l = [4321]
    g.replay()
    cases[0].check(*outs[0])


def test_another_stream():
    case = Case([3000, 5], 8, 2, 128, 0, 16)
    want = case.run()
    side = torch.cuda.Stream()
    got = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    side.wait_stream(torch.cuda.current_stream())
    spax.spax_paged_attention(case.c, case.q, case.table, case.lens, got[0], case.status, case.ws,
                              scale=case.scale, lse=got[1], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_calls_at_once():
    """Two streams, a workspace each, neither waiting for the other."""
    cases = [Case([5000, 1, 0, 900], 8, 2, 128, i, 16, seed=i) for i in (0, 1)]
    want = [c.run() for c in cases]
    got = [tuple(torch.zeros_like(t) for t in w) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(30):
        for c, s, (out, lse) in zip(cases, streams, got):
            spax.spax_paged_attention(c.c, c.q, c.table, c.lens, out, c.status, c.ws,
                                      scale=c.scale, lse=lse, stream=s)
    torch.cuda.synchronize()
    for (a, b), (o, l) in zip(want, got):
        assert torch.equal(a, o) and torch.equal(b, l)


def test_offsets_past_32_bits():
    """Keys and values in one allocation whose pages lie 2^30 elements apart."""
    big = torch.zeros((1 << 31) + (1 << 14), dtype=torch.bfloat16, device="cuda")
    shape, stride = (3, 16, 2, 64), (1 << 30, 128, 64, 1)
    k = big.as_strided(shape, stride)
    v = big.as_strided(shape, stride, 1 << 12)
    small = Case([45], 4, 2, 64, 0, 16)
    small.table[0] = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    keys, vals = torch.randn(2, 3, 16, 2, 64, device="cuda").to(torch.bfloat16)
    k.copy_(keys), v.copy_(vals)
    small.c = spax.KvCache(k, v)
    out, lse = small.run()
    small.check(out, lse)
    # and the append's offsets
    small.lens.fill_(46)
    small.lens_l = [46]
    new = torch.randn(2, 1, 2, 64, device="cuda")
    st = small.status
    spax.spax_kv_append(small.c, None, new[0], new[1], small.lens - 1, small.table, st)
    assert torch.equal(k[1, 13], new[0, 0].to(torch.bfloat16)) and torch.equal(v[1, 13], new[1, 0].to(torch.bfloat16))
    out, lse = small.run()
    small.check(out, lse)
    # a prompt's last page at the far end
    spax.spax_kv_append(small.c, None, new[0], new[1], torch.full_like(small.lens, 2), small.table, st)
    assert torch.equal(k[2, 2], new[0, 0].to(torch.bfloat16)) and st.item() == 0


def test_a_contiguous_cache_is_one_page_each():
    case = Case([300, 77], 8, 2, 128, 0, 320, hnd=True)
    out, lse = case.run()
    case.check(out, lse)


def test_the_binding_refuses():
    case = Case([20, 30], 4, 2, 64)
    out, _ = case.run()
    ok = dict(cache=case.c, q=case.q, page_table=case.table, seq_lens=case.lens, out=out,
              status=case.status, ws=case.ws, scale=1.0)
    for change, err in [(dict(q=case.q.double()), TypeError), (dict(seq_lens=case.lens.long()), TypeError),
                        (dict(seq_lens=case.lens[:1]), ValueError), (dict(out=out[:1]), ValueError),
                        (dict(page_table=case.table[:1]), ValueError), (dict(page_table=case.table.t()), ValueError),
                        (dict(lse=out[0]), ValueError), (dict(q=case.q.cpu()), TypeError),
                        (dict(ws=case.ws[:8]), spax.SpaxError), (dict(scale=math.nan), spax.SpaxError),
                        (dict(window=-1), spax.SpaxError), (dict(ws=case.ws.float()), TypeError),
                        (dict(out=case.q), ValueError)]:
        with pytest.raises(err):
            spax.spax_paged_attention(**{**ok, **change})
