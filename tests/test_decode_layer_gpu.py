"""A decoder layer's step with the library's calls in a row, as a decoder runs it: norm, qkv, append,
attention, o, norm, gate/up, down, for some tokens, every input of a call the output of the one
before; against the fp64 oracle of each step on the inputs that the step had on the GPU, and against a
captured graph of the same calls. The tolerances of each step are those of its own tests: the norms
and the attention by their bounds, the tiered products by rel L2 2e-3.
"""
import math

import numpy as np
import pytest
import torch

from conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

if cuda_ok():
    import oracle
    from oracle import layer
    from tiered_weight_gemv_b200 import spax, synth
    from gpu_helpers import bf16_bits, check_y
    from test_paged_attention_gpu import U
    from test_residual_norm_gpu import check as check_norm

H, K, D, FF = 8, 2, 64, 1152
WIDTH = H * D
PAGE, PAGES = 16, 6


class Site:
    def __init__(self, d_out, d_in, tensor):
        W = synth.weight(d_out, d_in, 11, tensor, device="cuda")
        self.pm = spax.alloc_packed(d_out, d_in, spax.FULL_BF16)
        spax.spax_pack_weights(W, spax.FULL_BF16, self.pm)
        self.pools = oracle.pack(bf16_bits(W), 0)
        self.ws = spax.alloc_workspace(spax.OP_TIERED_GEMV, d_out, d_in)
        k = d_in * 3 // 10
        self.k, self.prm = k, spax.mask_params(spax.MASK_TOPK, k_full=k, k_approx=k)
        self.y = torch.zeros(d_out, device="cuda")

    def check(self, x):
        x = x.cpu().numpy()
        _, tier, _, _, _ = oracle.tiers(x, oracle.MODE_TOPK, k_full=self.k, k_approx=self.k)
        want = oracle.tiered_gemv(*self.pools, 0, self.pm.d_out, self.pm.d_in, x, tier)
        check_y(self.y.cpu().numpy(), want)


class Layer:
    def __init__(self, dtype):
        torch.manual_seed(dtype)
        self.qkv, self.o = Site((H + 2 * K) * D, WIDTH, 1), Site(WIDTH, WIDTH, 2)
        self.gu, self.down = Site(2 * FF, WIDTH, 3), Site(WIDTH, FF, 4)
        scale = (0.05, 0.05) if dtype else (1.0, 1.0)
        self.c = spax.alloc_kv_cache(PAGES + 1, PAGE, K, D, dtype, k_scale=scale[0], v_scale=scale[1])
        self.table = torch.tensor([[3, 1, 6, 0, 2, 5]], dtype=torch.int32, device="cuda")
        f = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
        self.rope = spax.Rope(f)
        self.n1, self.n2 = (spax.Norm((1 + 0.1 * torch.randn(WIDTH, device="cuda")).to(torch.bfloat16))
                            for _ in range(2))
        self.ws = spax.alloc_attention_workspace(self.c, H)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.pos = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.len = torch.ones(1, dtype=torch.int32, device="cuda")
        z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        self.h, self.r, self.r2, self.x1, self.x2 = (z(1, WIDTH) for _ in range(5))
        self.a, self.ff, self.lse = z(1, H, D), z(FF), z(1, H)
        self.q_rot = z(1, H, D)

    def step(self):
        st = self.status
        row = self.qkv.y.view(1, -1)
        q, k, v = (t.unflatten(1, (-1, D)) for t in row.split([WIDTH, K * D, K * D], 1))
        spax.spax_residual_norm(self.h, None, None, self.x1, pre=self.n1)
        spax.spax_masked_gemv(self.qkv.pm, self.x1[0], self.qkv.prm, self.qkv.y, st, self.qkv.ws)
        spax.spax_kv_append(self.c, q, k, v, self.pos, self.table, st, rope=self.rope, q_out=self.q_rot)
        spax.spax_paged_attention(self.c, self.q_rot, self.table, self.len, self.a, st, self.ws,
                                  scale=1 / math.sqrt(D), lse=self.lse)
        spax.spax_masked_gemv(self.o.pm, self.a.view(-1), self.o.prm, self.o.y, st, self.o.ws)
        spax.spax_residual_norm(self.h, self.o.y.view(1, -1), self.r, self.x2, pre=self.n2)
        spax.spax_masked_gemv(self.gu.pm, self.x2[0], self.gu.prm, self.gu.y, st, self.gu.ws)
        spax.spax_masked_gemv_swiglu(self.down.pm, self.gu.y, self.down.prm, self.down.y, st,
                                     self.down.ws, x_out=self.ff)
        spax.spax_residual_norm(self.r, self.down.y.view(1, -1), self.r2, None)

    def check(self):
        check_norm(self.h, None, self.n1, None, None, 1.0, 1.0, None, self.x1)
        self.qkv.check(self.x1[0])
        pos, n = int(self.pos), int(self.len)
        q = self.qkv.y[:WIDTH].view(1, H, D)
        f = self.rope.inv_freq.cpu().numpy()
        want = layer.rotate(q.cpu().numpy(), [pos], f, False)
        x = np.abs(q.double().cpu().numpy())
        assert np.all(np.abs(self.q_rot.double().cpu().numpy() - want) <= (x + np.roll(x, D // 2, -1)) * 2.0 ** -21)
        pg, rw = layer.place(self.table.cpu().numpy(), PAGES + 1, PAGE, 0, pos)
        v = self.qkv.y[WIDTH + K * D:].view(K, D)
        v = v if self.c.dtype == 0 else (v / self.c.v_scale).clamp(-448, 448)
        assert torch.equal(self.c.v[pg, rw].float(), v.to(self.c.v.dtype).float())
        keys, vals = (t.float().double().cpu().numpy() * np.float64(np.float32(s))
                      for t, s in ((self.c.k, self.c.k_scale), (self.c.v, self.c.v_scale)))
        o, ls, A, spread = layer.attention(self.q_rot.double().cpu().numpy(), keys, vals,
                                           self.table.cpu().numpy(), [n], np.float64(np.float32(1 / math.sqrt(D))))
        e = 2 * (4 * D * U * A + 8 * U * A + 8 * U) + 4 * (n / 64 + 160) * U
        assert np.all(np.abs(self.a.double().cpu().numpy() - o) <= e[:, :, None] * spread)
        assert np.all(np.abs(self.lse.double().cpu().numpy() - ls) <= e + 2 * U * np.abs(ls))
        self.o.check(self.a.view(-1))
        check_norm(self.h, self.o.y.view(1, -1), self.n2, None, None, 1.0, 1.0, self.r, self.x2)
        self.gu.check(self.x2[0])
        self.down.check(self.ff)
        check_norm(self.r, self.down.y.view(1, -1), None, None, None, 1.0, 1.0, self.r2, None)
        assert self.status.item() == 0


@pytest.mark.parametrize("dtype", [0, 1])
def test_a_layer_decodes(dtype, oracle_lib):
    lay = Layer(dtype)
    tokens = torch.randn(PAGE * 3 + 5, WIDTH, device="cuda")
    eager = []
    for t, x in enumerate(tokens):
        lay.h.copy_(x[None])
        lay.pos.fill_(t)
        lay.len.fill_(t + 1)
        lay.step()
        if t in (0, 1, 15, 16, 17, 40, len(tokens) - 1):
            lay.check()
        eager.append(lay.r2.clone())
    assert lay.status.item() == 0
    # the same tokens through one captured step: position, length and input change, the graph stays
    for pool in (lay.c.k, lay.c.v):
        (pool.view(torch.uint8) if dtype else pool).zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lay.step()
    for t, x in enumerate(tokens):
        lay.h.copy_(x[None])
        lay.pos.fill_(t)
        lay.len.fill_(t + 1)
        g.replay()
        assert torch.equal(lay.r2, eager[t]), t
    assert lay.status.item() == 0


def test_tensors_of_another_device_than_the_current_one_are_refused(monkeypatch, oracle_lib):
    """Where the current device is another (here: is said to be), no call takes the tensors."""
    lay = Layer(0)
    lay.step()
    row = lay.qkv.y.view(1, -1)
    q, k, v = (t.unflatten(1, (-1, D)) for t in row.split([WIDTH, K * D, K * D], 1))
    monkeypatch.setattr(spax, "_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        spax.spax_kv_append(lay.c, q, k, v, lay.pos, lay.table, lay.status, rope=lay.rope)
    with pytest.raises(ValueError, match="current device"):
        spax.spax_paged_attention(lay.c, q, lay.table, lay.len, lay.a, lay.status, lay.ws, scale=1.0)
    with pytest.raises(ValueError, match="current device"):
        spax.spax_residual_norm(lay.h, None, None, lay.x1, pre=lay.n1)
