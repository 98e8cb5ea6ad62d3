"""Decode attention over a 4-bit cache, relative accuracy: an attention sink before thousands of
keys, V scales from 1 down to 1e-3 and far apart between blocks, against fp64 per (row, block)."""
import numpy as np
import pytest
import torch

from decode_step_kv_gb300 import binding as fa

from _cache_ops import dequantize, pack, quantize

pytestmark = pytest.mark.gpu


class Shared:
    """One sequence's rows, which the block tables of all sequences name: many units for few bytes."""

    def __init__(self, hkv, n, k, v, batch):
        """k, v: [Hkv, n, D] fp32, n a multiple of 16."""
        self.n, self.batch, self.hkv = n, batch, hkv
        self.args, self.values = [], []
        for x in (k, v):
            codes, s = quantize(x)
            by = pack(codes)
            self.values.append(torch.from_numpy(dequantize(by, s)).cuda())
            for a in (by, s):
                a = a.reshape(hkv, n // 16, 16, -1)
                self.args.append(torch.from_numpy(np.ascontiguousarray(np.moveaxis(a, 1, 0))).cuda())
        self.table = torch.arange(n // 16, dtype=torch.int32, device="cuda").expand(batch, -1).contiguous()
        self.lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")

    def decode(self, q, scale, acc=None):
        B, tq, Hq, D = q.shape
        out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
        ws = fa.alloc_workspace_int4(B, tq, Hq, self.hkv, D, self.n, weights=acc is not None)
        fa.fa_decode_int4(q, *self.args, self.table, self.lens, Hq, self.hkv, D, scale, None, out,
                          acc=acc, workspace=ws)
        return out

    def rows(self, q, scale):
        """Of up to 50 sequences: fp64 weights [Hkv, tq, G, n] of their rows."""
        B, tq, Hq, D = q.shape
        t = torch.arange(self.n, device="cuda")
        dead = t.view(1, 1, 1, -1) > (self.n - tq + torch.arange(tq, device="cuda")).view(1, tq, 1, 1)
        k = self.values[0]
        for b in range(0, B, -(-B // 50)):
            x = q[b].double().view(tq, self.hkv, Hq // self.hkv, D).transpose(0, 1)
            s = torch.einsum("htgd,hnd->htgn", x, k) * scale
            yield b, torch.softmax(s.masked_fill(dead, -np.inf), dim=-1)


def relative_check(c, q, scale, got):
    """Per row and block of 32 elements, the error's norm.  A key's weight and its product with a
    scale are each rounded to fp16: eps/2 = 2^-11 of it, in either direction and apart from the
    other keys', so the keys' errors add in quadrature; twice the largest such sum (2 x 2 x 2^-11)
    covers how far they can stray from it and the scores' fp32 errors (2^-18 of a weight and
    less).  The result is rounded once more, by 2^-11 or, below 2^-14, by up to 2^-25."""
    B, tq, Hq, D = q.shape
    v = c.values[1]
    blocks = v.view(c.hkv, c.n, D // 32, 32)
    v2 = blocks.square().sum(-1)                                     # [Hkv, n, blocks]
    worst = 0.0
    for b, p in c.rows(q, scale):
        want = torch.einsum("htgn,hnd->htgd", p, v).unflatten(-1, (D // 32, 32))
        g = got[b].double().view(tq, c.hkv, Hq // c.hkv, D).transpose(0, 1).unflatten(-1, (D // 32, 32))
        spread = torch.einsum("htgn,hnj->htgj", p.square(), v2).sqrt()
        bound = (4 * 2.0 ** -11 * spread + 2.0 ** -11 * want.norm(dim=-1) + 32 ** 0.5 * 2.0 ** -25)
        worst = max(worst, float(((g - want).norm(dim=-1) / bound).max()))
    assert worst <= 1, f"{worst:.2f} times the bound"


# columns per KV head and sequences: a worker covers whole units of every kernel
PLANS = [pytest.param(128, 1, 1024, 8192, id="one group"), pytest.param(256, 1, 640, 4096, id="one group, 256"),
         pytest.param(128, 4, 640, 4096, id="two groups"), pytest.param(128, 16, 256, 4096, id="64 columns"),
         pytest.param(256, 16, 160, 4096, id="64 columns, 256"), pytest.param(128, 1, 2, 8192, id="cluster"),
         pytest.param(256, 1, 1, 4096, id="cluster, 256")]


def sink_case(D, tq, batch, n, spread, hkv=2, group=4, seed=0):
    """N(0, 1) scores after a first key that takes half of every row's weight and has a small value;
    V of standard deviation `spread` ([D] or one number)."""
    r = np.random.RandomState(seed)
    scale, a = D ** -0.5, 4.0
    u = r.standard_normal(D)
    u /= np.linalg.norm(u)
    k = r.standard_normal((hkv, n, D))
    k -= (k @ u)[..., None] * u
    k[:, 0] = u * (np.log(n) + 0.5) / (a * scale)
    v = r.standard_normal((hkv, n, D)) * spread
    v[:, 0] *= 0.01
    q = r.standard_normal((batch, tq, hkv * group, D))
    q += (a - q @ u)[..., None] * u
    return (Shared(hkv, n, k.astype(np.float32), v.astype(np.float32), batch),
            torch.from_numpy(q.astype(np.float16)).cuda(), scale)


@pytest.mark.parametrize("sigma", [2e4, 1.0, 0.02, 1e-3, 3e-5])
@pytest.mark.parametrize("D,tq,batch,n", PLANS)
def test_sink_before_many_keys(D, tq, batch, n, sigma):
    c, q, scale = sink_case(D, tq, batch, n, sigma)
    relative_check(c, q, scale, c.decode(q, scale))


@pytest.mark.parametrize("D,tq,batch,n", PLANS)
def test_blocks_of_very_different_scales(D, tq, batch, n):
    """Each block of V is carried by its own power of two: 2^-10 beside 2^6."""
    spread = np.repeat(2.0 ** np.linspace(6, -10, D // 32), 32)
    c, q, scale = sink_case(D, tq, batch, n, spread, seed=1)
    relative_check(c, q, scale, c.decode(q, scale))


@pytest.mark.parametrize("D,tq,batch,n", [(128, 1, 512, 4096), (256, 16, 100, 4096), (256, 1, 1, 4096)])
def test_sink_with_recorded_weights(D, tq, batch, n):
    c, q, scale = sink_case(D, tq, batch, n, 0.005, seed=2)
    acc = torch.zeros(n // 16, 2, 16, device="cuda")
    relative_check(c, q, scale, c.decode(q, scale, acc))
    rows = batch * tq * 4                                # per KV head, each with weights of sum 1
    total = acc.double().sum(dim=(0, 2))
    assert torch.all((total - rows).abs() <= rows * 2.0 ** -12)


@pytest.mark.parametrize("D,tq,batch,n", PLANS)
def test_small_queries_and_large_keys(D, tq, batch, n):
    """Queries mostly below 2^-10, scores of N(0, 3): no query element loses bits."""
    r = np.random.RandomState(3)
    k = r.standard_normal((2, n, D)) * 3 * 2.0 ** 13
    v = r.standard_normal((2, n, D))
    q = torch.from_numpy((r.standard_normal((batch, tq, 8, D)) * 2.0 ** -13).astype(np.float16)).cuda()
    c = Shared(2, n, k.astype(np.float32), v.astype(np.float32), batch)
    relative_check(c, q, D ** -0.5, c.decode(q, D ** -0.5))


@pytest.mark.parametrize("D,tq,batch,n", PLANS)
def test_a_query_of_nan_gives_nan(D, tq, batch, n):
    """Its own row only, in every plan.  (The others may move their references at other keys, so
    each may be off by its two roundings of 2^-11, twice over, on either side.)"""
    r = np.random.RandomState(4)
    k, v = (r.standard_normal((2, n, D)).astype(np.float32) for _ in range(2))
    c = Shared(2, n, k, v, batch)
    q = torch.from_numpy(r.standard_normal((batch, tq, 8, D)).astype(np.float16)).cuda()
    clean = c.decode(q, 0.1)
    q[0, 0, 5, 7] = float("nan")
    got = c.decode(q, 0.1)
    bad = torch.zeros(batch, tq, 8, dtype=torch.bool, device="cuda")
    bad[0, 0, 5] = True
    assert torch.all(torch.isnan(got[bad]))
    diff = (got[~bad].double() - clean[~bad].double()).norm(dim=-1)
    assert torch.all(diff <= 2 * 5 * 2.0 ** -11 * clean[~bad].double().norm(dim=-1))


def test_large_and_small_queries_side_by_side():
    """Each column has its own factor: heads of queries of 2^13 beside heads of 2^-13."""
    r = np.random.RandomState(5)
    D, n = 128, 2048
    mag = np.where(np.arange(8) % 2, 2.0 ** 13, 2.0 ** -13).reshape(1, 1, 8, 1)
    k = r.standard_normal((2, n, D)) * 2.0 ** 13 * 3
    k[1] *= 2.0 ** -26
    v = r.standard_normal((2, n, D))
    c = Shared(2, n, k.astype(np.float32), v.astype(np.float32), 2)
    q = torch.from_numpy((np.clip(r.standard_normal((2, 1, 8, D)), -4, 4) * mag).astype(np.float16)).cuda()
    got = c.decode(q, D ** -0.5)
    for head, keep in ((0, 0), (1, 1)):              # rows whose scores are of N(0, 3)
        sub = Shared(1, n, k[head:head + 1].astype(np.float32), v[head:head + 1].astype(np.float32), 2)
        at = slice(4 * head + keep, 4 * head + 4, 2)
        relative_check(sub, q[:, :, at].contiguous(), D ** -0.5, got[:, :, at].contiguous())
