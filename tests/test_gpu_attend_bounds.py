"""Chunk attention and decode with sinks within the bounds of what they round: a weight that is carried 2^10
above the reference's 1, V of int8 codes where it becomes fp16, and the output.  Long contexts are held by the
norm of a row's error, in which a lost tile, half a tile or a key shows."""
import numpy as np
import pytest
import torch

import decode_step_kv_gb300 as fa
from decode_step_kv_gb300 import binding
from _cache_ops import Layout
from _step_ops import f64

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gpu(*arrays):
    return [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in arrays]


def rows(q, at, k, v, scale, window, sink, hkv):
    """fp64: out, sum p |v| and sqrt(sum p^2 |v|^2), by row: q [n, Hq, D], k and v [Hkv, L, D]."""
    q, k, v = (torch.from_numpy(np.ascontiguousarray(x)).double().cuda() for x in (q, k, v))
    n, hq, d = q.shape
    t = torch.arange(k.shape[1], device="cuda")
    at = torch.as_tensor(np.asarray(at), device="cuda").view(-1, 1)
    live = t <= at
    if window:
        live &= (t > at - window) | (t < sink)
    k, v = (torch.nan_to_num(x) for x in (k, v))
    s = torch.einsum("nhgd,htd->nhgt", q.view(n, hkv, hq // hkv, d), k) * scale
    p = torch.softmax(s.masked_fill(~live[:, None, None], -np.inf), dim=-1)
    got = (torch.einsum("nhgt,htd->nhgd", p, v), torch.einsum("nhgt,htd->nhgd", p, v.abs()),
           torch.einsum("nhgt,ht->nhg", p.square(), v.square().sum(-1)).sqrt())
    return [x.reshape(n, hq, -1).cpu().numpy() for x in got]


def check(got, want, size, spread, keys, vmax, roundings):
    """`roundings` of each weight and value: 2^-11 each, and one of the output; a weight below 2^-24 of the
    largest, which a row's reference may lie 2^5 beneath, is a subnormal, off by 2^-25 of 2^-10 of that.
    Scores in 32 bits are off by under 2^-17.  By element that is the worst case.  By row the keys'
    errors are apart from one another and add in quadrature: a rounding's mean square is a third of its
    most, so twice the root of the sum of the most is beyond what they reach."""
    half = 2.0 ** -11
    tol = ((roundings + 1) * half + 2.0 ** -15) * size + keys * 2.0 ** -35 * vmax + 2.0 ** -25
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), (err / tol).max()
    norm = np.linalg.norm(err, axis=-1, keepdims=True)
    most = (2 * roundings * half * spread + half * np.linalg.norm(want, axis=-1, keepdims=True) +
            2.0 ** -16 * spread + np.sqrt(want.shape[-1]) * 2.0 ** -25)
    assert (norm <= most).all(), (norm / most).max()


def cache(lay, D, codes, rng, spread=1.0):
    """K, V, V's scales and V's values, in the layout's rows."""
    k = rng.randn(*lay.rows, D).astype(np.float16)
    v = (rng.randn(*lay.rows, D) * spread).astype(np.float16).astype(np.float64)
    if not codes:
        return k, v.astype(np.float16), None, v
    blk = v.reshape(*lay.rows, -1, 32)
    s = (np.abs(blk).max(-1) / 127).astype(np.float16)
    c = np.clip(np.rint(blk / s[..., None].astype(np.float64)), -127, 127)
    return k, c.reshape(v.shape).astype(np.int8), s, (c * s[..., None].astype(np.float64)).reshape(v.shape)


def prefill(lay, lens, new, hq, D, codes, window=None, sink=0, seed=0):
    rng = np.random.RandomState(seed)
    k, v, s, val = cache(lay, D, codes, rng)
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = rng.randn(starts[-1], hq, D).astype(np.float16)
    out = torch.full(q.shape, 9.0, dtype=torch.float16, device="cuda")
    qd, kd, vd, sd = gpu(q, k, v, s)
    fa.fa_prefill(qd, kd, vd, sd, lay.table_gpu(), ints(starts), ints(lens), hq, lay.hkv, D, D ** -0.5,
                  ints(window) if window else None, out, n_sink=sink,
                  workspace=fa.alloc_workspace_prefill(lay.batch, starts[-1], hq, lay.hkv, D, lay.capacity))
    assert binding.fa_decode_device_status() == 0
    got = f64(out)
    for b, n in enumerate(new):
        if not n:
            continue
        r = slice(starts[b], starts[b] + n)
        m = rows(q[r], np.arange(lens[b] - n, lens[b]), lay.dense(k, b)[:, :lens[b]], lay.dense(val, b)[:, :lens[b]],
                 D ** -0.5, window[b] if window else 0, sink, lay.hkv)
        check(got[r], *m, lens[b], 6.0, 2 if codes else 1)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("L,n,hq,hkv,window,sink", [
    (20011, 1, 4, 1, 0, 0), (20011, 20, 8, 2, 0, 0), (20011, 300, 8, 1, 0, 0), (40009, 3, 4, 1, 0, 0),
    (20011, 33, 4, 1, 9000, 130), (700, 700, 4, 1, 0, 0), (5003, 1000, 8, 1, 0, 0)])
def test_prefill(D, codes, L, n, hq, hkv, window, sink):
    prefill(Layout(1, hkv, L, True, page=16, seed=1), [L], [n], hq, D, codes, [window] if window else None, sink)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (8, 1)])
def test_a_long_chunk_beside_single_tokens(D, codes, hq, hkv):
    """What a server that batches continuously sends: a prompt's chunk and one token of every chat."""
    new = [1, 1, 1, 700, 1, 0, 1, 1]
    lens = [900, 1, 129, 1500, 2000, 7, 128, 3000]
    prefill(Layout(8, hkv, 3000, True, page=16, seed=2), lens, new, hq, D, codes, seed=3)
    prefill(Layout(8, hkv, 3000, True, page=16, seed=2), lens, new, hq, D, codes, [0, 5, 100, 600, 1000, 0, 1, 0], 4)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("tq", [1, 3])
@pytest.mark.parametrize("lens,window,sink", [([20011, 40009, 5], [0, 20000, 3], 4), ([300, 2000, 16], [33, 200, 1], 17),
                                              ([5000, 40, 4999], [100, 0, 2000], 500)])
def test_sinks(D, codes, tq, lens, window, sink):
    """int8 V: the scale is split into a power of two and a factor on the weight, so that a weight is rounded
    once, as with fp16 V."""
    hq, hkv = 8, 2
    lay = Layout(3, hkv, max(lens), True, page=16, seed=4)
    rng = np.random.RandomState(5)
    k, v, s, val = cache(lay, D, codes, rng)
    q = rng.randn(3, tq, hq, D).astype(np.float16)
    out = torch.full(q.shape, 9.0, dtype=torch.float16, device="cuda")
    qd, kd, vd, sd = gpu(q, k, v, s)
    fa.fa_decode_sinks(qd, kd, vd, sd, lay.table_gpu(), ints(lens), hq, hkv, D, D ** -0.5, ints(window), out,
                       n_sink=sink, workspace=fa.alloc_workspace_sinks(3, tq, hq, hkv, D, lay.capacity))
    assert binding.fa_decode_device_status() == 0
    for b in range(3):
        m = rows(q[b], np.arange(lens[b] - tq, lens[b]), lay.dense(k, b)[:, :lens[b]], lay.dense(val, b)[:, :lens[b]],
                 D ** -0.5, window[b], sink, hkv)
        check(f64(out[b]), *m, lens[b], 6.0, 1)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("L", [4096, 32768])
def test_prefill_behind_a_dominant_key(D, codes, L):
    """A first key with half of every row's weight and V of 0: the keys behind it keep fp16's bits."""
    hq, hkv, n = 4, 1, 20
    rng = np.random.RandomState(3)
    lay = Layout(1, hkv, L, False)
    k, v, s, val = cache(lay, D, codes, rng)
    k = (k * np.float16(0.02)).astype(np.float16)
    k[:, :, 0, 0], k[:, :, 1:, 0] = np.log(L) / 4.0, 0
    v[:, :, 0], val[:, :, 0] = 0, 0
    q = rng.randn(n, hq, D).astype(np.float16)
    q[..., 0] = 4.0
    out = torch.empty(n, hq, D, dtype=torch.float16, device="cuda")
    qd, kd, vd, sd = gpu(q, k, v, s)
    fa.fa_prefill(qd, kd, vd, sd, None, ints([0, n]), ints([L]), hq, hkv, D, 1.0, None, out,
                  workspace=fa.alloc_workspace_prefill(1, n, hq, hkv, D, L))
    check(f64(out), *rows(q, np.arange(L - n, L), k[0], val[0], 1.0, 0, 0, hkv), L, 6.0, 2 if codes else 1)
