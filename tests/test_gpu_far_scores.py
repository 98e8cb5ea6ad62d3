"""Scores of any size that finite inputs give: up to 2^36 in either direction, where a 32-bit score is a
multiple of 2^13, so that a shift of the softmax's reference by a few powers of two is lost or doubled.

Keys have levels: within a level they are the same key, so their scores are equal whatever the rounding, and
levels lie at least 2^11 apart (in log2 units), so that the highest level takes all the weight.  The result is
the mean of V over its visible keys."""
import numpy as np
import pytest
import torch

import decode_step_kv_gb300 as fa
from decode_step_kv_gb300 import binding
from _cache_ops import dequantize, pack, quantize
from _step_ops import f64

pytestmark = pytest.mark.gpu

HKV, G = 2, 4
SIZES = [20, 27, 30, 31, 33, 36]        # log2 of q . k


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def levels(L, order):
    """Level of every key, 0 the smallest."""
    if order == "flat":
        return np.zeros(L, dtype=int)
    up = np.arange(L) * 4 // L
    return {"up": up, "down": 3 - up, "mixed": np.arange(L) * 7 % 4}[order]


def inputs(D, n, L, e, order, sign):
    """q [n, Hq, D] and k [Hkv, L, D] with q . k of about 2^e; level i of the keys is 1 + i / 32 of the first
    (sign < 0: the score's sign; the level of the largest score is then the lowest)."""
    a = 2.0 ** ((e - np.log2(D)) // 2)
    b = 2.0 ** e / D / a
    q = np.full((n, HKV * G, D), a * (1 + 5 / 1024), dtype=np.float16)
    lev = levels(L, order)
    k = np.broadcast_to((b * (1 + lev / 32 + 3 / 1024))[None, :, None], (HKV, L, D)).astype(np.float16)
    return q, k, lev if sign > 0 else -lev


def check(got, v, lev, at, window=0, sink=0):
    """got [n, Hq, D]; v [Hkv, L, D]; at [n]."""
    got = f64(got)
    assert np.isfinite(got).all()
    for i, p in enumerate(at):
        t = np.arange(p + 1)
        if window:
            t = t[(t > p - window) | (t < sink)]
        t = t[lev[t] == lev[t].max()]
        for h in range(HKV):
            want, size = v[h][t].mean(0), np.abs(v[h][t]).mean(0)
            # fp16: the weights, V's values or weights times scales where V has scales, and the output
            err = np.abs(got[i, h * G:(h + 1) * G] - want)
            assert (err <= (3 * 2.0 ** -11 + 2.0 ** -15) * size + 2.0 ** -24).all(), (i, err.max())


def int8(v):
    s = (np.abs(v.reshape(*v.shape[:-1], -1, 32)).max(-1) / 127).astype(np.float16)
    c = np.clip(np.rint(v.reshape(*v.shape[:-1], -1, 32) / s[..., None].astype(np.float64)), -127, 127)
    return c.reshape(v.shape).astype(np.int8), s, (c * s[..., None].astype(np.float64)).reshape(v.shape)


def values(L, D, codes):
    v = np.random.RandomState(1).randn(HKV, L, D).astype(np.float16)
    if codes:
        return int8(v.astype(np.float64))
    return v, None, v.astype(np.float64)


def gpu(*arrays):
    return [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in arrays]


@pytest.mark.parametrize("e", SIZES)
@pytest.mark.parametrize("D,codes", [(128, False), (256, False), (128, True), (256, True)])
@pytest.mark.parametrize("order,sign", [("flat", 1), ("flat", -1), ("up", 1), ("down", 1), ("mixed", -1)])
@pytest.mark.parametrize("n,L", [(40, 700), (1, 6000)])
def test_prefill(e, D, codes, order, sign, n, L):
    q, k, lev = inputs(D, n, L, e, order, sign)
    v, s, val = values(L, D, codes)
    out = torch.zeros(n, HKV * G, D, dtype=torch.float16, device="cuda")
    qd, kd, vd, sd = gpu(q, k[None], v[None], None if s is None else s[None])
    fa.fa_prefill(qd, kd, vd, sd, None, ints([0, n]), ints([L]), HKV * G, HKV, D, sign * D ** -0.5, None, out,
                  workspace=fa.alloc_workspace_prefill(1, n, HKV * G, HKV, D, L))
    check(out, val, lev, range(L - n, L))
    assert binding.fa_decode_device_status() == 0


@pytest.mark.parametrize("e", SIZES)
@pytest.mark.parametrize("D,codes", [(128, False), (256, False), (128, True), (256, True)])
@pytest.mark.parametrize("order,sign", [("flat", 1), ("flat", -1), ("up", 1), ("down", 1), ("mixed", -1)])
@pytest.mark.parametrize("tq,L", [(1, 704), (3, 704), (1, 6000)])
def test_sinks(e, D, codes, order, sign, tq, L):
    q, k, lev = inputs(D, tq, L, e, order, sign)
    v, s, val = values(L, D, codes)
    out = torch.zeros(1, tq, HKV * G, D, dtype=torch.float16, device="cuda")
    qd, kd, vd, sd = gpu(q[None], k[None], v[None], None if s is None else s[None])
    fa.fa_decode_sinks(qd, kd, vd, sd, None, ints([L]), HKV * G, HKV, D, sign * D ** -0.5, ints([400]), out, n_sink=5,
                       workspace=fa.alloc_workspace_sinks(1, tq, HKV * G, HKV, D, L))
    check(out[0], val, lev, range(L - tq, L), 400, 5)
    assert binding.fa_decode_device_status() == 0


@pytest.mark.parametrize("e", SIZES)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("order,sign", [("flat", 1), ("flat", -1), ("up", 1), ("down", 1), ("mixed", -1)])
@pytest.mark.parametrize("tq,L", [(1, 704), (4, 704), (16, 704), (1, 6000), (16, 6000)])
def test_int4(e, D, order, sign, tq, L):
    """4-bit caches.  A level's keys have the same codes and scale; levels differ by their scales."""
    q, k, lev = inputs(D, tq, L, e, order, sign)
    v, _, _ = values(L, D, False)
    (kc, ks), (vc, vs) = (quantize(x.astype(np.float64)) for x in (k, v))
    kc, vc = pack(kc), pack(vc)
    out = torch.zeros(1, tq, HKV * G, D, dtype=torch.float16, device="cuda")
    qd, *caches = gpu(q[None], kc[None], ks[None], vc[None], vs[None])
    fa.fa_decode_int4(qd, *caches, None, ints([L]), HKV * G, HKV, D, sign * D ** -0.5, None, out,
                      workspace=fa.alloc_workspace_int4(1, tq, HKV * G, HKV, D, L))
    check(out[0], dequantize(vc, vs), lev, range(L - tq, L))
    assert binding.fa_decode_device_status() == 0
