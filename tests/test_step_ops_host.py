"""Rotation tables and refusals of the rotation, chunk and sink calls (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import decode_step_kv_gb300 as fa
from decode_step_kv_gb300 import binding
from _step_ops import rates

P = ctypes.c_void_p
FAKE = 1 << 40                     # a 16-byte aligned address that is never read


def at(i, off=0):
    """Address i of arrays far apart."""
    return P(FAKE + (i << 36) + off)


def code(name, *args):
    rc = getattr(binding.load(), name)(*args)
    if rc:
        assert name in binding.load().fa_decode_last_error().decode() or \
            "fa_decode" in binding.load().fa_decode_last_error().decode()
    return rc


@pytest.mark.parametrize("rot", [2, 16, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0), ("yarn", 1.0)])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_table(rot, scaling, factor, base):
    table, mag = fa.fa_rope_table(rot, base, scaling=scaling, factor=factor, original_len=4096, device="cpu")
    want, want_mag = rates(rot, base, scaling, factor, 4096)
    got = table.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * np.pi
    assert table.shape == (rot // 2,)
    # two 64-bit powers and products, each within a few steps
    assert np.allclose(got, want, rtol=2.0 ** -48, atol=2.0 ** -60)
    assert mag == pytest.approx(want_mag, rel=2.0 ** -23)


def test_table_refusals():
    for kw, want in [(dict(rot_dim=3), -6), (dict(rot_dim=0), -6), (dict(base=1.0), -5), (dict(factor=0.5), -5),
                     (dict(factor=float("nan")), -5), (dict(scaling="yarn", original_len=0), -5)]:
        with pytest.raises(fa.FaDecodeError) as e:
            fa.fa_rope_table(**{"rot_dim": 128, "device": "cpu", **kw})
        assert e.value.code == want
    with pytest.raises(ValueError):
        fa.fa_rope_table(128, scaling="other", device="cpu")


def rope(**kw):
    a = dict(x=at(0), dtype=1, out=at(1), out_dtype=1, weight=None, eps=1e-6, positions=at(2), freqs=at(3), rot=128,
             inter=0, mag=1.0, n=4, h=2, d=128, xs=256, os=256)
    a.update(kw)
    return code("fa_rope", a["x"], a["dtype"], a["out"], a["out_dtype"], a["weight"], a["eps"], a["positions"],
                a["freqs"], a["rot"], a["inter"], a["mag"], a["n"], a["h"], a["d"], a["xs"], a["os"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=64), -2), (dict(dtype=3), -6), (dict(out_dtype=-1), -6), (dict(rot=8), -6), (dict(rot=144), -6),
    (dict(rot=-16), -6), (dict(mag=float("inf")), -5), (dict(eps=-1.0), -5), (dict(eps=float("nan")), -5),
    (dict(freqs=None), -1), (dict(freqs=at(3, 4)), -9), (dict(h=0), -3), (dict(n=-1), -6), (dict(xs=255), -6),
    (dict(os=128), -6), (dict(x=None), -1), (dict(out=None), -1), (dict(positions=None), -1), (dict(x=at(0, 8)), -9),
    (dict(xs=260), -9), (dict(positions=at(2, 2)), -9), (dict(weight=at(4, 2)), -9), (dict(out=at(0, 16)), -7),
    (dict(out=at(0), os=512), -7), (dict(out=at(0), out_dtype=2), -7), (dict(out=at(2)), -7), (dict(out=at(3)), -7),
    (dict(weight=at(1, 64)), -7), (dict(n=0, x=None, out=None, positions=None), 0)])
def test_rope_refusals(kw, want):
    assert rope(**kw) == want


def append(**kw):
    a = dict(q=at(0), k=at(1), v=at(2), dtype=1, qs=1024, ks=256, vs=256, qw=None, kw=None, eps=1e-6, freqs=at(3),
             rot=128, inter=0, mag=1.0, qo=at(4), kc=at(5), vc=at(6), vsc=None, bt=at(7), st=at(8), pos=at(9), rp=None,
             B=2, n=5, hq=8, hkv=2, d=128, page=16, blocks=4, total=9)
    a.update(kw)
    return code("fa_rope_append_kv", *(a[x] for x in (
        "q", "k", "v", "dtype", "qs", "ks", "vs", "qw", "kw", "eps", "freqs", "rot", "inter", "mag", "qo", "kc", "vc",
        "vsc", "bt", "st", "pos", "rp", "B", "n", "hq", "hkv", "d", "page", "blocks", "total")), None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=96), -2), (dict(rot=20), -6), (dict(hkv=0), -3), (dict(hq=-1), -3), (dict(B=-1), -6), (dict(n=-1), -6),
    (dict(blocks=0), -6), (dict(page=24), -6), (dict(total=0), -6), (dict(st=None), -6), (dict(qs=512), -6),
    (dict(ks=128), -6), (dict(vs=0), -6), (dict(q=None), -1), (dict(k=None), -1), (dict(qo=None), -1),
    (dict(pos=None), -1), (dict(kc=None), -1), (dict(k=at(1, 2)), -9), (dict(ks=260), -9), (dict(kc=at(5, 8)), -9),
    (dict(vsc=at(10, 1)), -9), (dict(st=at(8, 2)), -9), (dict(rp=at(11, 1)), -9), (dict(qo=at(0)), -7),
    (dict(kc=at(6)), -7), (dict(vc=at(5, 4096)), -7), (dict(qo=at(5)), -7), (dict(pos=at(5)), -7),
    (dict(bt=None, blocks=(1 << 30) + 1), -6), (dict(n=0, k=None, v=None), 0), (dict(B=0), 0)])
def test_append_refusals(kw, want):
    assert append(**kw) == want


def prefill(**kw):
    a = dict(q=at(0), k=at(1), v=at(2), vsc=None, bt=at(3), st=at(4), lens=at(5), hq=8, hkv=2, d=128, scale=0.1,
             window=None, sink=0, out=at(6), B=2, n=5, page=16, blocks=4, total=9, ws=at(7), bytes=1 << 34)
    a.update(kw)
    return code("fa_prefill", *(a[x] for x in (
        "q", "k", "v", "vsc", "bt", "st", "lens", "hq", "hkv", "d", "scale", "window", "sink", "out", "B", "n", "page",
        "blocks", "total", "ws", "bytes")), None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=64), -2), (dict(hq=7), -3), (dict(hq=130), -3), (dict(hkv=0), -3), (dict(scale=float("nan")), -5),
    (dict(B=-1), -6), (dict(B=65536), -6), (dict(n=-1), -6), (dict(page=8), -6), (dict(total=0), -6),
    (dict(blocks=0), -6), (dict(sink=-1), -6), (dict(st=None), -6), (dict(vsc=at(9, 8)), -9), (dict(total=1 << 26), -6),
    (dict(bt=None, blocks=(1 << 30) + 1), -6), (dict(q=None), -1), (dict(lens=None), -1), (dict(out=None), -1),
    (dict(q=at(0, 8)), -9), (dict(window=at(8, 2)), -9), (dict(st=at(4, 1)), -9), (dict(ws=at(7, 8)), -9),
    (dict(B=0, q=None), 0), (dict(n=0, q=None, out=None), 0)])
def test_prefill_refusals(kw, want):
    assert prefill(**kw) == want


def sinks(**kw):
    a = dict(q=at(0), k=at(1), v=at(2), vsc=None, bt=at(3), lens=at(5), tq=1, hq=8, hkv=2, d=128, scale=0.1,
             window=at(8), sink=4, out=at(6), B=2, page=16, blocks=4, total=9, ws=at(7), bytes=1 << 34)
    a.update(kw)
    return code("fa_decode_sinks", *(a[x] for x in (
        "q", "k", "v", "vsc", "bt", "lens", "tq", "hq", "hkv", "d", "scale", "window", "sink", "out", "B", "page",
        "blocks", "total", "ws", "bytes")), None)


@pytest.mark.parametrize("kw,want", [
    (dict(d=64), -2), (dict(hq=7), -3), (dict(tq=0), -6), (dict(tq=257), -6), (dict(sink=-1), -6),
    (dict(sink=(1 << 30) + 1), -6), (dict(page=20), -6), (dict(q=None), -1), (dict(out=at(0)), -7),
    (dict(window=at(8, 1)), -9), (dict(B=0, q=None), 0)])
def test_sinks_refusals(kw, want):
    assert sinks(**kw) == want


def test_workspace_sizes():
    for f in (fa.fa_prefill_workspace_size, fa.fa_decode_sinks_workspace_size):
        assert f(0, 1, 8, 2, 128, 100, 152) == 0
        assert f(1, 0, 8, 2, 128, 100, 152) == 0
        assert f(1, 1, 8, 3, 128, 100, 152) == 0
        assert f(1, 1, 8, 2, 64, 100, 152) == 0
        assert f(1, 1, 8, 2, 128, -1, 152) == 0
        assert 0 < f(2, 7, 8, 2, 128, 5000, 152) < 1 << 30


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("size", [fa.fa_prefill_workspace_size, fa.fa_decode_sinks_workspace_size])
def test_workspace_serves_smaller_calls(D, size):
    rng = np.random.RandomState(1)
    for _ in range(300):
        hkv = int(rng.choice([1, 2, 8]))
        hq = hkv * int(rng.choice([1, 3, 4, 8]))
        most = [int(2 ** rng.uniform(0, x)) for x in (8, 8, 16)]
        less = [int(rng.randint(1, m + 1)) for m in most]
        assert size(less[0], less[1], hq, hkv, D, less[2], 152) <= size(most[0], most[1], hq, hkv, D, most[2], 152)
