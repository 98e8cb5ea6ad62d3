"""Host-side checks of the 4-bit cache, recorded-weights and eviction entry points (no GPU)."""
import numpy as np
import pytest
import torch

from decode_step_kv_gb300 import binding

from _cache_ops import pack, quantize, unpack

A = 1 << 24            # fake, 16-byte aligned device addresses: never dereferenced


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def rc_of(lib, name, defaults, kw):
    args = dict(defaults)
    args.update(kw)
    return getattr(lib, name)(*args.values()), lib.fa_decode_last_error().decode()


APPEND = dict(k=A, v=2 * A, kc=3 * A, ks=4 * A, vc=5 * A, vs=6 * A, bt=7 * A, pos=8 * A, n_new=None,
              batch=2, T=3, hkv=2, d=128, page=16, maxb=4, nblk=20, stream=None)
GATHER = dict(kc=3 * A, ks=4 * A, vc=5 * A, vs=6 * A, bt=7 * A, pos=8 * A, n_rows=None, k=A, v=2 * A,
              batch=2, T=3, hkv=2, d=128, page=16, maxb=4, nblk=20, stream=None)
DECODE = dict(q=A, kc=3 * A, ks=4 * A, vc=5 * A, vs=6 * A, bt=7 * A, sl=8 * A, tq=1, hq=8, hkv=2,
              d=128, scale=0.1, win=None, out=9 * A, acc=None, batch=2, page=16, maxb=4, nblk=20,
              ws=10 * A, wsb=1 << 23, stream=None)
WEIGHTS = dict(q=A, kc=3 * A, vc=5 * A, vs=None, bt=7 * A, sl=8 * A, tq=1, hq=8, hkv=2, d=128,
               scale=0.1, win=None, out=9 * A, acc=11 * A, batch=2, page=16, maxb=4, nblk=20,
               ws=10 * A, wsb=1 << 23, stream=None)
EVICT = dict(kc=A, vc=2 * A, ks=None, vs=None, acc=3 * A, bt=4 * A, sl=5 * A, nl=6 * A, kept=7 * A,
             budget=32, sink=4, recent=8, batch=2, hkv=2, d=128, page=16, maxb=4, nblk=20, stream=None)

CACHE = [(dict(d=64), -2), (dict(d=192), -2), (dict(hkv=0), -3), (dict(hkv=5000), -3),
         (dict(batch=-1), -6), (dict(batch=70000), -6), (dict(maxb=0), -6), (dict(page=8), -6),
         (dict(page=24), -6), (dict(nblk=0), -6), (dict(bt=None, maxb=30), -6),
         (dict(maxb=1 << 27, page=16), -6)]


@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(kc=None), -1), (dict(ks=None), -1),
    (dict(vc=None), -1), (dict(vs=None), -1), (dict(pos=None), -1), (dict(T=-1), -6),
    (dict(k=A + 4), -9), (dict(kc=3 * A + 8), -9), (dict(ks=4 * A + 2), -9), (dict(pos=8 * A + 2), -9),
    (dict(n_new=9 * A + 1), -9), (dict(bt=7 * A + 2), -9),
    (dict(kc=A), -7), (dict(vs=2 * A), -7), (dict(kc=5 * A), -7), (dict(ks=8 * A), -7),
    (dict(vc=7 * A), -7),
    (dict(batch=0), 0), (dict(T=0), 0)])
def test_append_checks(lib, kw, code):
    rc, msg = rc_of(lib, "fa_append_kv_int4", APPEND, kw)
    assert rc == code, msg
    assert (msg == "") == (code == 0) and (code == 0 or msg.startswith("fa_append_kv_int4"))


@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(kc=None), -1), (dict(ks=None), -1),
    (dict(vc=None), -1), (dict(vs=None), -1), (dict(pos=None), -1), (dict(T=-1), -6),
    (dict(k=A + 8), -9), (dict(vc=5 * A + 4), -9), (dict(n_rows=9 * A + 2), -9),
    (dict(k=2 * A), -7), (dict(k=3 * A), -7), (dict(v=6 * A), -7), (dict(v=7 * A), -7),
    (dict(batch=0), 0), (dict(T=0), 0)])
def test_gather_checks(lib, kw, code):
    rc, msg = rc_of(lib, "fa_gather_kv_int4", GATHER, kw)
    assert rc == code, msg


@pytest.mark.parametrize("kw,code", CACHE + [
    (dict(q=None), -1), (dict(kc=None), -1), (dict(ks=None), -1), (dict(vc=None), -1),
    (dict(vs=None), -1), (dict(sl=None), -1), (dict(out=None), -1),
    (dict(hq=7), -3), (dict(hq=0), -3), (dict(hq=130), -3), (dict(tq=0), -6), (dict(tq=257), -6),
    (dict(scale=float("nan")), -5), (dict(scale=float("inf")), -5),
    (dict(q=A + 2), -9), (dict(ks=4 * A + 8), -9), (dict(out=9 * A + 8), -9), (dict(ws=10 * A + 4), -9),
    (dict(acc=11 * A + 2), -9), (dict(win=12 * A + 2), -9), (dict(sl=8 * A + 1), -9),
    (dict(out=A), -7), (dict(out=3 * A), -7), (dict(out=8 * A), -7), (dict(acc=9 * A), -7),
    (dict(acc=4 * A), -7), (dict(acc=7 * A), -7), (dict(batch=0), 0)])
def test_decode_checks(lib, kw, code):
    rc, msg = rc_of(lib, "fa_decode_int4", DECODE, kw)
    assert rc == code, msg


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(kc=None), -1), (dict(acc=None), -1), (dict(out=None), -1),
    (dict(d=64), -2), (dict(hq=7), -3), (dict(hkv=0), -3), (dict(tq=0), -6), (dict(tq=300), -6),
    (dict(page=20), -6), (dict(scale=float("nan")), -5), (dict(out=9 * A + 4), -9),
    (dict(acc=11 * A + 1), -9), (dict(out=A), -7), (dict(acc=9 * A), -7), (dict(acc=3 * A), -7),
    (dict(acc=5 * A), -7), (dict(vs=12 * A, acc=12 * A), -7), (dict(acc=8 * A), -7),
    (dict(batch=0), 0)])
def test_weights_checks(lib, kw, code):
    rc, msg = rc_of(lib, "fa_decode_weights", WEIGHTS, kw)
    assert rc == code, msg


@pytest.mark.parametrize("kw,code", [
    (dict(kc=None), -1), (dict(vc=None), -1), (dict(acc=None), -1), (dict(sl=None), -1),
    (dict(nl=None), -1), (dict(kept=None), -1), (dict(ks=8 * A), -1),
    (dict(d=64), -2), (dict(hkv=0), -3), (dict(batch=-1), -6), (dict(maxb=0), -6), (dict(page=8), -6),
    (dict(nblk=0), -6), (dict(budget=0), -6), (dict(sink=-1), -6), (dict(recent=-1), -6),
    (dict(sink=20, recent=13), -6), (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), -6),
    (dict(kc=A + 8), -9), (dict(vs=8 * A + 8), -9), (dict(acc=3 * A + 2), -9), (dict(kept=7 * A + 2), -9),
    (dict(nl=5 * A), -7), (dict(kept=A), -7), (dict(acc=2 * A), -7), (dict(kc=2 * A), -7),
    (dict(vs=2 * A + 16), -7), (dict(kept=4 * A), -7), (dict(batch=0), 0)])
def test_evict_checks(lib, kw, code):
    rc, msg = rc_of(lib, "fa_evict_kv", EVICT, kw)
    assert rc == code, msg


@pytest.mark.parametrize("kw", [dict(nblk=1 << 26), dict(bt=None, maxb=1 << 29, hq=4)])
def test_caches_of_too_many_rows(lib, kw):
    """Cache rows are counted in 32 bits: 2^31 of them are refused, one block fewer is not."""
    far = {n: (i + 1) << 44 for i, n in enumerate(("kc", "ks", "vc", "vs", "acc", "ws"))}
    at = {n: x for n, x in far.items() if DECODE.get(n) is not None}
    rc, msg = rc_of(lib, "fa_decode_int4", DECODE, {**at, **kw})
    assert rc == -6 and "2^31 rows" in msg
    if "nblk" in kw:
        rc, msg = rc_of(lib, "fa_decode_int4", DECODE, {**at, "nblk": (1 << 26) - 1, "wsb": 0})
        assert rc in (-4, -8) and "2^31 rows" not in msg, msg       # the workspace, or no device
    at = {n: x for n, x in far.items() if WEIGHTS.get(n) is not None}
    rc, msg = rc_of(lib, "fa_decode_weights", WEIGHTS, {**at, **kw})
    assert rc == -6 and "rows" in msg or rc == -8                   # planned for a device first


def test_workspace_sizes():
    plain = binding.fa_decode_int4_workspace_size(4, 1, 8, 2, 128, 1000, False, 152)
    with_weights = binding.fa_decode_int4_workspace_size(4, 1, 8, 2, 128, 1000, True, 152)
    assert 0 < plain < with_weights
    # scores: 4 sequences x 8 heads x 1008 keys, and the 32 rows' log-sum-exps
    assert with_weights >= plain + 4 * (4 * 8 * 1008 + 32)
    assert binding.fa_decode_weights_workspace_size(4, 1, 8, 2, 128, 1000, 152) >= 4 * 4 * 8 * 1008
    for bad in ((0, 1, 8, 2, 128, 1000), (4, 0, 8, 2, 128, 1000), (4, 1, 7, 2, 128, 1000),
                (4, 1, 8, 2, 64, 1000), (4, 1, 8, 2, 128, -1)):
        assert binding.fa_decode_int4_workspace_size(*bad, True, 152) == 0
        assert binding.fa_decode_weights_workspace_size(*bad, 152) == 0


def test_binding_refuses_wrong_types_and_shapes():
    codes, scales = torch.zeros((4, 2, 16, 64), dtype=torch.uint8), torch.zeros((4, 2, 16, 4)).half()
    table, pos = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    new = torch.zeros((1, 1, 2, 128))
    for bad in (dict(k_codes=codes.float()), dict(k_scales=scales[..., :2]), dict(v_codes=codes[:3]),
                dict(k_codes=codes[0]), dict(block_table=table[0]), dict(block_table=None)):
        a = dict(k_codes=codes, k_scales=scales, v_codes=codes.clone(), v_scales=scales.clone(),
                 block_table=table, positions=pos)
        a.update(bad)
        with pytest.raises(ValueError):
            binding.fa_append_kv_int4(new, new, **a)
    with pytest.raises(ValueError, match="current CUDA device"):
        binding.fa_append_kv_int4(new, new, codes, scales, codes, scales, table, pos)
    with pytest.raises(ValueError, match="q must be"):
        binding.fa_decode_int4(torch.zeros(1, 8, 64).half(), codes, scales, codes, scales, table, pos,
                               8, 2, 128, 0.1, None, torch.zeros(1, 8, 64).half())
    with pytest.raises(ValueError, match="kv heads"):
        binding.fa_decode_weights(torch.zeros(1, 8, 128).half(), codes[0], codes[0], None, None, pos, 8,
                                  2, 128, 0.1, None, torch.zeros(1, 8, 128).half(), torch.zeros(1))


def test_plain_codec_round_trip():
    """The tests' own packing: words in the documented order, every code back."""
    x = np.random.RandomState(0).standard_normal((3, 256)).astype(np.float32)
    codes, s = quantize(x)
    by = pack(codes)
    assert np.array_equal(unpack(by), codes) and np.abs(codes).max() == 7
    assert np.all(np.abs(codes * np.repeat(s.astype(float), 32, -1) - x) <= np.repeat(s.astype(float), 32, -1) * 0.51)
    one = np.zeros((1, 128), dtype=np.int64)
    one[0, 32 * 2 + 8 * 3 + 5] = 7                 # block 2, octet 3, element 5: word 3 * 4 + 2
    want = np.full(64, 0x88, dtype=np.uint8)
    want[(3 * 4 + 2) * 4 + 2] = 0xf8
    assert np.array_equal(pack(one)[0], want)
