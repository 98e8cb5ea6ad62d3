"""Documented no-ops with the null pointers that empty tensors have."""
import pytest
import torch

from decode_step_kv_gb300 import binding as fa

from test_cache_ops_host import APPEND, DECODE, EVICT, GATHER, WEIGHTS, rc_of


@pytest.fixture(scope="module")
def lib():
    return fa.load()


@pytest.mark.parametrize("name,args,kw", [
    ("fa_append_kv_int4", APPEND, dict(batch=0, k=None, v=None, bt=None, pos=None)),
    ("fa_append_kv_int4", APPEND, dict(T=0, k=None, v=None)),
    ("fa_append_kv_int4", APPEND, dict(batch=0, k=None, v=None, kc=None, ks=None, vc=None, vs=None,
                                       bt=None, pos=None)),
    ("fa_gather_kv_int4", GATHER, dict(batch=0, k=None, v=None, bt=None, pos=None)),
    ("fa_gather_kv_int4", GATHER, dict(T=0, k=None, v=None)),
    ("fa_decode_int4", DECODE, dict(batch=0, q=None, out=None, bt=None, sl=None, ws=None, wsb=0)),
    ("fa_decode_weights", WEIGHTS, dict(batch=0, q=None, out=None, bt=None, sl=None, ws=None, wsb=0)),
    ("fa_decode_weights", WEIGHTS, dict(batch=0, q=None, out=None, bt=None, sl=None, kc=None, vc=None,
                                        acc=None, ws=None, wsb=0)),
    ("fa_evict_kv", EVICT, dict(batch=0, sl=None, bt=None, nl=None, kept=None)),
    ("fa_evict_kv", EVICT, dict(batch=0, sl=None, bt=None, nl=None, kept=None, kc=None, vc=None, acc=None)),
])
def test_nothing_to_do(lib, name, args, kw):
    rc, msg = rc_of(lib, name, args, kw)
    assert rc == 0 and msg == ""


@pytest.mark.parametrize("name,args,kw,code", [
    ("fa_append_kv_int4", APPEND, dict(batch=0, d=64), -2), ("fa_append_kv_int4", APPEND, dict(T=0, hkv=0), -3),
    ("fa_gather_kv_int4", GATHER, dict(batch=-1, k=None), -6), ("fa_gather_kv_int4", GATHER, dict(T=-1), -6),
    ("fa_append_kv_int4", APPEND, dict(k=None), -1), ("fa_gather_kv_int4", GATHER, dict(v=None), -1),
    ("fa_decode_weights", WEIGHTS, dict(batch=0, d=64), -2), ("fa_evict_kv", EVICT, dict(batch=0, budget=0), -6)])
def test_sizes_are_checked_all_the_same(lib, name, args, kw, code):
    rc, msg = rc_of(lib, name, args, kw)
    assert rc == code and msg.startswith("fa_decode" if name == "fa_decode_weights" else name)


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [False, True])
def test_empty_tensors_through_the_binding(paged):
    """No sequence (a paged pool stays), and no token of two sequences."""
    def z(*shape, dtype=torch.float16):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    for b, t in ((0, 3), (2, 0)):
        n = 5 if paged else b
        table = z(b, 3, dtype=torch.int32) if paged else None
        rows = (n, 2, 16 if paged else 48)
        codes = [z(*rows, 64, dtype=torch.uint8) for _ in range(2)]
        scales = [z(*rows, 4) for _ in range(2)]
        c = (codes[0], scales[0], codes[1], scales[1], table)
        lens, acc = z(b, dtype=torch.int32), z(*rows, dtype=torch.float32)
        fa.fa_append_kv_int4(z(b, t, 2, 128, dtype=torch.float32), z(b, t, 2, 128, dtype=torch.float32), *c, lens)
        fa.fa_gather_kv_int4(*c, lens, z(b, t, 2, 128), z(b, t, 2, 128))
        if b:
            continue
        q, out = z(0, 1, 4, 128), z(0, 1, 4, 128)
        fa.fa_decode_int4(q, *c, lens, 4, 2, 128, 0.1, None, out, acc=acc)
        k, v = z(*rows, 128), z(*rows, 128)
        fa.fa_decode_weights(q, k, v, None, table, lens, 4, 2, 128, 0.1, None, out, acc)
        fa.fa_evict_kv(k, v, acc, table, lens, z(0, dtype=torch.int32), budget=16, n_sink=2, n_recent=4,
                       kept=z(0, 2, 16, dtype=torch.int32))
