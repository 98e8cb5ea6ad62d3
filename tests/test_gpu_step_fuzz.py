"""Random shapes of chunk attention, decode with sinks and the rotated append, against 64-bit forms."""
import numpy as np
import pytest
import torch

import decode_step_kv_gb300 as fa
from decode_step_kv_gb300 import binding
from _cache_ops import Layout
from _step_ops import attend_rows, attend_tolerance, f64, rates, turn, turn_tolerance
from test_gpu_prefill import caches, ints, run_prefill, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(40))
def test_prefill(seed):
    rng = np.random.RandomState(1000 + seed)
    D = int(rng.choice([128, 256]))
    hkv = int(rng.choice([1, 1, 2, 4]))
    hq = hkv * int(rng.choice([1, 2, 3, 4, 7, 8, 16]))
    B = int(rng.randint(1, 7))
    most = int(rng.choice([3, 40, 300, 900]))
    new = [int(x) for x in rng.randint(0, most + 1, B)]
    while sum(new) > 1200:
        new[int(np.argmax(new))] //= 2
    if not sum(new):
        new[0] = 1
    lens = [max(0, n + int(rng.choice([0, -3, rng.randint(0, 900), rng.randint(0, 60)]))) for n in new]
    cap = max(max(lens), 1) + int(rng.randint(0, 40))
    paged = bool(rng.rand() < 0.7)
    lay = Layout(B, hkv, cap, paged, page=int(rng.choice([16, 16, 32, 48, 64, 80, 128])), seed=seed,
                 room=int(rng.choice([0, 5000])))
    window, sink = None, 0
    if rng.rand() < 0.6:
        window = [int(rng.choice([0, rng.randint(1, 200), rng.randint(1, 1000)])) for _ in range(B)]
        sink = int(rng.choice([0, 1, 4, 30, 140, 500]))
    gap = int(rng.choice([0, 5]))
    starts = (gap + np.concatenate([[0], np.cumsum(new)])).tolist()
    run_prefill(lay, lens, new, hq, D, window=window, sink=sink, seed=seed, starts=starts, tokens=starts[-1] + gap,
                scale=float(rng.choice([D ** -0.5, -0.05, 0.2])), int8=bool(seed % 3 == 2))


@pytest.mark.parametrize("seed", range(30))
def test_sinks(seed):
    rng = np.random.RandomState(2000 + seed)
    D = int(rng.choice([128, 256]))
    hkv = int(rng.choice([1, 2, 4]))
    hq = hkv * int(rng.choice([1, 3, 4, 8, 12]))
    B, tq = int(rng.randint(1, 9)), int(rng.choice([1, 1, 2, 3, 6, 20]))
    cap = int(rng.choice([40, 300, 2000, 6000]))
    lens = [int(x) for x in rng.randint(0, cap + 1, B)]
    int8 = bool(rng.rand() < 0.5)
    paged = bool(rng.rand() < 0.6)
    room = int(rng.choice([0, 0, 600000]))          # a table with room for a pool that streams: 16 columns a unit
    lay = Layout(B, hkv, -(-cap // 16) * 16, paged, page=int(rng.choice([16, 32, 48])), seed=seed, room=room)
    w = [int(rng.choice([0, rng.randint(1, 100), rng.randint(1, cap + 10)])) for _ in range(B)]
    sink = int(rng.choice([0, 1, 4, 17, 200]))
    k, v, s = caches(lay, lens, [tq] * B, w, sink, D, seed, int8=int8)
    q = rng.randn(B, tq, hq, D).astype(np.float16)
    out = torch.full((B, tq, hq, D), 9.0, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_sinks(B, tq, hq, hkv, D, lay.capacity)
    ws.fill_(255)
    fa.fa_decode_sinks(*(torch.from_numpy(x).cuda() for x in (q, k, v)), None if s is None else
                       torch.from_numpy(s).cuda(), lay.table_gpu(), ints(lens), hq, hkv, D, D ** -0.5, ints(w), out,
                       n_sink=sink, workspace=ws)
    got, val = f64(out), values(v, s)
    for b in range(B):
        at = np.arange(lens[b] - tq, lens[b])
        want, size = attend_rows(q[b].astype(np.float64), at, lay.dense(k, b).astype(np.float64), lay.dense(val, b),
                                 D ** -0.5, w[b], sink, hkv)
        assert np.isfinite(got[b]).all()
        assert (np.abs(got[b] - want) <= attend_tolerance(size, max(lens[b], 1), 5.0)).all()
        assert (got[b][at < 0] == 0).all()
    assert binding.fa_decode_device_status() == 0


@pytest.mark.parametrize("seed", range(30))
def test_append(seed):
    rng = np.random.RandomState(3000 + seed)
    D = int(rng.choice([128, 256]))
    hkv = int(rng.choice([1, 2, 3, 8]))
    hq = int(rng.choice([0, 1, 4, 24, 40]))
    dtype = [torch.float16, torch.bfloat16, torch.float32][int(rng.randint(3))]
    B = int(rng.randint(1, 6))
    new = [int(x) for x in rng.randint(0, int(rng.choice([2, 20, 400])) + 1, B)]
    N = max(sum(new), 1)
    at = [int(x) for x in rng.randint(0, 60, B)]
    cap = max(a + n for a, n in zip(at, new)) + 1
    lay = Layout(B, hkv, cap, bool(rng.rand() < 0.6), page=int(rng.choice([16, 48])), seed=seed)
    rot = 16 * int(rng.randint(0, D // 16 + 1))
    inter = bool(rng.rand() < 0.5)
    table, mag = fa.fa_rope_table(rot, 10000.0, scaling="linear", factor=3.0) if rot else (None, 1.0)
    rate = rates(rot, 10000.0, "linear", 3.0)[0] if rot else np.zeros(0)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, hq + 2 * hkv, D, generator=g).to(dtype).cuda()
    qw, kw = ((torch.rand(D, generator=g) + 0.5).to(dtype).cuda() if rng.rand() < 0.5 else None for _ in range(2))
    kc, vc = (torch.full((*lay.rows, D), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    qo = torch.full((N, hq, D), 9.0, dtype=torch.float16, device="cuda") if hq else None
    rope_at = [int(x) for x in rng.randint(0, 1 << 20, B)]
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    fa.fa_rope_append_kv(q if hq else None, k, v, qo, kc, vc, None, lay.table_gpu(), ints(starts), ints(at), table,
                         q_weight=qw, k_weight=kw, eps=1e-5, interleaved=inter, magnitude=mag,
                         rope_positions=ints(rope_at))
    pos = np.concatenate([np.arange(n) + r for n, r in zip(new, rope_at)] + [np.zeros(0)])
    n = sum(new)
    for b, (m, a) in enumerate(zip(new, at)):
        rows = slice(starts[b], starts[b] + m)
        for src, cache, w in ((k, kc, kw), (v, vc, None)):
            if src is k:
                want, size = turn(f64(src[rows]), pos[rows], rate, mag, None if w is None else f64(w), 1e-5, inter)
            else:
                want, size = f64(src[rows]), np.zeros((m, hkv, D))
            got = np.moveaxis(lay.dense(f64(cache), b)[:, a:a + m], 0, 1)
            assert (np.abs(got - want) <= turn_tolerance(want, size, torch.float16)).all()
    assert int((kc != 7.0).any(-1).sum()) == n * hkv
    if hq:
        want, size = turn(f64(q[:n]), pos[:n], rate, mag, None if qw is None else f64(qw), 1e-5, inter)
        assert (np.abs(f64(qo[:n]) - want) <= turn_tolerance(want, size, torch.float16)).all()
        assert bool((qo[n:] == 9.0).all())
    assert binding.fa_decode_device_status() == 0
