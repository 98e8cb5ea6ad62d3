"""Recorded weights on fp16 and int8-V caches, eviction bit for bit, and the operators
together as a served batch uses them."""
import numpy as np
import pytest
import torch

import oracle
from decode_step_kv_gb300 import binding as fa

from _cache_ops import (Int4Cache, Layout, acc_tolerance, attend, cuda, evict, lens_gpu,
                        out_tolerance, pack, quantize, queries)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ recorded weights
class Cache:
    """fp16 K and fp16 or int8 V; rows behind the lengths hold NaN."""

    def __init__(self, lay, D, lens, int8, seed=0):
        r = np.random.RandomState(seed)
        used = lay.used(lens)
        self.lay, self.D, self.int8 = lay, D, int8
        self.k = r.standard_normal((*lay.rows, D)).astype(np.float16)
        v = r.standard_normal((*lay.rows, D)).astype(np.float32)
        self.vs = None
        if int8:
            self.v, s = oracle.pack_v_int8(v)
            self.vs = s.view(np.float16).copy()
            self.vs[~used] = np.nan
        else:
            self.v = v.astype(np.float16)
            self.v[~used] = np.nan
        self.k[~used] = np.nan

    def key(self, b):
        return self.lay.dense(self.k, b).astype(np.float64)

    def value(self, b):
        v = self.lay.dense(self.v, b).astype(np.float64)
        if self.int8:
            v = v * np.repeat(self.lay.dense(self.vs, b).astype(np.float64), 32, -1)
        return v

    def gpu(self):
        return cuda(self.k), cuda(self.v), None if self.vs is None else cuda(self.vs)


def weigh(lay, cache, q, lens, Hq, scale, window, acc):
    B, tq, _, D = q.shape
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_weights(B, tq, Hq, lay.hkv, D, lay.cap)
    ws.fill_(0xFF)
    k, v, vs = cache.gpu()
    fa.fa_decode_weights(cuda(q), k, v, vs, lay.table_gpu(), lens_gpu(lens), Hq, lay.hkv, D, scale,
                         None if window is None else lens_gpu(window), out, acc, workspace=ws)
    return out


def check(lay, cache, q, lens, Hq, scale, window=None):
    D = q.shape[3]
    want, absum, size, wt = attend(q, cache.key, cache.value, lens, lay, scale, window)
    before = np.random.RandomState(9).random_sample(lay.rows).astype(np.float32)
    acc = cuda(before)
    got = weigh(lay, cache, q, lens, Hq, scale, window, acc).cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    # P is rounded to fp16, and code * scale of int8 V, as P * scale of the 4-bit cache; a
    # weight below 2^-14 is off by up to 2^-25, over at most cap keys of |v| at most vmax
    vmax = max((np.nanmax(np.abs(cache.value(b)[:, :max(n, 0)])) for b, n in enumerate(lens) if n > 0),
               default=0.0)
    over = np.abs(got - want) - out_tolerance(want, absum, size, D) - lay.cap * 2.0 ** -25 * vmax
    assert over.max() <= 0, f"out: {over.max():.3e} over its bound"
    after = acc.cpu().numpy().astype(np.float64)
    full, tol = before.astype(np.float64), np.zeros(lay.rows)
    for b in range(lay.batch):
        base = lay.dense(before.astype(np.float64), b)
        lay.put(full, b, base + wt[b])
        lay.put(tol, b, np.where(wt[b] > 0, acc_tolerance(base, wt[b], size, D,
                                                          q.shape[1] * Hq // lay.hkv), 0.0))
    over = np.abs(after - full) - tol
    assert over.max() <= 0, f"acc: {over.max():.3e} over its bound"


LENS = [0, 1, 15, 16, 17, 100, 333]


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("tq,Hq,Hkv,windowed", [(1, 2, 2, False), (1, 6, 2, True), (1, 12, 1, False),
                                                (3, 8, 2, True), (33, 2, 1, False)])
def test_weights(D, int8, paged, tq, Hq, Hkv, windowed):
    lay = Layout(len(LENS), Hkv, 336, paged, seed=tq)
    window = [0, 1, 3, 16, 5, 50, 200] if windowed else None
    check(lay, Cache(lay, D, LENS, int8, seed=Hq), queries(len(LENS), tq, Hq, D, 1), LENS, Hq,
          D ** -0.5, window)


@pytest.mark.parametrize("int8", [False, True])
def test_weights_of_a_long_batch(int8):
    lens = [9000, 4097, 1, 700]
    lay = Layout(4, 4, 9008, True)
    check(lay, Cache(lay, 128, lens, int8, seed=1), queries(4, 1, 16, 128, 4), lens, 16, 128 ** -0.5)


def test_weights_of_shared_blocks_add_up():
    """Two sequences whose tables name the same blocks: both add to their rows."""
    lay = Layout(2, 2, 64, True, seed=2)
    lay.table[1] = lay.table[0]
    cache = Cache(lay, 128, [64, 64], False, seed=2)
    q = queries(2, 1, 4, 128, 2)
    acc = torch.zeros(lay.rows, device="cuda")
    weigh(lay, cache, q, [64, 40], 4, 0.1, None, acc)
    _, _, size, wt = attend(q, cache.key, cache.value, [64, 40], lay, 0.1)
    got = lay.dense(acc.cpu().numpy(), 0)
    assert np.all(np.abs(got - wt[0] - wt[1]) <= acc_tolerance(0, wt[0] + wt[1], size, 128, 5))


def test_weights_in_a_graph():
    lay = Layout(2, 2, 208, True, seed=3)
    cache = Cache(lay, 128, [208, 208], False, seed=3)
    q = queries(2, 1, 8, 128, 3)
    k, v, _ = cache.gpu()
    qd, table, ln = cuda(q), lay.table_gpu(), lens_gpu([200, 77])
    out, acc = torch.empty_like(qd), torch.zeros(lay.rows, device="cuda")
    ws = fa.alloc_workspace_weights(2, 1, 8, 2, 128, lay.cap)

    def step():
        fa.fa_decode_weights(qd, k, v, None, table, ln, 8, 2, 128, 0.1, None, out, acc, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
        step()
    for n in (5, 208):
        ln.copy_(lens_gpu([n, 77]))
        acc.zero_()
        step()
        once, o = acc.clone(), out.clone()
        acc.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(acc, once + once)


# ------------------------------------------------------------------ eviction
KINDS = ["fp16", "int8v", "int4"]


def arrays_of(kind, lay, D, seed):
    """Random bytes in the cache's types: K, V, K scales, V scales (None where absent)."""
    r = np.random.RandomState(seed)

    def fill(n, dtype):
        return r.randint(0, 256, (*lay.rows, n * np.dtype(dtype).itemsize)).astype(np.uint8).view(dtype)

    if kind == "int4":
        return [fill(D // 2, np.uint8), fill(D // 2, np.uint8), fill(D // 32, np.float16),
                fill(D // 32, np.float16)]
    if kind == "int8v":
        return [fill(D, np.float16), fill(D, np.int8), None, fill(D // 32, np.float16)]
    return [fill(D, np.float16), fill(D, np.float16), None, None]


def totals(lay, seed, kind="heavy"):
    r = np.random.RandomState(seed)
    a = r.random_sample(lay.rows).astype(np.float32)
    if kind == "heavy":
        a = np.where(a < 0.2, 0.0, a ** 8 * 50).astype(np.float32)
    elif kind == "ties":
        a = np.floor(a * 4).astype(np.float32)
    elif kind == "odd":
        a = (a - 0.5).astype(np.float32)
        special = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, 1e-42, -1e-42, 3e38], np.float32)
        pick = r.randint(0, 16, lay.rows)
        a = np.where(pick < 8, special[pick % 8], a).astype(np.float32)
    return a


def check_evict(kind, lay, D, lens, budget, sink, recent, acc, seed=0):
    arr = arrays_of(kind, lay, D, seed)
    have = [a for a in arr if a is not None]
    new, want_acc, want_kept, want_lens = evict([a.view(np.uint8) for a in have], acc, lay, lens,
                                                budget, sink, recent)
    g = [None if a is None else cuda(a) for a in arr]
    accd = cuda(acc)
    nl = torch.full((lay.batch,), -7, dtype=torch.int32, device="cuda")
    kept = torch.full((lay.batch, lay.hkv, budget), -9, dtype=torch.int32, device="cuda")
    fa.fa_evict_kv(g[0], g[1], accd, lay.table_gpu(), lens_gpu(lens), nl, budget=budget, n_sink=sink,
                   n_recent=recent, kept=kept, k_scales=g[2], v_scales=g[3])
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(nl.cpu().numpy(), want_lens)
    assert np.array_equal(accd.cpu().numpy().view(np.uint32), want_acc.view(np.uint32))
    for a, b in zip([x for x in g if x is not None], new):
        assert np.array_equal(a.cpu().numpy().view(np.uint8), b)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("paged,page", [(False, 16), (True, 16), (True, 48)])
def test_evict(kind, D, paged, page):
    lens = [0, 1, 31, 32, 33, 100, 500]
    lay = Layout(len(lens), 2, 528, paged, page, seed=D)
    check_evict(kind, lay, D, lens, 32, 4, 8, totals(lay, 1))


@pytest.mark.parametrize("how", ["heavy", "ties", "odd"])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (50, 0, 0), (50, 50, 0),
                                                (50, 0, 50), (50, 20, 30), (299, 3, 5), (300, 3, 5)])
def test_evict_budgets_and_ties(how, budget, sink, recent):
    lens = [300, 299, 57]
    lay = Layout(3, 3, 304, True, seed=budget)
    check_evict("fp16", lay, 128, lens, budget, sink, recent, totals(lay, budget, how))


@pytest.mark.parametrize("kind", KINDS)
def test_evict_many_rounds(kind):
    """More kept rows than a cluster stages at a time, most of them moving."""
    lens = [20011]
    lay = Layout(1, 1, 20016, True, seed=1)
    check_evict(kind, lay, 256, lens, 15000, 4, 100, totals(lay, 3))


@pytest.mark.parametrize("B", [40, 170])
def test_evict_many_units(B):
    lens = [(61 * b) % 900 for b in range(B)]
    lay = Layout(B, 2, 912, True, seed=B)
    check_evict("fp16", lay, 128, lens, 250, 1, 16, totals(lay, B, "ties"))


def test_evict_flags():
    lay = Layout(2, 1, 64, True, seed=1)
    acc = totals(lay, 1)
    fa.fa_decode_device_status()
    check_evict("fp16", lay, 128, [10 ** 6, -5], 20, 2, 2, acc)
    assert fa.fa_decode_device_status() == fa.FA_STATUS_LEN_CLAMPED
    # tokens of an unmapped block lose to every total and nothing of them moves
    table = lay.table.copy()
    lay.table[0, 1] = -1
    k = torch.zeros((*lay.rows, 128), dtype=torch.float16, device="cuda")
    kept = torch.empty((2, 1, 20), dtype=torch.int32, device="cuda")
    nl = torch.empty(2, dtype=torch.int32, device="cuda")
    accd = torch.ones(lay.rows, device="cuda")
    fa.fa_evict_kv(k, k.clone(), accd, lay.table_gpu(), lens_gpu([64, 3]), nl, budget=20, n_sink=2,
                   n_recent=2, kept=kept)
    assert fa.fa_decode_device_status() == fa.FA_STATUS_BAD_BLOCK
    assert kept[0, 0].tolist() == list(range(16)) + [32, 33] + [62, 63]
    assert kept[1, 0].tolist() == [0, 1, 2] + [-1] * 17 and nl.tolist() == [20, 3]
    lay.table = table


def test_evict_in_a_graph_on_a_side_stream():
    lay = Layout(3, 2, 400, True, seed=4)
    lens = [400, 90, 333]
    arr = arrays_of("int8v", lay, 128, 5)
    acc = totals(lay, 7)
    start = [cuda(a) for a in (arr[0], arr[1], arr[3], acc)]
    work = [a.clone() for a in start]
    nl = torch.empty(3, dtype=torch.int32, device="cuda")
    kept = torch.empty((3, 2, 64), dtype=torch.int32, device="cuda")
    table, ln = lay.table_gpu(), lens_gpu(lens)

    def step():
        fa.fa_evict_kv(work[0], work[1], work[3], table, ln, nl, budget=64, n_sink=4, n_recent=9,
                       kept=kept, v_scales=work[2])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    once = [a.clone() for a in work] + [nl.clone(), kept.clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for a, b in zip(work, start):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(work + [nl, kept], once):
        assert np.array_equal(a.cpu().numpy().view(np.uint8), b.cpu().numpy().view(np.uint8))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("kind", ["fp16", "int4"])
def test_served_batch(kind):
    """A prompt's chunk, decode steps that record weights, an eviction, further steps: every
    output against fp64 on a mirror of the cache."""
    B, H, Hq, D, budget = 3, 2, 8, 128, 40
    lay = Layout(B, H, 128, True, seed=11)
    r = np.random.RandomState(12)
    lens = np.array([60, 33, 90])
    T = int(lens.max())
    kn, vn = (r.standard_normal((B, T, H, D)).astype(np.float32) for _ in range(2))
    mirror = [np.zeros((B, H, lay.cap, D)) for _ in range(2)]

    def stored(x):
        if kind == "int4":
            c, s = quantize(x)
            return c * np.repeat(s.astype(np.float64), 32, -1)
        return x.astype(np.float16).astype(np.float64)

    def mirror_put(new, pos, count):
        for m, x in zip(mirror, new):
            val = stored(x)
            for b in range(B):
                m[b, :, pos[b]:pos[b] + count[b]] = np.moveaxis(val[b, :count[b]], 0, 1)

    table = lay.table_gpu()
    if kind == "int4":
        c = [torch.zeros((*lay.rows, n), dtype=t, device="cuda")
             for n, t in ((64, torch.uint8), (4, torch.float16)) * 2]
        fa.fa_append_kv_int4(cuda(kn), cuda(vn), *c, table, lens_gpu([0] * B), n_new=lens_gpu(lens))
    else:
        c = [torch.zeros((*lay.rows, D), dtype=torch.float16, device="cuda") for _ in range(2)]
        for i in range(T):
            pos = lens_gpu([i if i < n else -1 for n in lens])
            fa.fa_append_kv(cuda(kn[:, i]), cuda(vn[:, i]), *c, None, table, pos, n_kv_heads=H,
                            head_dim=D)
        fa.fa_decode_device_status()              # the short sequences' skipped rows
    mirror_put((kn, vn), [0] * B, lens)
    acc = torch.zeros(lay.rows, device="cuda")
    model = np.zeros((B, H, lay.cap))
    ws = (fa.alloc_workspace_int4(B, 1, Hq, H, D, lay.cap, weights=True) if kind == "int4"
          else fa.alloc_workspace_weights(B, 1, Hq, H, D, lay.cap))
    dense = Layout(B, H, lay.cap, False)

    for step in range(12):
        if step == 6:
            nl = torch.empty(B, dtype=torch.int32, device="cuda")
            kept = torch.empty((B, H, budget), dtype=torch.int32, device="cuda")
            kw = {"k_scales": c[1], "v_scales": c[3]} if kind == "int4" else {}
            fa.fa_evict_kv(c[0], c[2] if kind == "int4" else c[1], acc, table, lens_gpu(lens), nl,
                           budget=budget, n_sink=2, n_recent=8, kept=kept, **kw)
            ids = kept.cpu().numpy()
            got = np.stack([lay.dense(acc.cpu().numpy(), b) for b in range(B)])
            for b in range(B):
                if lens[b] <= budget:
                    continue
                for h in range(H):
                    # the kernel's totals and the model's may order near ties differently,
                    # so the model follows the kernel's choice and checks its quality
                    out = np.setdiff1d(np.arange(2, lens[b] - 8), ids[b, h])
                    mid = ids[b, h][(ids[b, h] >= 2) & (ids[b, h] < lens[b] - 8)]
                    assert model[b, h, mid].min() >= model[b, h, out].max() - 1e-4
                    assert np.array_equal(ids[b, h, :2], [0, 1])
                    assert np.array_equal(ids[b, h, -8:], np.arange(lens[b] - 8, lens[b]))
                    for m in mirror:
                        m[b, h, :budget] = m[b, h, ids[b, h]]
                    model[b, h, :budget] = model[b, h, ids[b, h]]
                    model[b, h, budget:] = 0
            assert np.all(np.abs(got - model) <= 1e-4 * (1 + model))
            lens = np.minimum(lens, budget)
            assert np.array_equal(nl.cpu().numpy(), lens)
        kn, vn = (r.standard_normal((B, 1, H, D)).astype(np.float32) for _ in range(2))
        if kind == "int4":
            fa.fa_append_kv_int4(cuda(kn), cuda(vn), *c, table, lens_gpu(lens))
        else:
            fa.fa_append_kv(cuda(kn[:, 0]), cuda(vn[:, 0]), *c, None, table, lens_gpu(lens),
                            n_kv_heads=H, head_dim=D)
        mirror_put((kn, vn), lens, [1] * B)
        lens = lens + 1
        q = queries(B, 1, Hq, D, 100 + step)
        want, absum, size, wt = attend(q, lambda b: mirror[0][b], lambda b: mirror[1][b], lens, dense,
                                       D ** -0.5)
        out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
        if kind == "int4":
            fa.fa_decode_int4(cuda(q), *c, table, lens_gpu(lens), Hq, H, D, D ** -0.5, None, out,
                              acc=acc, workspace=ws)
        else:
            fa.fa_decode_weights(cuda(q), *c, None, table, lens_gpu(lens), Hq, H, D, D ** -0.5, None,
                                 out, acc, workspace=ws)
        over = np.abs(out.cpu().numpy() - want) - out_tolerance(want, absum, size, D, lay.cap, 1.0)
        assert over.max() <= 0
        for b in range(B):
            model[b] += wt[b]
    assert fa.fa_decode_device_status() == 0
    assert pack(quantize(np.zeros((1, D)))[0]).tolist() == [[0x88] * (D // 2)]


def test_evict_then_decode_reads_the_kept_rows():
    """After the eviction, decode attention over the first budget rows equals attention over
    the kept tokens of the old cache."""
    lens = [150, 80]
    lay = Layout(2, 2, 160, True, seed=8)
    cache = Int4Cache(lay, 128, lens, seed=8)
    acc = totals(lay, 3)
    c = cache.gpu()
    nl = torch.empty(2, dtype=torch.int32, device="cuda")
    kept = torch.empty((2, 2, 64), dtype=torch.int32, device="cuda")
    fa.fa_evict_kv(c[0], c[2], cuda(acc), lay.table_gpu(), lens_gpu(lens), nl, budget=64, n_sink=4,
                   n_recent=16, kept=kept, k_scales=c[1], v_scales=c[3])
    ids = kept.cpu().numpy()
    k = [np.stack([cache.key(b)[h, ids[b, h]] for h in range(2)]) for b in range(2)]
    v = [np.stack([cache.value(b)[h, ids[b, h]] for h in range(2)]) for b in range(2)]
    q = queries(2, 1, 8, 128, 8)
    want, absum, size, _ = attend(q, lambda b: k[b], lambda b: v[b], [64, 64],
                                  Layout(2, 2, 64, False), 0.1)
    out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_int4(2, 1, 8, 2, 128, lay.cap)
    fa.fa_decode_int4(cuda(q), *c, lay.table_gpu(), nl, 8, 2, 128, 0.1, None, out, workspace=ws)
    assert np.all(np.abs(out.cpu().numpy() - want) <= cache.tolerance(want, absum, size))
