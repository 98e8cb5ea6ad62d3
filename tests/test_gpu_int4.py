"""4-bit cache: append and gather bit for bit, decode attention against fp64."""
import numpy as np
import pytest
import torch

from decode_step_kv_gb300 import binding as fa

from _cache_ops import (Int4Cache, Layout, acc_tolerance, attend, cuda, dequantize, lens_gpu,
                        pack, quantize, queries)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append, gather
def rows_for_codec(B, T, H, D, seed):
    """Rows with the codec's hard values: ties, tiny, huge, infinities, NaN, zero blocks."""
    r = np.random.RandomState(seed)
    x = r.standard_normal((B, T, H, D)).astype(np.float32)
    f = x.reshape(-1, 32)
    f[0] = 0.0
    f[1 % len(f)] = np.linspace(-7, 7, 32)                       # scale 1: ties at every half
    f[1 % len(f), :16] = np.arange(16) - 7.5
    f[1 % len(f), 31] = 7.0
    if len(f) > 8:
        f[2] *= 1e-9
        f[3] *= 3e-7
        f[4] = [1e6 * (-1) ** i / (i + 1) for i in range(32)]
        f[5, 3], f[5, 4], f[5, 5] = np.inf, -np.inf, np.nan
        f[6, ::2] = -0.0
        f[7] = np.nan
    return x


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("paged,page", [(False, 16), (True, 16), (True, 48)])
@pytest.mark.parametrize("B,T,H", [(3, 1, 2), (1, 1, 1), (2, 37, 3)])
def test_append_and_gather(D, paged, page, B, T, H):
    lay = Layout(B, H, 96, paged, page, seed=D)
    kn, vn = rows_for_codec(B, T, H, D, 1), rows_for_codec(B, T, H, D, 2)
    pos = [(5 * b + 11) % 59 for b in range(B)]
    start = np.random.RandomState(3).randint(0, 256, (*lay.rows, D // 2)).astype(np.uint8)
    want, got = [], []
    c = [cuda(start), torch.full((*lay.rows, D // 32), 3.0, dtype=torch.float16, device="cuda"),
         cuda(start), torch.full((*lay.rows, D // 32), 3.0, dtype=torch.float16, device="cuda")]
    fa.fa_append_kv_int4(cuda(kn), cuda(vn), *c, lay.table_gpu(), lens_gpu(pos))
    for i, x in enumerate((kn, vn)):
        codes, s = quantize(x)
        by, sc = start.copy(), np.full((*lay.rows, D // 32), 3.0, dtype=np.float16)
        for b in range(B):
            d, e = lay.dense(by, b).copy(), lay.dense(sc, b).copy()
            d[:, pos[b]:pos[b] + T] = np.moveaxis(pack(codes[b]), 0, 1)
            e[:, pos[b]:pos[b] + T] = np.moveaxis(s[b], 0, 1)
            lay.put(by, b, d)
            lay.put(sc, b, e)
        assert np.array_equal(c[2 * i + 1].cpu().numpy().view(np.uint16), sc.view(np.uint16))
        assert np.array_equal(c[2 * i].cpu().numpy(), by)
        with np.errstate(over="ignore"):            # beyond fp16 the value reads as infinity
            want.append((codes * np.repeat(s.astype(np.float64), 32, -1)).astype(np.float16))
        got.append(torch.full((B, T, H, D), 9.0, dtype=torch.float16, device="cuda"))
    fa.fa_gather_kv_int4(*c, lay.table_gpu(), lens_gpu(pos), *got)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert fa.fa_decode_device_status() == 0


def test_append_padded_batch_and_out_of_range():
    """Rows behind n_new, tokens outside the cache and unmapped blocks are not stored."""
    lay = Layout(4, 2, 64, True, 16, seed=5)
    lay.table[3, 1] = 10 ** 6
    x = np.random.RandomState(0).standard_normal((4, 6, 2, 128)).astype(np.float32)
    c = [torch.full((*lay.rows, 64), 0x5a, dtype=torch.uint8, device="cuda"),
         torch.full((*lay.rows, 4), 2.0, dtype=torch.float16, device="cuda")]
    c += [t.clone() for t in c]
    fa.fa_decode_device_status()
    n_new, pos = [2, 0, 6, 6], [3, 8, 61, 14]                # row 2 runs out of the cache
    fa.fa_append_kv_int4(cuda(x), cuda(x), *c, lay.table_gpu(), lens_gpu(pos),
                         n_new=lens_gpu(n_new))
    assert fa.fa_decode_device_status() == fa.FA_STATUS_POS_RANGE | fa.FA_STATUS_BAD_BLOCK
    codes, s = quantize(x)
    by = np.full((*lay.rows, 64), 0x5a, dtype=np.uint8)
    sc = np.full((*lay.rows, 4), 2.0, dtype=np.float16)
    packed = pack(codes)
    for b in range(4):
        for i in range(n_new[b]):
            t = pos[b] + i
            if t >= 64 or lay.table[b, t // 16] == 10 ** 6:
                continue
            by[lay.table[b, t // 16], :, t % 16] = packed[b, i]
            sc[lay.table[b, t // 16], :, t % 16] = s[b, i]
    for i in (0, 2):
        assert np.array_equal(c[i].cpu().numpy(), by)
        assert np.array_equal(c[i + 1].cpu().numpy(), sc)
    out = [torch.full((4, 6, 2, 128), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    fa.fa_gather_kv_int4(*c, lay.table_gpu(), lens_gpu([3, 8, 61, -1]), *out,
                         n_rows=lens_gpu([2, 0, 4, 1]))
    assert fa.fa_decode_device_status() == fa.FA_STATUS_POS_RANGE
    got = out[0].cpu().numpy()
    val = (codes * np.repeat(s.astype(np.float64), 32, -1)).astype(np.float16)
    assert np.array_equal(got[0, :2], val[0, :2]) and np.all(got[0, 2:] == 7) and np.all(got[1] == 7)
    assert np.array_equal(got[2, :3], val[2, :3]) and np.all(got[2, 3] == 0) and np.all(got[2, 4:] == 7)
    assert np.all(got[3, 0] == 0) and np.all(got[3, 1:] == 7)
    assert torch.equal(out[0], out[1])


# ------------------------------------------------------------------ attention
def run(lay, cache, q, lens, Hq, scale, window=None, acc=None, stream=None, ws=None):
    B, tq, _, D = q.shape
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    if ws is None:
        ws = fa.alloc_workspace_int4(B, tq, Hq, lay.hkv, D, lay.capacity, weights=acc is not None)
        ws.fill_(0xFF)
    fa.fa_decode_int4(cuda(q), *cache.gpu(), lay.table_gpu(), lens_gpu(lens), Hq, lay.hkv, D, scale,
                      None if window is None else lens_gpu(window), out, acc=acc, workspace=ws,
                      stream=stream)
    return out


def check(lay, cache, q, lens, Hq, scale, window=None, weights=True):
    D = q.shape[3]
    want, absum, size, wt = attend(q, cache.key, cache.value, lens, lay, scale, window)
    got = run(lay, cache, q, lens, Hq, scale, window).cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    over = np.abs(got - want) - cache.tolerance(want, absum, size)
    assert over.max() <= 0, f"out: {over.max():.3e} over its bound"
    if not weights:
        return
    before = np.random.RandomState(9).random_sample(lay.rows).astype(np.float32)
    acc = cuda(before)
    # with acc another plan may serve the call: held to the same derived bound
    got2 = run(lay, cache, q, lens, Hq, scale, window, acc=acc).cpu().numpy().astype(np.float64)
    assert (np.abs(got2 - want) - cache.tolerance(want, absum, size)).max() <= 0
    after = acc.cpu().numpy().astype(np.float64)
    cols = q.shape[1] * Hq // lay.hkv
    full = before.astype(np.float64)
    tol = np.zeros(lay.rows)
    for b in range(lay.batch):
        base = lay.dense(before.astype(np.float64), b)
        lay.put(full, b, base + wt[b])
        lay.put(tol, b, np.where(wt[b] > 0, acc_tolerance(base, wt[b], size, D, cols), 0.0))
    over = np.abs(after - full) - tol
    assert over.max() <= 0, f"acc: {over.max():.3e} over its bound"


LENS = [0, 1, 15, 16, 17, 100, 333]


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("paged,page", [(False, 16), (True, 16), (True, 48)])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (6, 2), (8, 1), (12, 1)])
def test_decode(D, paged, page, Hq, Hkv):
    lay = Layout(len(LENS), Hkv, 336, paged, page, seed=D + Hq)
    cache = Int4Cache(lay, D, LENS, seed=Hq)
    check(lay, cache, queries(len(LENS), 1, Hq, D, 1), LENS, Hq, D ** -0.5)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("tq,Hq,Hkv", [(2, 4, 2), (3, 3, 1), (5, 16, 2), (40, 4, 2)])
@pytest.mark.parametrize("windowed", [False, True])
def test_several_queries(D, tq, Hq, Hkv, windowed):
    lay = Layout(len(LENS), Hkv, 352, True, 16, seed=tq)
    cache = Int4Cache(lay, D, LENS, seed=tq)
    window = [0, 1, 3, 16, 5, 50, 200] if windowed else None
    check(lay, cache, queries(len(LENS), tq, Hq, D, tq), LENS, Hq, D ** -0.5, window)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("tq,Hq,Hkv", [(16, 1, 1), (17, 1, 1), (3, 16, 2), (31, 2, 2), (8, 8, 2), (11, 3, 1),
                                       (21, 3, 1), (16, 8, 2), (13, 20, 4), (26, 5, 1), (256, 1, 1)])
def test_many_columns(D, tq, Hq, Hkv):
    """Around and beyond 16, 32 and 64 (query, head) columns per KV head."""
    lens = [700, 3, 65, 64, 0, 290]
    lay = Layout(len(lens), Hkv, 704, True, 16, seed=tq)
    window = [0, 2, 20, 0, 5, 33] if tq % 2 else None
    check(lay, Int4Cache(lay, D, lens, seed=Hq), queries(len(lens), tq, Hq, D, tq), lens, Hq, D ** -0.5,
          window)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("paged,page", [(False, 16), (True, 16), (True, 80)])
def test_many_columns_layouts_and_magnitudes(D, paged, page):
    """Long enough to be split over workers; V from tiny to large along the sequence."""
    lens = [3000, 1111, 16, 2999]
    lay = Layout(4, 2, 3040, paged, page, seed=1)
    ramp = np.ones((*lay.rows, 1))
    for b, n in enumerate(lens):
        d = np.ones((2, lay.cap, 1))
        d[:, :n, 0] = 2.0 ** np.linspace(-20 + 4 * b, 12, n)
        lay.put(ramp, b, d)
    cache = Int4Cache(lay, D, lens, seed=2, v_mag=ramp)
    for tq, Hq in ((5, 8), (12, 8)):
        check(lay, cache, queries(4, tq, Hq, D, tq, mag=1.5), lens, Hq, D ** -0.5)


@pytest.mark.parametrize("tq,Hq,windowed", [(3, 6, False), (4, 8, True), (5, 16, False), (12, 2, True)])
def test_two_column_groups(tq, Hq, windowed):
    """Enough capacity that units of 16 columns are taken (9 to 40 columns, head_dim 128)."""
    lens = [2000, 17, 0, 999, 40, 16, 64]
    lay = Layout(7, 2, 2000, True, 16, seed=3, room=1 << 17)
    cache = Int4Cache(lay, 128, lens, seed=tq)
    window = [0, 5, 3, 77, 0, 33, 1] if windowed else None
    check(lay, cache, queries(7, tq, Hq, 128, tq), lens, Hq, 0.1, window)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_many_columns_scales(scale):
    lens = [300, 19]
    lay = Layout(2, 2, 304, False)
    check(lay, Int4Cache(lay, 128, lens, seed=8), queries(2, 7, 8, 128, 5), lens, 8, scale)


@pytest.mark.parametrize("tq,Hq", [(1, 4), (8, 8), (32, 4)])
def test_rows_outside_the_ranges_may_hold_anything(tq, Hq):
    """Rows before the window and in unmapped blocks: NaN scales, out-of-range ids."""
    lens = [200, 133]
    lay = Layout(2, 2, 208, True, seed=9)
    cache = Int4Cache(lay, 128, lens, seed=9)
    q = queries(2, tq, Hq, 128, 9)
    window = [40, 17]
    want, absum, size, _ = attend(q, cache.key, cache.value, lens, lay, 0.1, window)
    for b, (n, w) in enumerate(zip(lens, window)):
        first = n - tq + 1 - w                          # the first key any query attends
        for s in (cache.ks, cache.vs):
            d = lay.dense(s, b).copy()
            d[:, :first] = np.nan
            lay.put(s, b, d)
        lay.table[b, :first // 16] = 2 ** 30
        lay.table[b, -(-n // 16):] = -5
    fa.fa_decode_device_status()
    acc = torch.zeros(lay.rows, device="cuda")
    got = run(lay, cache, q, lens, Hq, 0.1, window, acc=acc).cpu().numpy()
    assert fa.fa_decode_device_status() == 0
    assert np.all(np.abs(got - want) <= cache.tolerance(want, absum, size))
    assert abs(float(acc.sum()) - 2 * tq * Hq) < 1e-3


@pytest.mark.parametrize("D", [128, 256])
def test_windows(D):
    lens = [400, 17, 64, 399, 1]
    lay = Layout(5, 2, 400, True, 16, seed=4)
    cache = Int4Cache(lay, D, lens, seed=4)
    for window in ([37, 17, 64, 1, 1], [16, 1, 63, 400, 5], [0, 16, 0, 33, 0]):
        # rows before the window may hold anything, NaN too
        other = Int4Cache(lay, D, lens, seed=4)
        for b, (n, w) in enumerate(zip(lens, window)):
            if 0 < w < n:
                for s in (other.ks, other.vs):
                    d = lay.dense(s, b).copy()
                    d[:, :n - w] = np.nan
                    lay.put(s, b, d)
        want, absum, size, _ = attend(queries(5, 1, 8, D, 2), cache.key, cache.value, lens, lay,
                                      D ** -0.5, window)
        got = run(lay, other, queries(5, 1, 8, D, 2), lens, 8, D ** -0.5, window)
        assert np.all(np.abs(got.cpu().numpy() - want) <= cache.tolerance(want, absum, size))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.3, 0.0884, 2.0])
def test_scales_of_the_softmax(D, scale):
    lens = [300, 19]
    lay = Layout(2, 2, 304, False)
    check(lay, Int4Cache(lay, D, lens, seed=8), queries(2, 1, 4, D, 5), lens, 4, scale)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("v_mag", [1e-6, 1e-4, 1e-3, 300.0, 6e4])
def test_value_magnitudes(D, v_mag):
    """V scales far from 1: carried by a power of two, so the error stays relative."""
    lens = [500, 33]
    lay = Layout(2, 2, 512, True)
    cache = Int4Cache(lay, D, lens, seed=3, v_mag=v_mag)
    q = queries(2, 1, 8, D, 3)
    want, absum, size, _ = attend(q, cache.key, cache.value, lens, lay, D ** -0.5)
    got = run(lay, cache, q, lens, 8, D ** -0.5).cpu().numpy().astype(np.float64)
    # below 2^-14 the output itself is a subnormal fp16, rounded to 2^-24 steps
    over = np.abs(got - want) - cache.tolerance(want, absum, size)
    assert over.max() <= 0


@pytest.mark.parametrize("D", [128, 256])
def test_magnitudes_that_grow_along_the_sequence(D):
    """Keys and values that grow token by token (the running maximum and the power of two
    move many times), and ones that start at zero."""
    lens = [640, 640]
    lay = Layout(2, 1, 640, False)
    ramp = np.ones((2, 1, 640, 1))
    ramp[0, 0, :, 0] = 2.0 ** np.linspace(-20, 12, 640)
    ramp[1, 0, :200, 0] = 0.0
    ramp[1, 0, 200:, 0] = 2.0 ** np.linspace(-18, 0, 440)
    cache = Int4Cache(lay, D, lens, seed=6, v_mag=ramp, k_mag=np.linspace(0.1, 3, 640).reshape(1, 1, -1, 1))
    check(lay, cache, queries(2, 1, 4, D, 6, mag=2.0), lens, 4, D ** -0.5)


def test_peaked_scores():
    """One key takes all the weight; scores reach hundreds."""
    lens = [513]
    lay = Layout(1, 1, 528, True)
    cache = Int4Cache(lay, 128, lens, seed=2, k_mag=8.0)
    check(lay, cache, queries(1, 1, 4, 128, 2, mag=6.0), lens, 4, 0.5)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("B,Hkv", [(1, 1), (3, 6), (19, 1), (37, 2), (38, 2), (39, 2)])
@pytest.mark.parametrize("G,tq,windowed", [(1, 1, False), (4, 1, True), (3, 3, True)])
def test_small_steps(D, B, Hkv, G, tq, windowed):
    """Clusters of 8, 4 and 2 CTAs per unit, and the first step too large for them; column groups."""
    lens = [(97 * b) % 130 if b else 128 for b in range(B)]
    lay = Layout(B, Hkv, 128, B % 2 == 1, 32, seed=B)
    window = [(b % 4) * 25 for b in range(B)] if windowed else None
    check(lay, Int4Cache(lay, D, lens, seed=G), queries(B, tq, G * Hkv, D, 1), lens, G * Hkv, D ** -0.5,
          window, weights=tq == 1 or G < 3)


@pytest.mark.parametrize("D,cap", [(128, 8192), (128, 8208), (256, 4096), (256, 4112)])
def test_cluster_and_split_plan_border(D, cap):
    lens = [cap, 1, cap - 1500]
    lay = Layout(3, 2, cap, True)
    check(lay, Int4Cache(lay, D, lens, seed=1), queries(3, 1, 8, D, 4), lens, 8, D ** -0.5, weights=False)


def test_small_step_in_a_graph():
    lens = [200, 0, 77]
    lay = Layout(3, 2, 208, False, seed=3)
    cache = Int4Cache(lay, 256, [208] * 3, seed=3)
    q = queries(3, 2, 8, 256, 3)
    dev, qd, ln, out = cache.gpu(), cuda(q), lens_gpu(lens), torch.empty((3, 2, 8, 256), dtype=torch.float16,
                                                                         device="cuda")
    ws = fa.alloc_workspace_int4(3, 2, 8, 2, 256, lay.cap)
    want = {n: run(lay, cache, q, [n, 0, 77], 8, 0.1) for n in (200, 3, 208)}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_decode_int4(qd, *dev, None, ln, 8, 2, 256, 0.1, None, out, workspace=ws)
    for n in (200, 3, 208):
        ln.copy_(lens_gpu([n, 0, 77]))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[n]) and torch.all(out[1] == 0)


@pytest.mark.parametrize("B", [33, 140, 300])
def test_many_sequences(B):
    lens = [(37 * b) % 70 for b in range(B)]
    lay = Layout(B, 1, 80, True)
    check(lay, Int4Cache(lay, 128, lens, seed=B), queries(B, 1, 4, 128, B), lens, 4, 0.1)


def test_long_sequences_split_over_the_gpu():
    lens = [9000, 4097, 1]
    lay = Layout(3, 4, 9008, True)
    check(lay, Int4Cache(lay, 128, lens, seed=1), queries(3, 1, 16, 128, 4), lens, 16, 128 ** -0.5)


@pytest.mark.parametrize("tq", [1, 9])
def test_bad_blocks_and_lengths_are_flagged(tq):
    lens = [64, 64]
    lay = Layout(2, 2, 64, True, seed=1)
    cache = Int4Cache(lay, 128, lens, seed=1)
    q = queries(2, tq, 4, 128, 1)
    fa.fa_decode_device_status()
    good = run(lay, cache, q, [64, 64], 4, 0.1)
    over = run(lay, cache, q, [10 ** 6, -3], 4, 0.1)
    assert fa.fa_decode_device_status() == fa.FA_STATUS_LEN_CLAMPED
    assert torch.equal(good[0], over[0]) and torch.all(over[1] == 0)
    lay.table[1, 2] = -1                            # tokens 32..47 of sequence 1 are unmapped
    acc = torch.zeros(lay.rows, device="cuda")
    got = run(lay, cache, q, [64, 64], 4, 0.1)
    assert fa.fa_decode_device_status() == fa.FA_STATUS_BAD_BLOCK
    assert torch.equal(got[0], good[0])
    run(lay, cache, q, [64, 64], 4, 0.1, acc=acc)        # another plan may serve it
    assert fa.fa_decode_device_status() == fa.FA_STATUS_BAD_BLOCK
    if tq == 1:
        keep = np.r_[0:32, 48:64]
        kb, vb = cache.key(1)[:, keep], cache.value(1)[:, keep]
        sub = Layout(1, 2, 48, False)
        want, absum, size, _ = attend(q[1:], lambda b: kb, lambda b: vb, [48], sub, 0.1)
        assert np.all(np.abs(got[1:].cpu().numpy() - want) <= cache.tolerance(want, absum, size))
    assert abs(float(acc.sum()) - 2 * 4 * tq) < 1e-3     # every (query, head) row sums to 1


def test_stream_graph_and_new_lengths():
    """On a side stream, and captured once and replayed with other lengths."""
    lens = [200, 77]
    lay = Layout(2, 2, 208, True, seed=3)
    cache = Int4Cache(lay, 128, [208, 208], seed=3)
    q = queries(2, 1, 8, 128, 3)
    alone = run(lay, cache, q, lens, 8, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(lay, cache, q, lens, 8, 0.1)
    side.synchronize()
    assert torch.equal(got, alone)
    want = {n: run(lay, cache, q, [n, 77], 8, 0.1, acc=torch.zeros(lay.rows, device="cuda"))
            for n in (200, 5, 208)}
    dev = cache.gpu()
    qd, table, ln = cuda(q), lay.table_gpu(), lens_gpu(lens)
    out = torch.empty_like(qd)
    acc = torch.zeros(lay.rows, device="cuda")
    ws = fa.alloc_workspace_int4(2, 1, 8, 2, 128, lay.cap, weights=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_decode_int4(qd, *dev, table, ln, 8, 2, 128, 0.1, None, out, acc=acc, workspace=ws)
    for n in (200, 5, 208):
        ln.copy_(lens_gpu([n, 77]))
        acc.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[n])
        assert abs(float(acc.sum()) - 16) < 1e-4


def test_three_dimensional_queries():
    lens = [50]
    lay = Layout(1, 2, 64, False)
    cache = Int4Cache(lay, 128, lens, seed=1)
    q = queries(1, 1, 4, 128, 1)
    want = run(lay, cache, q, lens, 4, 0.1)
    out = torch.empty((1, 4, 128), dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_int4(1, 1, 4, 2, 128, 64)
    fa.fa_decode_int4(cuda(q[:, 0]), *cache.gpu(), None, lens_gpu(lens), 4, 2, 128, 0.1, None, out,
                      workspace=ws)
    assert torch.equal(out, want[:, 0])


def test_gather_matches_what_attention_reads():
    """A query that selects one key returns that key's V row as fa_gather_kv_int4 reads it."""
    lens = [40]
    lay = Layout(1, 1, 48, True, seed=2)
    cache = Int4Cache(lay, 128, lens, seed=5)
    k, v = (torch.empty((1, 40, 1, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    fa.fa_gather_kv_int4(*cache.gpu(), lay.table_gpu(), lens_gpu([0]), k, v)
    assert np.array_equal(v[0, :, 0].cpu().numpy(),
                          dequantize(lay.dense(cache.v, 0), lay.dense(cache.vs, 0))[0, :40].astype(np.float16))
    q = k[0, 17, 0].cpu().numpy().reshape(1, 1, 1, 128)
    got = run(lay, cache, q, lens, 1, 5.0)
    assert np.all(np.abs(got[0, 0, 0].cpu().numpy() - v[0, 17, 0].cpu().numpy().astype(np.float64))
                  <= 3 * 2.0 ** -11 * np.abs(v[0, 17, 0].cpu().numpy().astype(np.float64)) + 2.0 ** -24)
