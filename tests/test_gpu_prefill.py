"""Attention of chunks over the cache, and decode with sinks, against 64-bit forms."""
import numpy as np
import pytest
import torch

import decode_step_kv_gb300 as fa
from decode_step_kv_gb300 import binding
from _cache_ops import Layout
from _step_ops import attend_rows, attend_tolerance, f64

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def visible(lay, lens, new, window, sink):
    """Cache rows that some query of its sequence sees, as a bool array of the rows' shape."""
    m = np.zeros(lay.rows, dtype=bool)
    for b, (n, q) in enumerate(zip(lens, new)):
        d = np.zeros((lay.hkv, lay.cap), dtype=bool)
        first = max(0, n - q - window[b] + 1) if window[b] else 0
        if q and n > 0:
            d[:, first:n] = True
            d[:, :min(sink, n)] = True
        lay.put(m, b, d | lay.dense(m, b))
    return m


def caches(lay, lens, new, window, sink, D, seed, int8=False):
    """K and V with NaN in every row that nothing may look at."""
    rng = np.random.RandomState(seed)
    live = visible(lay, lens, new, window, sink)[..., None]
    k = np.where(live, rng.randn(*lay.rows, D), np.nan).astype(np.float16)
    v = rng.randn(*lay.rows, D)
    if not int8:
        return k, np.where(live, v, np.nan).astype(np.float16), None
    s = np.where(live, 0.01 + 0.02 * rng.rand(*lay.rows, D // 32), np.nan).astype(np.float16)
    return k, np.clip(np.rint(v * 60), -127, 127).astype(np.int8), s


def values(v, s):
    return v.astype(np.float64) if s is None else v * np.repeat(s.astype(np.float64), 32, axis=-1)


def run_prefill(lay, lens, new, hq, D, window=None, sink=0, seed=0, scale=None, starts=None, tokens=None, table=None,
                int8=False):
    B = lay.batch
    w = window or [0] * B
    k, v, s = caches(lay, lens, new, w, sink, D, seed, int8=int8)
    val = values(v, s)
    if starts is None:
        starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    N = tokens or starts[-1]
    q = np.random.RandomState(seed + 1).randn(N, hq, D).astype(np.float16)
    out = torch.full((N, hq, D), 9.0, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_prefill(B, N, hq, lay.hkv, D, lay.capacity)
    ws.fill_(255)                                      # a NaN wherever it is read unwritten
    fa.fa_prefill(torch.from_numpy(q).cuda(), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(),
                  None if s is None else torch.from_numpy(s).cuda(), lay.table_gpu() if table is None else torch.from_numpy(table).cuda(), ints(starts), ints(lens), hq,
                  lay.hkv, D, scale or D ** -0.5,
                  ints(window) if window else None, out, n_sink=sink, workspace=ws)
    got = f64(out)
    rest = np.ones(N, dtype=bool)
    for b, n in enumerate(new):
        rows = slice(starts[b], starts[b] + n)
        rest[rows] = False
        at = np.arange(lens[b] - n, lens[b])
        kk = lay.dense(k, b).astype(np.float64)
        vv = lay.dense(val, b)
        want, size = attend_rows(q[rows].astype(np.float64), at, kk, vv, scale or D ** -0.5, w[b], sink, lay.hkv)
        # int8 V: one more rounding, of code * scale to fp16
        tol = attend_tolerance(size, max(lens[b], 1), 5.0) + (2.0 ** -11 * size if int8 else 0)
        err = np.abs(got[rows] - want)
        assert np.isfinite(got[rows]).all(), b
        assert (err <= tol).all(), (b, (err / tol).max(), np.argwhere(err > tol)[:4].tolist())
        assert (got[rows][at < 0] == 0).all()
    assert (got[rest] == 9.0).all()
    assert binding.fa_decode_device_status() == 0
    return out


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (8, 2), (3, 1), (14, 2), (16, 1)])
@pytest.mark.parametrize("paged,page", [(True, 16), (False, 16)])
def test_heads(D, hq, hkv, paged, page):
    run_prefill(Layout(3, hkv, 300, paged, page=page, seed=2), [300, 1, 129], [70, 1, 129], hq, D)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("new,lens", [([1], [1]), ([1], [128]), ([1], [129]), ([127], [127]), ([128], [128]),
                                      ([129], [129]), ([257], [300]), ([64], [640]), ([33], [1000]),
                                      ([1, 200, 0, 63], [500, 200, 70, 64])])
def test_lengths(D, new, lens):
    run_prefill(Layout(len(new), 2, max(lens), True, page=16, seed=1), lens, new, 8, D, seed=3)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (10, 2)])
@pytest.mark.parametrize("new,lens,window,sink", [
    ([600], [600], [0], 0), ([1100], [1700], [0], 0), ([513, 1, 700, 0], [513, 300, 701, 9], [0, 0, 0, 0], 0),
    ([650, 1000], [900, 1000], [100, 300], 5), ([900, 300], [500, 2000], [0, 0], 0)])
def test_clusters(D, hq, hkv, new, lens, window, sink):
    """Chunks long enough for two CTAs side by side on one KV head, ends in the first or the second."""
    run_prefill(Layout(len(new), hkv, max(lens), True, page=16, seed=12), lens, new, hq, D,
                window=window if any(window) else None, sink=sink, seed=4)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 256])
def test_pages(page):
    run_prefill(Layout(2, 2, 400, True, page=page, seed=5), [400, 333], [150, 20], 8, 128)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("hq,hkv,new,lens,window,sink,page", [
    (8, 2, [1], [1], [0], 0, 16), (8, 2, [70, 1, 129], [300, 1, 129], [0] * 3, 0, 16),
    (3, 1, [257, 0, 40], [700, 3, 41], [0] * 3, 0, 48), (8, 1, [700, 300], [900, 2000], [0, 0], 0, 16),
    (8, 1, [650, 1000], [900, 1000], [100, 300], 5, 64), (4, 2, [20, 90, 200], [700, 90, 513], [129, 0, 129], 40, 16),
    (16, 1, [9], [9001], [0], 0, 16), (4, 4, [64, 3], [40, 2], [0, 0], 0, 0), (8, 1, [600], [777], [0], 0, 0)])
def test_int8_v(D, hq, hkv, new, lens, window, sink, page):
    """V in codes and scales: paged (page > 0) or contiguous, one CTA per row tile or clusters of two."""
    run_prefill(Layout(len(new), hkv, max(lens), page > 0, page=page or 16, seed=13), lens, new, hq, D,
                window=window if any(window) else None, sink=sink, seed=5, int8=True)


@pytest.mark.parametrize("cap", [200, 333, 1])
def test_contiguous_of_any_capacity(cap):
    run_prefill(Layout(2, 2, cap, False), [cap, max(1, cap // 2)], [min(cap, 60), 1], 4, 128)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window,sink", [(1, 0), (5, 3), (64, 0), (100, 4), (128, 130), (300, 1), (129, 1000)])
def test_windows_and_sinks(D, window, sink):
    run_prefill(Layout(3, 2, 700, True, page=16, seed=6), [700, 90, 513], [40, 90, 200], 8, D,
                window=[window, 0, window], sink=sink)


@pytest.mark.parametrize("scale", [-0.09, 1e-20, 0.5])
def test_scale_of_any_sign(scale):
    run_prefill(Layout(2, 2, 200, True, page=16, seed=6), [200, 90], [40, 90], 8, 128, scale=scale)


def test_far_pages_may_be_unmapped():
    """Pages behind a window that hold no sink are not looked up; those beyond the length neither."""
    lay = Layout(2, 1, 900, True, page=16, seed=8)
    table = lay.table.copy()
    table[0, 1:42] = -1
    table[1, 20:] = 1 << 30
    run_prefill(lay, [900, 320], [20, 320], 4, 128, window=[200, 0], sink=16, table=table)


def test_a_block_that_is_not_mapped_is_skipped():
    """As in decode: its keys are left out and the status bit is set."""
    D, hq, hkv = 128, 4, 2
    lay = Layout(1, hkv, 200, True, page=16, seed=9)
    k, v, _ = caches(lay, [200], [50], [0], 0, D, 1)
    dense_k, dense_v = (lay.dense(x, 0).astype(np.float64) for x in (k, v))
    lay.table[0, 3] = -5
    q = np.random.RandomState(2).randn(50, hq, D).astype(np.float16)
    out = torch.empty(50, hq, D, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_prefill(1, 50, hq, hkv, D, lay.capacity)
    fa.fa_prefill(*(torch.from_numpy(x).cuda() for x in (q, k, v)), None, lay.table_gpu(),
                  ints([0, 50]), ints([200]), hq, hkv, D, D ** -0.5, None, out, workspace=ws)
    assert binding.fa_decode_device_status() == binding.FA_STATUS_BAD_BLOCK
    keep = np.r_[0:48, 64:200]
    want, size = attend_rows(q.astype(np.float64), np.arange(150, 200) - 16, dense_k[:, keep], dense_v[:, keep],
                             D ** -0.5, 0, 0, hkv)
    assert (np.abs(f64(out) - want) <= attend_tolerance(size, 200, 5.0)).all()


def test_rows_of_no_sequence_stay():
    run_prefill(Layout(3, 2, 100, True), [50, 0, 100], [20, 0, 30], 4, 128, starts=[3, 23, 23, 53], tokens=60)


def test_more_new_tokens_than_keys():
    """Rows at negative positions get zeros; a length of zero gives zeros."""
    run_prefill(Layout(3, 2, 100, True), [5, 0, 1], [20, 3, 300], 4, 128)


def test_lengths_are_clamped_and_flagged():
    lay = Layout(2, 1, 64, False)
    rng = np.random.RandomState(0)
    k, v = (rng.randn(*lay.rows, 128).astype(np.float16) for _ in range(2))
    q = rng.randn(6, 2, 128).astype(np.float16)
    out = torch.empty(6, 2, 128, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_prefill(2, 6, 2, 1, 128, 64)
    fa.fa_prefill(*(torch.from_numpy(x).cuda() for x in (q, k, v)), None, None, ints([0, 4, 6]), ints([70, -3]), 2, 1,
                  128, 0.1, None, out, workspace=ws)
    assert binding.fa_decode_device_status() == binding.FA_STATUS_LEN_CLAMPED
    want, size = attend_rows(q[:4].astype(np.float64), np.arange(60, 64), k[0].astype(np.float64),
                             v[0].astype(np.float64), 0.1, 0, 0, 1)
    assert (np.abs(f64(out)[:4] - want) <= attend_tolerance(size, 64, 5.0)).all()
    assert bool((out[4:] == 0).all())


@pytest.mark.parametrize("D", [128, 256])
def test_scores_that_grow_along_the_keys(D):
    """Scores over hundreds of units, rising with the key index (every tile a new maximum) and
    falling (none): the running maximum and the rescaling of what is summed already."""
    hq, hkv, L, n = 4, 1, 1500, 40
    lay = Layout(2, hkv, L, False)
    rng = np.random.RandomState(4)
    k = np.zeros((2, hkv, L, D), dtype=np.float16)
    k[0, 0, :, 0] = np.linspace(-40, 40, L)
    k[1, 0, :, 0] = np.linspace(40, -40, L)
    k[..., 1:] = rng.randn(2, hkv, L, D - 1) * 0.1
    v = rng.randn(2, hkv, L, D).astype(np.float16)
    q = rng.randn(2 * n, hq, D).astype(np.float16)
    q[..., 0] = rng.choice([4.0, -4.0, 0.25], size=(2 * n, hq))
    out = torch.empty(2 * n, hq, D, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_prefill(2, 2 * n, hq, hkv, D, L)
    fa.fa_prefill(*(torch.from_numpy(x).cuda() for x in (q, k, v)), None, None, ints([0, n, 2 * n]), ints([L, L]), hq,
                  hkv, D, 1.0, None, out, workspace=ws)
    for b in range(2):
        want, size = attend_rows(q[b * n:(b + 1) * n].astype(np.float64), np.arange(L - n, L), k[b].astype(np.float64),
                                 v[b].astype(np.float64), 1.0, 0, 0, hkv)
        # scores reach 160, where 32 bits hold 2^-17 at best and a sum of D products a few of them
        tol = attend_tolerance(size, L, 5.0) + 2.0 ** -13 * size
        assert (np.abs(f64(out)[b * n:(b + 1) * n] - want) <= tol).all()


def test_long_context_split_over_the_gpu():
    """Few rows over many keys: every SM takes a part of the axis, and the parts are joined."""
    run_prefill(Layout(1, 2, 20011, True, page=16, seed=3), [20011], [9], 8, 128)


def test_many_sequences():
    B = 150
    rng = np.random.RandomState(1)
    new = rng.randint(0, 12, B).tolist()
    lens = [n + int(rng.randint(0, 200)) for n in new]
    run_prefill(Layout(B, 1, 220, True, page=16, seed=3), lens, new, 4, 128, window=[50 * (b % 2) for b in range(B)],
                sink=2)


def test_one_token_each_without_starts():
    lay = Layout(4, 2, 300, True, seed=2)
    lens = [300, 1, 17, 128]
    k, v, _ = caches(lay, lens, [1] * 4, [0] * 4, 0, 128, 1)
    q = np.random.RandomState(2).randn(4, 8, 128).astype(np.float16)
    out = torch.empty(4, 8, 128, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_prefill(4, 4, 8, 2, 128, lay.capacity)
    fa.fa_prefill(*(torch.from_numpy(x).cuda() for x in (q, k, v)), None, lay.table_gpu(), None, ints(lens), 8, 2, 128,
                  0.09, None, out, workspace=ws)
    for b in range(4):
        want, size = attend_rows(q[b:b + 1].astype(np.float64), [lens[b] - 1], lay.dense(k, b).astype(np.float64),
                                 lay.dense(v, b).astype(np.float64), 0.09, 0, 0, 2)
        assert (np.abs(f64(out)[b:b + 1] - want) <= attend_tolerance(size, 300, 5.0)).all()


def test_captured_replayed_with_other_lengths_and_repeatable():
    hq, hkv, D, L = 8, 2, 128, 1000
    lay = Layout(2, hkv, L, True, seed=7)
    rng = np.random.RandomState(5)
    k, v = (rng.randn(*lay.rows, D).astype(np.float16) for _ in range(2))
    q = rng.randn(80, hq, D).astype(np.float16)
    dk, dv, dq, bt = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), torch.from_numpy(q).cuda(), lay.table_gpu()
    starts, lens, window = ints([0, 30, 80]), ints([500, 80]), ints([0, 0])
    out = torch.empty(80, hq, D, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_prefill(2, 80, hq, hkv, D, lay.capacity)

    def call():
        fa.fa_prefill(dq, dk, dv, None, bt, starts, lens, hq, hkv, D, D ** -0.5, window, out, n_sink=3, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    for st, ln, w in (([0, 30, 80], [500, 80], [0, 0]), ([0, 1, 41], [1000, 999], [0, 100]), ([0, 80, 80], [81, 5], [7, 0])):
        starts.copy_(ints(st))
        lens.copy_(ints(ln))
        window.copy_(ints(w))
        out.fill_(9.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        first = out.clone()
        g.replay()
        torch.cuda.synchronize()
        assert bool((first == out).all())
        for b in range(2):
            rows = slice(st[b], st[b + 1])
            n = st[b + 1] - st[b]
            want, size = attend_rows(q[rows].astype(np.float64), np.arange(ln[b] - n, ln[b]),
                                     lay.dense(k, b).astype(np.float64), lay.dense(v, b).astype(np.float64), D ** -0.5,
                                     w[b], 3, hkv)
            assert (np.abs(f64(out)[rows] - want) <= attend_tolerance(size, 1000, 5.0)).all()
        assert bool((out[st[2]:] == 9.0).all())


def dominated(L, D, hkv, rng):
    """Keys whose first takes about half of every query's weight, the others an even share."""
    k = rng.randn(1, hkv, L, D) * 0.02
    k[:, :, 0, 0] = np.log(L) / 4.0
    k[:, :, 1:, 0] = 0.0
    return k.astype(np.float16), rng.randn(1, hkv, L, D).astype(np.float16)


def dominated_error(got, q, at, k, v, scale, hkv):
    want, _ = attend_rows(q, at, k[0].astype(np.float64), v, scale, 0, 0, hkv)
    # the first key's part is the same value for all: what is left is the others' weights
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("L", [4096, 32768])
@pytest.mark.parametrize("vscale", [1.0, 0.02])
def test_keys_behind_a_dominant_one(L, vscale):
    """Weights of 2^-13 to 2^-16 behind a key that takes half of all keep fp16's 11 bits: the error of
    independent roundings (2^-11 / sqrt(3) each at most, of the weights and of the output) stays below
    5e-4 of the output's norm; weights rounded as subnormals (steps of 2^-24) would give 1e-3 and more."""
    D, hq, hkv, n = 128, 4, 1, 20
    rng = np.random.RandomState(3)
    k, v = dominated(L, D, hkv, rng)
    v = (v * vscale).astype(np.float16)
    v[:, :, 0] = 0
    q = rng.randn(n, hq, D).astype(np.float16)
    q[..., 0] = 4.0
    dev = [torch.from_numpy(x).cuda() for x in (q, k, v)]
    out = torch.empty(n, hq, D, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_prefill(1, n, hq, hkv, D, L)
    fa.fa_prefill(*dev, None, None, ints([0, n]), ints([L]), hq, hkv, D, 1.0, None, out, workspace=ws)
    err = dominated_error(f64(out), q.astype(np.float64), np.arange(L - n, L), k, v[0].astype(np.float64), 1.0, hkv)
    floor = np.sqrt(out.numel()) * 2.0 ** -25 / np.linalg.norm(f64(out))     # subnormal outputs' own rounding
    assert err <= 5e-4 + floor, (err, floor)


@pytest.mark.parametrize("L", [4096, 32768])
@pytest.mark.parametrize("int8", [False, True])
def test_sinks_keep_the_keys_behind_them(L, int8):
    D, hq, hkv = 128, 4, 1
    rng = np.random.RandomState(3)
    k, v = dominated(L, D, hkv, rng)
    v[:, :, 0] = 0
    s = None
    val = v.astype(np.float64)
    if int8:
        s = (np.abs(v.astype(np.float64).reshape(1, hkv, L, D // 32, 32)).max(-1) / 127).astype(np.float16)
        codes = np.where(s[..., None] > 0, np.rint(v.astype(np.float64).reshape(1, hkv, L, D // 32, 32) /
                                                   np.maximum(s[..., None].astype(np.float64), 1e-30)), 0)
        v = np.clip(codes, -127, 127).reshape(1, hkv, L, D).astype(np.int8)
        val = values(v, s)
    q = rng.randn(1, hq, D).astype(np.float16)
    q[..., 0] = 4.0
    out = torch.empty(1, hq, D, dtype=torch.float16, device="cuda")
    fa.fa_decode_sinks(*(torch.from_numpy(x).cuda() for x in (q, k, v)), None if s is None else
                       torch.from_numpy(s).cuda(), None, ints([L]), hq, hkv, D, 1.0, None, out, n_sink=4,
                       workspace=fa.alloc_workspace_sinks(1, 1, hq, hkv, D, L))
    err = dominated_error(f64(out), q.astype(np.float64), [L - 1], k, val[0], 1.0, hkv)
    floor = np.sqrt(out.numel()) * 2.0 ** -25 / np.linalg.norm(f64(out))
    assert err <= 5e-4 + floor, (err, floor)


@pytest.mark.parametrize("scale", [2.0 ** -24, 3 * 2.0 ** -24, 2.0 ** -14, 500.0])
def test_sinks_int8_scales_of_any_size(scale):
    """Subnormal and large scales: code * scale itself, whatever its split."""
    D, hq, hkv, L = 128, 4, 1, 64
    rng = np.random.RandomState(5)
    k = rng.randn(1, hkv, L, D).astype(np.float16)
    v = rng.randint(-127, 128, (1, hkv, L, D)).astype(np.int8)
    s = np.full((1, hkv, L, D // 32), scale, dtype=np.float16)
    s[:, :, ::3] = 0
    q = rng.randn(1, hq, D).astype(np.float16)
    out = torch.empty(1, hq, D, dtype=torch.float16, device="cuda")
    fa.fa_decode_sinks(*(torch.from_numpy(x).cuda() for x in (q, k, v, s)), None, ints([L]), hq, hkv, D, 0.1, None,
                       out, n_sink=4, workspace=fa.alloc_workspace_sinks(1, 1, hq, hkv, D, L))
    val = values(v, s)[0]
    want, size = attend_rows(q.astype(np.float64), [L - 1], k[0].astype(np.float64), val, 0.1, 0, 0, hkv)
    assert (np.abs(f64(out) - want) <= attend_tolerance(size, L, 127 * scale)).all()


# ------------------------------------------------------------------ decode with sinks
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("tq,lens,cap", [(1, [300, 5, 0, 37], 304), (3, [2000, 1, 700, 16], 2000),
                                         (1, [5000, 40, 4999, 1000], 5008), (2, [30, 64, 17, 2], 64)])
@pytest.mark.parametrize("window,sink", [(1, 0), (20, 4), (33, 17), (200, 1), (100, 500)])
def test_sinks(D, int8, paged, tq, lens, cap, window, sink):
    hq, hkv = 8, 2
    lay = Layout(4, hkv, cap, paged, seed=3)
    w = [window, 0, window, window]
    k, v, s = caches(lay, lens, [tq] * 4, w, sink, D, 11, int8=int8)
    q = np.random.RandomState(12).randn(4, tq, hq, D).astype(np.float16)
    out = torch.full((4, tq, hq, D), 9.0, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_sinks(4, tq, hq, hkv, D, lay.capacity)
    ws.fill_(255)
    fa.fa_decode_sinks(*(torch.from_numpy(x).cuda() for x in (q, k, v)), None if s is None else
                       torch.from_numpy(s).cuda(), lay.table_gpu(), ints(lens), hq, hkv, D, D ** -0.5, ints(w), out,
                       n_sink=sink, workspace=ws)
    got, val = f64(out), values(v, s)
    for b in range(4):
        at = np.arange(lens[b] - tq, lens[b])
        want, size = attend_rows(q[b].astype(np.float64), at, lay.dense(k, b).astype(np.float64), lay.dense(val, b),
                                 D ** -0.5, w[b], sink, hkv)
        # int8 V: one more rounding, of code * scale to fp16
        tol = attend_tolerance(size, max(lens[b], 1), 5.0) + (2.0 ** -11 * size if int8 else 0)
        assert np.isfinite(got[b]).all() and (np.abs(got[b] - want) <= tol).all()
        assert (got[b][at < 0] == 0).all()
    assert binding.fa_decode_device_status() == 0


def test_sinks_far_pages_may_be_unmapped():
    D, hq, hkv, lens = 128, 4, 1, [4000, 50]
    lay = Layout(2, hkv, 4000, True, seed=3)
    k, v, _ = caches(lay, lens, [1, 1], [100, 100], 20, D, 1)
    dense = [[lay.dense(x, b).astype(np.float64) for x in (k, v)] for b in range(2)]
    lay.table[0, 2:243] = -1
    q = np.random.RandomState(2).randn(2, hq, D).astype(np.float16)
    out = torch.empty(2, hq, D, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_sinks(2, 1, hq, hkv, D, lay.capacity)
    fa.fa_decode_sinks(*(torch.from_numpy(x).cuda() for x in (q, k, v)), None, lay.table_gpu(), ints(lens), hq, hkv, D,
                       D ** -0.5, ints([100, 100]), out, n_sink=20, workspace=ws)
    assert binding.fa_decode_device_status() == 0
    for b in range(2):
        want, size = attend_rows(q[b:b + 1].astype(np.float64), [lens[b] - 1], *dense[b], D ** -0.5, 100, 20, hkv)
        assert (np.abs(f64(out)[b:b + 1] - want) <= attend_tolerance(size, 4000, 5.0)).all()


def test_sinks_without_a_window_is_plain_decode():
    D, hq, hkv = 128, 8, 2
    lay = Layout(3, hkv, 700, True, seed=3)
    lens = [700, 3, 333]
    k, v, _ = caches(lay, lens, [1] * 3, [0] * 3, 0, D, 1)
    q = torch.from_numpy(np.random.RandomState(2).randn(3, hq, D).astype(np.float16)).cuda()
    kd, vd, bt = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), lay.table_gpu()
    a = torch.empty(3, hq, D, dtype=torch.float32, device="cuda")
    b = torch.empty(3, hq, D, dtype=torch.float16, device="cuda")
    fa.fa_decode(q, kd, vd, None, bt, ints(lens), hq, hkv, D, 0.1, None, a,
                 workspace=fa.alloc_workspace(3, hq, hkv, D, lay.capacity))
    fa.fa_decode_sinks(q, kd, vd, None, bt, ints(lens), hq, hkv, D, 0.1, None, b, n_sink=4,
                       workspace=fa.alloc_workspace_sinks(3, 1, hq, hkv, D, lay.capacity))
    assert float((a - b.float()).abs().max()) <= 2.0 ** -10


def test_sinks_of_many_sequences():
    """More than 128 sequences: the starts published for the merge."""
    D, hq, hkv, B = 128, 4, 1, 140
    rng = np.random.RandomState(7)
    lens = rng.randint(0, 3000, B).tolist()
    lay = Layout(B, hkv, 3000, True, seed=3)
    w = [int(x) for x in rng.randint(1, 1500, B)]
    k, v, _ = caches(lay, lens, [1] * B, w, 33, D, 1)
    q = rng.randn(B, hq, D).astype(np.float16)
    out = torch.empty(B, hq, D, dtype=torch.float16, device="cuda")
    fa.fa_decode_sinks(*(torch.from_numpy(x).cuda() for x in (q, k, v)), None, lay.table_gpu(), ints(lens), hq, hkv, D,
                       D ** -0.5, ints(w), out, n_sink=33,
                       workspace=fa.alloc_workspace_sinks(B, 1, hq, hkv, D, lay.capacity))
    for b in range(B):
        want, size = attend_rows(q[b:b + 1].astype(np.float64), [lens[b] - 1], lay.dense(k, b).astype(np.float64),
                                 lay.dense(v, b).astype(np.float64), D ** -0.5, w[b], 33, hkv)
        assert (np.abs(f64(out)[b:b + 1] - want) <= attend_tolerance(size, 3000, 5.0)).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("D,window,sink", [(128, 0, 0), (128, 90, 4), (256, 0, 0)])
def test_prompt_in_chunks_then_decode(D, window, sink):
    """A prompt taken whole and taken in chunks with a decode step between give the same rows, and the
    step after it, by fa_prefill and by fa_decode_sinks, too."""
    hq, hkv, B = 8, 2, 2
    lens = [300, 211]
    lay = Layout(B, hkv, 320, True, seed=1)
    bt = lay.table_gpu()
    table, mag = fa.fa_rope_table(D, 10000.0, scaling="yarn", factor=4.0, original_len=128)
    g = torch.Generator(device="cuda").manual_seed(2)
    xs = [torch.randn(n, hq + 2 * hkv, D, generator=g, device="cuda").to(torch.bfloat16) for n in lens]
    w = torch.rand(D, generator=g, device="cuda").to(torch.bfloat16) + 0.5
    win = ints([window] * B)

    def go(cuts):
        kc, vc = (torch.zeros(*lay.rows, D, dtype=torch.float16, device="cuda") for _ in range(2))
        outs = [[], []]
        for lo, hi in zip(cuts, cuts[1:]):
            part = [x[min(lo, len(x)):min(hi, len(x))] for x in xs]
            new = [len(x) for x in part]
            x = torch.cat(part)
            starts = ints([0, new[0], new[0] + new[1]])
            at = [min(lo, n) for n in lens]
            q = torch.empty(len(x), hq, D, dtype=torch.float16, device="cuda")
            fa.fa_rope_append_kv(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], q, kc, vc, None, bt, starts, ints(at),
                                 table, q_weight=w, k_weight=w, magnitude=mag)
            out = torch.empty_like(q)
            fa.fa_prefill(q, kc, vc, None, bt, starts, ints([a + n for a, n in zip(at, new)]), hq, hkv, D, D ** -0.5,
                          win, out, n_sink=sink, workspace=fa.alloc_workspace_prefill(B, len(x), hq, hkv, D, 320))
            for b in range(B):
                outs[b].append(out[sum(new[:b]):sum(new[:b + 1])])
        one = torch.empty(B, hq, D, dtype=torch.float16, device="cuda")
        last = torch.stack([x[-1] for x in xs])
        q = torch.empty(B, hq, D, dtype=torch.float16, device="cuda")
        fa.fa_rope(last[:, :hq], ints([n - 1 for n in lens]), table, q, weight=w, magnitude=mag)
        fa.fa_decode_sinks(q, kc, vc, None, bt, ints(lens), hq, hkv, D, D ** -0.5, win, one, n_sink=sink,
                           workspace=fa.alloc_workspace_sinks(B, 1, hq, hkv, D, 320))
        return [torch.cat(x) for x in outs], one, (kc, vc)

    whole, one, cache = go([0, 300])
    parts, two, cache2 = go([0, 100, 101, 211, 300])
    for a, b in zip(cache, cache2):
        assert bool((a == b).all())
    for b in range(B):
        # each side within a rounding of the weights and one of the output of the exact value, |v| under 5
        assert float((whole[b].float() - parts[b].float()).abs().max()) <= 2 * (2.0 ** -10 + 2.0 ** -14) * 5
        assert float((whole[b][-1].float() - one[b].float()).abs().max()) <= 2 * (2.0 ** -10 + 2.0 ** -14) * 5
    assert bool((one == two).all())


def test_offsets_beyond_32_bits():
    """A pool of more than 4 GiB per array, its last blocks in use: append, prefill and decode with sinks."""
    D, hq, hkv, page, n = 128, 4, 2, 16, 200
    total = (5 << 30) // (hkv * page * D * 2)
    kc, vc = (torch.zeros(total, hkv, page, D, dtype=torch.float16, device="cuda") for _ in range(2))
    assert kc.numel() * 2 > 1 << 32
    blocks = -(-n // page)
    table = (total - 1 - torch.arange(blocks, dtype=torch.int32, device="cuda")).view(1, -1).contiguous()
    x = torch.randn(n, hq + 2 * hkv, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").half()
    q = torch.empty(n, hq, D, dtype=torch.float16, device="cuda")
    starts = ints([0, n])
    fa.fa_rope_append_kv(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], q, kc, vc, None, table, starts, ints([0]), None)
    out = torch.empty_like(q)
    fa.fa_prefill(q, kc, vc, None, table, starts, ints([n]), hq, hkv, D, 0.1, None, out,
                  workspace=fa.alloc_workspace_prefill(1, n, hq, hkv, D, blocks * page))
    one = torch.empty(1, hq, D, dtype=torch.float16, device="cuda")
    fa.fa_decode_sinks(q[-1:].contiguous(), kc, vc, None, table, ints([n]), hq, hkv, D, 0.1, ints([50]), one, n_sink=3,
                       workspace=fa.alloc_workspace_sinks(1, 1, hq, hkv, D, blocks * page))
    k, v = (f64(x[:, a:a + hkv]).transpose(1, 0, 2) for a in (hq, hq + hkv))
    want, size = attend_rows(f64(q), np.arange(n), k, v, 0.1, 0, 0, hkv)
    assert (np.abs(f64(out) - want) <= attend_tolerance(size, n, 5.0)).all()
    want, size = attend_rows(f64(q[-1:]), [n - 1], k, v, 0.1, 50, 3, hkv)
    assert (np.abs(f64(one) - want) <= attend_tolerance(size, n, 5.0)).all()


def test_two_streams_and_a_reader_right_behind():
    """Two chunks at once, each with its own workspace, each read by what follows it on its stream."""
    D, hq, hkv, L, n = 128, 16, 4, 5000, 150
    rng = np.random.RandomState(2)
    lay = Layout(1, hkv, L, False)
    data, want = [], []
    for i in range(2):
        k, v = (rng.randn(*lay.rows, D).astype(np.float16) for _ in range(2))
        q = rng.randn(n, hq, D).astype(np.float16)
        w, size = attend_rows(q.astype(np.float64), np.arange(L - n, L), k[0].astype(np.float64), v[0].astype(np.float64),
                              D ** -0.5, 0, 0, hkv)
        want.append((w, attend_tolerance(size, L, 5.0)))
        data.append([torch.from_numpy(a).cuda() for a in (q, k, v)] +
                    [torch.empty(n, hq, D, dtype=torch.float16, device="cuda"),
                     fa.alloc_workspace_prefill(1, n, hq, hkv, D, L)])
    starts, lens = ints([0, n]), ints([L])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            q, k, v, out, ws = data[i]
            with torch.cuda.stream(s):
                out.fill_(9.0)
                fa.fa_prefill(q, k, v, None, None, starts, lens, hq, hkv, D, D ** -0.5, None, out, workspace=ws)
                got[i].append(out.clone())
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert (np.abs(f64(out) - want[i][0]) <= want[i][1]).all()
            assert bool((out == got[i][0]).all())


def test_workspaces_of_exact_size_are_enough():
    """Every byte behind the workspace's end stays."""
    for B, n, L, hq, hkv, D in ((1, 1, 16, 1, 1, 128), (3, 700, 900, 8, 1, 256), (2, 40, 3000, 8, 2, 128)):
        size = fa.fa_prefill_workspace_size(B, B * n, hq, hkv, D, L)
        buf = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
        q = torch.randn(B * n, hq, D, device="cuda").half()
        k, v = (torch.randn(B, hkv, L, D, device="cuda").half() for _ in range(2))
        out = torch.empty_like(q)
        fa.fa_prefill(q, k, v, None, None, ints([n * i for i in range(B + 1)]), ints([L] * B), hq, hkv, D, 0.1, None,
                      out, workspace=buf[:size])
        assert bool((buf[size:] == 77).all()) and bool(torch.isfinite(out).all())


def test_refusals_of_tensors():
    q = torch.zeros(4, 8, 128, dtype=torch.float16, device="cuda")
    k = torch.zeros(1, 2, 64, 128, dtype=torch.float16, device="cuda")
    ws = fa.alloc_workspace_prefill(1, 4, 8, 2, 128, 64)
    good = dict(q=q, k=k, v=k.clone(), vs=None, starts=ints([0, 4]), lens=ints([4]), out=torch.empty_like(q), ws=ws)

    def call(**kw):
        a = {**good, **kw}
        fa.fa_prefill(a["q"], a["k"], a["v"], a["vs"], None, a["starts"], a["lens"], 8, 2, 128, 0.1, None, a["out"],
                      workspace=a["ws"])

    call()
    for kw in (dict(q=q.float()), dict(k=k.float()), dict(starts=ints([0, 4, 5])), dict(lens=torch.tensor([4])),
               dict(out=torch.empty(4, 8, 64, dtype=torch.float16, device="cuda")), dict(q=q.transpose(0, 1)),
               dict(starts=torch.tensor([0, 4], device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw, code in ((dict(ws=None), -4), (dict(ws=ws[:1000]), -4), (dict(out=q), -7)):
        with pytest.raises(fa.FaDecodeError) as e:
            call(**kw)
        assert e.value.code == code
    torch.cuda.synchronize()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("hq,n", [(5, 355), (3, 41), (8, 700)])
def test_bits_do_not_depend_on_what_lies_beside(D, hq, n):
    """A row tile's last rows hold tokens of others, or nothing: the rows beside them keep their bits."""
    rng = np.random.RandomState(6)
    L = n + 200
    k, v = (torch.from_numpy(rng.randn(1, 1, L, D).astype(np.float16)).cuda() for _ in range(2))
    q = torch.from_numpy(rng.randn(n + 130, hq, D).astype(np.float16)).cuda()
    ws = fa.alloc_workspace_prefill(1, n + 130, hq, 1, D, L)
    got = []
    for fill in (0.0, 300.0, float("nan"), float("inf"), 0.0):
        q[n:] = fill
        out = torch.full_like(q, 9.0)
        fa.fa_prefill(q, k, v, None, None, ints([0, n]), ints([L]), hq, 1, D, D ** -0.5, None, out, workspace=ws)
        got.append(out)
        assert bool((out[n:] == 9.0).all())
    for x in got[1:]:
        assert bool((x == got[0]).all())
