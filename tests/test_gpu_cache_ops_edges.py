"""4-bit cache, recorded weights and eviction at the ends of their ranges: the codec next to its
midpoints, hundreds of columns, large batches, byte offsets beyond 32 bits, captured graphs."""
import numpy as np
import pytest
import torch

from decode_step_kv_gb300 import binding as fa

import test_gpu_evict as ev
import test_gpu_int4 as i4
from _cache_ops import Int4Cache, Layout, attend, cuda, lens_gpu, pack, quantize, queries

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ codec
@pytest.mark.parametrize("low,high", [(-24, -10), (-10, 10), (10, 15.9)])
def test_codec_next_to_its_midpoints(low, high):
    """Elements within two fp32 steps of (c + 1/2) s, and largest magnitudes within two steps of
    7 times a midpoint of two fp16 scales."""
    r = np.random.RandomState(int(high) + 50)
    n = 1 << 15
    s = (2.0 ** r.uniform(low, high, (n, 1))).astype(np.float16).astype(np.float64)
    x = ((r.randint(-7, 7, (n, 32)) + 0.5) * s).astype(np.float32)
    x = (x.view(np.int32) + r.randint(-2, 3, x.shape).astype(np.int32)).view(np.float32)
    half = np.ldexp(1.0, np.maximum(np.frexp(s[:, 0])[1] - 1, -14) - 11)     # half a place of s
    top = np.where(r.random_sample(n) < 0.5, 7 * s[:, 0], 7 * (s[:, 0] + half)).astype(np.float32)
    top = (top.view(np.int32) + r.randint(-2, 3, n).astype(np.int32)).view(np.float32)
    x[np.arange(n), r.randint(0, 32, n)] = top * r.choice([-1, 1], n).astype(np.float32)
    x = x.reshape(2, n // 16, 2, 128)
    T = n // 16
    c = [torch.zeros((2, 2, T, w), dtype=t, device="cuda")
         for w, t in ((64, torch.uint8), (4, torch.float16)) * 2]
    fa.fa_append_kv_int4(cuda(x), cuda(-x), *c, None, lens_gpu([0, 0]))
    for got, scales, y in ((c[0], c[1], x), (c[2], c[3], -x)):
        codes, want = quantize(np.moveaxis(y, 1, 2))
        assert np.array_equal(scales.cpu().numpy(), want)
        assert np.array_equal(got.cpu().numpy(), pack(codes))
    assert fa.fa_decode_device_status() == 0


# ------------------------------------------------------------------ recorded weights
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("tq,Hq,Hkv", [(40, 16, 1), (200, 3, 1), (64, 16, 2)])
def test_hundreds_of_columns(D, tq, Hq, Hkv):
    lens = [0, 3, 130, 256]
    lay = Layout(4, Hkv, 256, True, 32, seed=tq)
    q = queries(4, tq, Hq, D, 3)
    i4.check(lay, Int4Cache(lay, D, lens, seed=1), q, lens, Hq, D ** -0.5)
    ev.check(lay, ev.Cache(lay, D, lens, True, seed=2), q, lens, Hq, D ** -0.5)


@pytest.mark.parametrize("B", [33, 140, 300])
def test_weights_of_many_sequences(B):
    lens = [(37 * b) % 70 for b in range(B)]
    lay = Layout(B, 1, 80, True)
    ev.check(lay, ev.Cache(lay, 128, lens, False, seed=B), queries(B, 1, 3, 128, B), lens, 3, 0.1,
             [b % 5 * 9 for b in range(B)])


@pytest.mark.parametrize("tq,Hq", [(8, 8), (3, 5)])
def test_many_sequences_of_many_columns(tq, Hq):
    lens = [(41 * b) % 130 for b in range(150)]
    lay = Layout(150, 1, 144, True, 48)
    i4.check(lay, Int4Cache(lay, 128, lens, seed=7), queries(150, tq, Hq, 128, 2), lens, Hq, 0.1,
             [b % 4 * 30 for b in range(150)])


# ------------------------------------------------------------------ offsets beyond 32 bits
def test_rows_behind_four_gigabytes():
    """The same tokens in the first and the last blocks of a pool: equal bytes everywhere."""
    Hkv, page, T = 8, 64, 700
    blocks = (9 << 29) // (Hkv * page * 64)                # 4.5 GiB of codes, K and V each
    rows = (blocks, Hkv, page)
    pools = [torch.empty((*rows, w), dtype=t, device="cuda")
             for w, t in ((64, torch.uint8), (4, torch.float16)) * 2]
    acc = torch.zeros(rows, device="cuda")
    need = -(-(T + 4) // page)
    x = torch.randn((1, T, Hkv, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    q = cuda(queries(1, 1, 32, 128, 1))
    ws = fa.alloc_workspace_int4(1, 1, 32, Hkv, 128, need * page, weights=True)
    got = []
    for first in (0, blocks - need):
        table = torch.arange(first + need - 1, first - 1, -1, dtype=torch.int32, device="cuda")[None]
        fa.fa_append_kv_int4(x, -x, *pools, table, lens_gpu([0]))
        out = torch.empty_like(q)
        fa.fa_decode_int4(q, *pools, table, lens_gpu([T]), 32, Hkv, 128, 0.1, None, out, acc=acc,
                          workspace=ws)
        totals = acc[table[0].long()].clone()
        kept = torch.empty((1, Hkv, 100), dtype=torch.int32, device="cuda")
        new = torch.empty(1, dtype=torch.int32, device="cuda")
        fa.fa_evict_kv(pools[0], pools[2], acc, table, lens_gpu([T]), new, budget=100, n_sink=4,
                       n_recent=20, kept=kept, k_scales=pools[1], v_scales=pools[3])
        k, v = (torch.empty((1, 100, Hkv, 128), dtype=torch.float16, device="cuda") for _ in range(2))
        fa.fa_gather_kv_int4(*pools, table, lens_gpu([0]), k, v)
        got.append((out, totals, kept, k, v, acc[table[0].long()].clone()))
    assert fa.fa_decode_device_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.all(got[0][3] == -got[0][4]) and float(got[0][1].sum()) > 31.9
    del pools, acc


def test_fp16_rows_behind_four_gigabytes():
    Hkv, page, T = 8, 64, 700
    blocks = (9 << 29) // (Hkv * page * 256)
    rows = (blocks, Hkv, page)
    k, v = (torch.empty((*rows, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    acc = torch.zeros(rows, device="cuda")
    need = -(-T // page)
    g = torch.Generator("cuda").manual_seed(1)
    kr, vr = (torch.randn((need, Hkv, page, 128), device="cuda", generator=g).half() for _ in range(2))
    q = cuda(queries(1, 1, 32, 128, 1))
    ws = fa.alloc_workspace_weights(1, 1, 32, Hkv, 128, need * page)
    got = []
    for first in (0, blocks - need):
        table = torch.arange(first, first + need, dtype=torch.int32, device="cuda")[None]
        k[first:first + need], v[first:first + need] = kr, vr
        out = torch.empty_like(q)
        fa.fa_decode_weights(q, k, v, None, table, lens_gpu([T]), 32, Hkv, 128, 0.1, None, out, acc,
                             workspace=ws)
        totals = acc[first:first + need].clone()
        kept = torch.empty((1, Hkv, 100), dtype=torch.int32, device="cuda")
        new = torch.empty(1, dtype=torch.int32, device="cuda")
        fa.fa_evict_kv(k, v, acc, table, lens_gpu([T]), new, budget=100, n_sink=4, n_recent=20,
                       kept=kept)
        got.append((out, totals, kept, k[first:first + need].clone(), v[first:first + need].clone(),
                    acc[first:first + need].clone()))
    assert fa.fa_decode_device_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    del k, v, acc


# ------------------------------------------------------------------ eviction
def test_evict_flags_unmapped_recent_tokens():
    """An unmapped block among the last n_recent tokens: its rows count as kept, none moves."""
    lay = Layout(1, 2, 64, True, seed=3)
    lay.table[0, 3] = -1                                    # tokens 48..63
    k = torch.arange(lay.rows[0] * 2 * 16, device="cuda").reshape(lay.rows)[..., None]
    k = (k % 2048).half().expand(*lay.rows, 128).contiguous()
    before, accd = k.clone(), torch.ones(lay.rows, device="cuda")
    kept = torch.empty((1, 2, 20), dtype=torch.int32, device="cuda")
    nl = torch.empty(1, dtype=torch.int32, device="cuda")
    fa.fa_decode_device_status()
    fa.fa_evict_kv(k, k.clone(), accd, lay.table_gpu(), lens_gpu([64]), nl, budget=20, n_sink=0,
                   n_recent=20, kept=kept)
    assert fa.fa_decode_device_status() == fa.FA_STATUS_BAD_BLOCK
    assert kept[0, 1].tolist() == list(range(44, 64))
    t = lay.table[0]
    assert torch.equal(k[t[0], :, :4], before[t[2], :, 12:])
    assert torch.equal(k[t[0], :, 4:], before[t[0], :, 4:])
    spare = [i for i in range(lay.rows[0]) if i not in t.tolist()]
    assert torch.equal(k[spare], before[spare])


@pytest.mark.parametrize("kind", ["fp16", "int4"])
def test_evict_of_everything_but_one_in_two_kernels(kind):
    """Few units and many rows: the far rows go in a second kernel; lengths at budget + 1."""
    lay = Layout(2, 1, 40016, False, seed=1)
    ev.check_evict(kind, lay, 256, [40011, 20001], 20000, 4, 100, ev.totals(lay, 5, "odd"))


@pytest.mark.parametrize("how", ["heavy", "ties", "odd"])
@pytest.mark.parametrize("n,budget", [(50000, 9000), (26000, 3000), (24001, 1300), (30001, 500)])
def test_evict_selects_from_more_tokens_than_a_cta_holds(n, budget, how):
    """Selection by clusters of 16, 8, 2 and 1 CTAs."""
    lay = Layout(1, 3, n, True, 64, seed=1)
    ev.check_evict("int4", lay, 128, [n], budget, 5, 60, ev.totals(lay, n, how))


def test_evict_again_after_more_steps():
    """Most kept tokens at their places already: an eviction of what an eviction left and new tokens."""
    lay = Layout(2, 2, 1504, True, seed=8)
    r = np.random.RandomState(4)
    acc = np.zeros(lay.rows, dtype=np.float32)
    for b in range(2):
        a = np.concatenate([r.random_sample((2, 1000)) + 1, r.random_sample((2, 504))], axis=1)
        a[:, 700 + 100 * b] = 0                             # the first dropped token
        lay.put(acc, b, a.astype(np.float32))
    ev.check_evict("int8v", lay, 128, [1500, 1100], 1000, 4, 50, acc)
    ev.check_evict("fp16", lay, 128, [1500, 1100], 1000, 0, 0, acc)
    for b in range(2):
        lay.put(acc, b, np.broadcast_to(-np.arange(1504, dtype=np.float32), (2, 1504)))
    ev.check_evict("fp16", lay, 128, [1500, 1001], 1000, 0, 0, acc)      # the first 1000 stay


def test_evict_contiguous_cache_of_odd_capacity():
    lay = Layout(3, 3, 307, False, seed=1)
    ev.check_evict("int8v", lay, 128, [307, 33, 301], 32, 3, 5, ev.totals(lay, 5))


# ------------------------------------------------------------------ graphs
@pytest.mark.parametrize("tq,Hq", [(1, 4), (4, 8), (16, 8)])
def test_two_graphs_of_two_workspaces(tq, Hq):
    """Graphs captured on two streams, replayed side by side, each with its own workspace."""
    lens = [900, 4000]
    lay = Layout(2, 2, 4000, True, seed=3)
    cache = Int4Cache(lay, 128, lens, seed=3)
    dev, table, ln = cache.gpu(), lay.table_gpu(), lens_gpu(lens)
    qs = [cuda(queries(2, tq, 2 * Hq, 128, s)) for s in (1, 2)]
    want = [i4.run(lay, cache, q.cpu().numpy(), lens, 2 * Hq, 0.1) for q in qs]
    outs = [torch.zeros_like(q) for q in qs]
    wss = [fa.alloc_workspace_int4(2, tq, 2 * Hq, 2, 128, lay.cap) for _ in qs]
    graphs, streams = [torch.cuda.CUDAGraph() for _ in qs], [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for g, q, out, ws in zip(graphs, qs, outs, wss):
        with torch.cuda.graph(g):
            fa.fa_decode_int4(q, *dev, table, ln, 2 * Hq, 2, 128, 0.1, None, out, workspace=ws)
    for _ in range(5):
        for g, s, out in zip(graphs, streams, outs):
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def test_a_step_in_one_graph():
    """Append, attention with weights and eviction captured together and replayed on new rows."""
    B, Hkv, Hq, cap, n = 3, 2, 8, 512, 400
    lay = Layout(B, Hkv, cap, True, 32, seed=6)
    table = lay.table_gpu()
    g = torch.Generator("cuda").manual_seed(2)
    prompt = torch.randn((B, n, Hkv, 128), device="cuda", generator=g)
    steps = [torch.randn((B, 1, Hkv, 128), device="cuda", generator=g) for _ in range(3)]
    queries_ = [torch.randn((B, 1, Hq, 128), device="cuda", generator=g).half() for _ in range(3)]

    def state():
        pools = [torch.zeros((*lay.rows, w), dtype=t, device="cuda")
                 for w, t in ((64, torch.uint8), (4, torch.float16)) * 2]
        fa.fa_append_kv_int4(prompt, prompt, *pools, table, lens_gpu([0] * B))
        return dict(pools=pools, acc=torch.zeros(lay.rows, device="cuda"), x=steps[0].clone(),
                    q=queries_[0].clone(), pos=lens_gpu([n, 90, 200]), lens=lens_gpu([n + 1, 91, 201]),
                    new=lens_gpu([0] * B), out=torch.zeros((B, 1, Hq, 128), dtype=torch.float16,
                                                           device="cuda"),
                    kept=torch.zeros((B, Hkv, 128), dtype=torch.int32, device="cuda"),
                    ws=fa.alloc_workspace_int4(B, 1, Hq, Hkv, 128, cap, weights=True))

    def step(s):
        fa.fa_append_kv_int4(s["x"], s["x"], *s["pools"], table, s["pos"])
        fa.fa_decode_int4(s["q"], *s["pools"], table, s["lens"], Hq, Hkv, 128, 0.1, None, s["out"],
                          acc=s["acc"], workspace=s["ws"])
        fa.fa_evict_kv(s["pools"][0], s["pools"][2], s["acc"], table, s["lens"], s["new"], budget=128,
                       n_sink=4, n_recent=16, kept=s["kept"], k_scales=s["pools"][1],
                       v_scales=s["pools"][3])
        s["pos"].copy_(s["new"])
        s["lens"].copy_(s["new"] + 1)

    eager, replayed = state(), state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(replayed)
    for x, q in zip(steps, queries_):
        for s in (eager, replayed):
            s["x"].copy_(x)
            s["q"].copy_(q)
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "acc", "new", "kept"):
            assert torch.equal(eager[name], replayed[name])
        for a, b in zip(eager["pools"], replayed["pools"]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert eager["new"].tolist() == [128, 93, 128]
