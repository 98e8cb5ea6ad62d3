"""Rotation of heads and the fused projection-to-cache pass against 64-bit forms."""
import numpy as np
import pytest
import torch

import decode_step_kv_gb300 as fa
from decode_step_kv_gb300 import binding
from _cache_ops import Layout
from _step_ops import f64, rates, turn, turn_tolerance

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def draw(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def check(got, want, size, dtype):
    err = np.abs(f64(got) - want)
    tol = turn_tolerance(want, size, dtype)
    assert np.isfinite(f64(got)).all()
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("src,dst", [(F16, F16), (BF16, BF16), (F32, F32), (F32, F16), (BF16, F32), (F16, BF16)])
@pytest.mark.parametrize("rot,inter,norm", [("all", False, True), ("all", True, False), (16, False, True),
                                            (48, True, True), (0, False, True), ("half", False, False)])
def test_rope(D, src, dst, rot, inter, norm):
    rot = {"all": D, "half": D // 2}.get(rot, rot)
    N, H = 13, 5
    x = draw((N, H, D), src, 1, 3.0)
    w = draw((D,), src, 2) if norm else None
    at = torch.randint(0, 1 << 20, (N,), dtype=torch.int32, generator=torch.Generator().manual_seed(3))
    at[0], at[1], at[2] = 0, (1 << 31) - 1, -7
    table, mag = fa.fa_rope_table(rot, 10000.0) if rot else (None, 1.0)
    out = torch.empty(N, H, D, dtype=dst, device="cuda")
    fa.fa_rope(x.cuda(), at.cuda(), table, out, weight=None if w is None else w.cuda(), eps=1e-5, interleaved=inter,
               magnitude=mag)
    rate = rates(rot, 10000.0)[0] if rot else np.zeros(0)
    want, size = turn(f64(x), at.numpy(), rate, 1.0, None if w is None else f64(w), 1e-5, inter)
    # positions near 2^31: the 64-bit reference angle itself is off by 2^31 * 2^-53 radians
    check(out, want, size + 2.0 ** -20, dst)


@pytest.mark.parametrize("N,H", [(1, 1), (1, 7), (3, 1), (1000, 3), (5000, 40)])
def test_rope_sizes_and_strides(N, H):
    """Token rows that lie apart, in and out, and what lies between them stays."""
    D = 128
    wide = draw((N, H + 3, D), F16, 5).cuda()
    x = wide[:, 1:1 + H]
    at = torch.arange(N, dtype=torch.int32, device="cuda") * 3
    table, mag = fa.fa_rope_table(D, 500000.0)
    to = torch.full((N, H + 2, D), 7.0, dtype=F16, device="cuda")
    fa.fa_rope(x, at, table, to[:, :H], magnitude=mag)
    want, size = turn(f64(x), at.cpu().numpy(), rates(D, 500000.0)[0], 1.0)
    check(to[:, :H], want, size, F16)
    assert bool((to[:, H:] == 7.0).all())


@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
@pytest.mark.parametrize("rot", [32, 128])
def test_scalings_in_place(scaling, factor, rot):
    N, H, D = 64, 4, 128
    x = draw((N, H, D), F32, 8)
    at = torch.linspace(0, 131071, N).int()
    table, mag = fa.fa_rope_table(rot, 10000.0, scaling=scaling, factor=factor, original_len=4096)
    rate, want_mag = rates(rot, 10000.0, scaling, factor, 4096)
    assert mag == pytest.approx(want_mag, rel=2.0 ** -24)
    y = x.cuda()
    fa.fa_rope(y, at.cuda(), table, y, magnitude=mag)
    want, size = turn(f64(x), at.numpy(), rate, mag)
    check(y, want, size, F32)


def test_positions_beyond_24_bits_keep_their_angle():
    """A quarter turn per position: exact at every position."""
    freqs = torch.full((8,), 1 << 62, dtype=torch.int64, device="cuda")
    x = torch.zeros(6, 1, 128, dtype=F32, device="cuda")
    x[..., 0] = 1.0
    at = torch.tensor([0, 1, 2, 3, (1 << 31) - 1, (1 << 30) + 2], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    fa.fa_rope(x, at, freqs, out)
    assert out[:, 0, 0].cpu().tolist() == [1, 0, -1, 0, 0, -1]
    assert out[:, 0, 8].cpu().tolist() == [0, 1, 0, -1, -1, 0]


def test_zeros_and_large_values_normed():
    """A zero head stays zero; a head of the largest fp16 values does not overflow."""
    x = torch.zeros(2, 1, 128, dtype=F16, device="cuda")
    x[1] = 65504.0
    w = torch.ones(128, dtype=F16, device="cuda")
    out = torch.empty_like(x)
    fa.fa_rope(x, None, None, out, weight=w)
    assert bool((out[0] == 0).all()) and bool((out[1] == 1).all())


# ------------------------------------------------------------------ the fused pass
def step(lay, new, at, hq, D, dtype, seed=0, rope_at=None, **kw):
    """Runs fa_rope_append_kv on fresh inputs; returns inputs, outputs and the caches before."""
    N = sum(new)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    x = draw((N, hq + 2 * lay.hkv, D), dtype, seed, 2.0).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + lay.hkv], x[:, hq + lay.hkv:]
    int8 = kw.pop("int8", False)
    kc = draw((*lay.rows, D), F16, seed + 1).cuda()
    vc = torch.randint(-127, 128, (*lay.rows, D), dtype=torch.int8).cuda() if int8 else \
        draw((*lay.rows, D), F16, seed + 2).cuda()
    vs = torch.rand(*lay.rows, D // 32).half().cuda() if int8 else None
    q_out = torch.full((N, hq, D), 9.0, dtype=F16, device="cuda")
    before = (kc.clone(), vc.clone(), None if vs is None else vs.clone())
    fa.fa_rope_append_kv(q, k, v, q_out, kc, vc, vs, lay.table_gpu(), torch.from_numpy(starts).cuda(),
                         torch.tensor(at, dtype=torch.int32, device="cuda"), kw.pop("table"),
                         rope_positions=None if rope_at is None else torch.tensor(rope_at, dtype=torch.int32,
                                                                                  device="cuda"), **kw)
    return (q, k, v), (q_out, kc, vc, vs), before


@pytest.mark.parametrize("D,hq,hkv", [(128, 8, 2), (128, 5, 1), (256, 6, 3)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("paged,page", [(True, 16), (True, 48), (False, 16)])
@pytest.mark.parametrize("int8,norm", [(False, True), (True, False)])
def test_append(D, hq, hkv, dtype, paged, page, int8, norm):
    new, at = [1, 0, 37, 100], [63, 5, 0, 17]
    lay = Layout(4, hkv, 128, paged, page=page, seed=4)
    rot = D // 2
    table, mag = fa.fa_rope_table(rot, 10000.0, scaling="yarn", factor=4.0, original_len=2048)
    rate, _ = rates(rot, 10000.0, "yarn", 4.0, 2048)
    qw = draw((D,), dtype, 20).cuda() if norm else None
    kw = draw((D,), dtype, 21).cuda() if norm else None
    (q, k, v), (q_out, kc, vc, vs), before = step(lay, new, at, hq, D, dtype, table=table, magnitude=mag, int8=int8,
                                                  q_weight=qw, k_weight=kw)
    pos = np.concatenate([np.arange(n) + a for n, a in zip(new, at)])
    want, size = turn(f64(q), pos, rate, mag, None if qw is None else f64(qw))
    check(q_out, want, size, F16)
    want_k, size_k = turn(f64(k), pos, rate, mag, None if kw is None else f64(kw))
    touched = np.zeros(lay.rows, dtype=bool)
    row = 0
    if int8:
        codes = torch.empty(v.shape, dtype=torch.int8, device="cuda")
        scales = torch.empty(*v.shape[:2], D // 32, dtype=F16, device="cuda")
        fa.fa_quantize_v_int8(v.float().contiguous(), codes, scales)
    for b, (n, a) in enumerate(zip(new, at)):
        kk, vv = lay.dense(f64(kc), b)[:, a:a + n], lay.dense(vc.cpu().numpy(), b)[:, a:a + n]
        err = np.abs(kk - np.moveaxis(want_k[row:row + n], 0, 1))
        assert (err <= turn_tolerance(np.moveaxis(want_k[row:row + n], 0, 1),
                                      np.moveaxis(size_k[row:row + n], 0, 1), F16)).all()
        if int8:
            assert (vv == np.moveaxis(codes[row:row + n].cpu().numpy(), 0, 1)).all()
            assert (lay.dense(vs.cpu().numpy(), b)[:, a:a + n] ==
                    np.moveaxis(scales[row:row + n].cpu().numpy(), 0, 1)).all()
        else:
            assert (vv == np.moveaxis(v[row:row + n].half().cpu().numpy(), 0, 1)).all()
        d = lay.dense(touched, b).copy()
        d[:, a:a + n] = True
        lay.put(touched, b, d)
        row += n
    for got, old in ((kc, before[0]), (vc, before[1]), (vs, before[2])):
        if got is not None:
            same = (got == old).cpu().numpy().reshape(*lay.rows, -1).all(-1)
            assert same[~touched].all()
    assert binding.fa_decode_device_status() == 0


def test_int8_codes_at_ties():
    """Values next to the codec's ties get the codes of the exact quotient."""
    g = torch.Generator().manual_seed(3)
    N, D = 400, 128
    s = torch.rand(N, 1, 1, generator=g) + 0.01
    s16 = s.half().float()
    k = torch.randint(-127, 127, (N, 1, D), generator=g).float() + 0.5
    x = k * s16
    x = torch.where(torch.rand(N, 1, D, generator=g) < 0.5, x, torch.nextafter(x, torch.zeros_like(x)))
    x = torch.where(torch.rand(N, 1, D, generator=g) < 0.5, x, torch.nextafter(x, 1e9 * torch.sign(x)))
    x[..., ::32] = 127 * s16
    x = x.cuda()
    codes = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    scales = torch.empty(N, 1, D // 32, dtype=F16, device="cuda")
    fa.fa_quantize_v_int8(x, codes, scales)
    kc = torch.zeros(1, 1, N, D, dtype=F16, device="cuda")
    vc = torch.zeros(1, 1, N, D, dtype=torch.int8, device="cuda")
    vs = torch.zeros(1, 1, N, D // 32, dtype=F16, device="cuda")
    starts = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    fa.fa_rope_append_kv(None, x, x, None, kc, vc, vs, None, starts, torch.zeros(1, dtype=torch.int32, device="cuda"),
                         None)
    assert bool((vc[0, 0] == codes[:, 0]).all()) and bool((vs[0, 0] == scales[:, 0]).all())


def test_append_bad_rows_are_left_out():
    """Rows outside the cache, in unmapped blocks or of no sequence: flagged or left alone."""
    D, hq, hkv = 128, 2, 1
    lay = Layout(3, hkv, 32, True, page=16, seed=1)
    lay.table[1, 1] = -1
    table, _ = fa.fa_rope_table(D)
    (q, *_), (q_out, kc, vc, _), before = step(lay, [3, 4, 2], [31, 14, -1], hq, D, F16, table=table)
    assert binding.fa_decode_device_status() == binding.FA_STATUS_POS_RANGE | binding.FA_STATUS_BAD_BLOCK
    changed = (kc != before[0]).any(-1).cpu().numpy()
    assert changed[lay.table[0, 1], 0, 15] and changed[lay.table[1, 0], 0, 14:].all()
    assert changed.sum() == 3
    want, size = turn(f64(q), [31, 32, 33, 14, 15, 16, 17, -1, 0], rates(D, 10000.0)[0], 1.0)
    check(q_out, want, size, F16)
    # rows before the first sequence and behind the last
    x = draw((9, 4, D), F16, 2).cuda()
    q_out.fill_(9.0)
    kc2 = kc.clone()
    fa.fa_rope_append_kv(x[:, :2], x[:, 2:3], x[:, 3:], q_out, kc, vc, None, lay.table_gpu(),
                         torch.tensor([2, 4, 4, 5], dtype=torch.int32, device="cuda"),
                         torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda"), table)
    assert bool((q_out[:2] == 9).all()) and bool((q_out[5:] == 9).all()) and not bool((q_out[2:5] == 9).any())
    assert (kc != kc2).any(-1).sum() == 3


def test_append_rope_positions_and_one_token_each():
    """After an eviction the cache index is not the position; starts None: one token each."""
    D, hkv = 256, 2
    lay = Layout(3, hkv, 64, False)
    table, _ = fa.fa_rope_table(D)
    x = draw((3, hkv, D), BF16, 6).cuda()
    kc, vc = (torch.zeros(*lay.rows, D, dtype=F16, device="cuda") for _ in range(2))
    at, rope_at = [5, 63, 0], [100005, 63, 7]
    fa.fa_rope_append_kv(None, x, x, None, kc, vc, None, None, None,
                         torch.tensor(at, dtype=torch.int32, device="cuda"), table,
                         rope_positions=torch.tensor(rope_at, dtype=torch.int32, device="cuda"))
    want, size = turn(f64(x), rope_at, rates(D, 10000.0)[0], 1.0)
    for b in range(3):
        check(kc[b, :, at[b]], want[b], size[b], F16)
        assert bool((vc[b, :, at[b]] == x[b].half()).all())
    assert int((kc != 0).any(-1).sum()) == 3 * hkv


def test_append_in_a_graph_on_another_stream():
    D, hq, hkv, B = 128, 4, 2, 5
    lay = Layout(B, hkv, 64, True, seed=3)
    x = draw((B, hq + 2 * hkv, D), F16, 9).cuda()
    at = torch.arange(B, dtype=torch.int32, device="cuda")
    table, _ = fa.fa_rope_table(D)
    bt = lay.table_gpu()
    kc, vc = (torch.zeros(*lay.rows, D, dtype=F16, device="cuda") for _ in range(2))
    q_out = torch.zeros(B, hq, D, dtype=F16, device="cuda")

    def call():
        fa.fa_rope_append_kv(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], q_out, kc, vc, None, bt, None, at, table)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    for shift in (7, 40):
        at.copy_(torch.arange(B, dtype=torch.int32) + shift)
        g.replay()
        torch.cuda.synchronize()
        want, size = turn(f64(x[:, :hq]), np.arange(B) + shift, rates(D, 10000.0)[0], 1.0)
        check(q_out, want, size, F16)
        for b in range(B):
            assert (lay.dense(vc.cpu().numpy(), b)[:, b + shift] == x[b, hq + hkv:].cpu().numpy()).all()


def test_refusals_of_tensors():
    D, hq, hkv, N = 128, 4, 2, 3
    x = draw((N, hq + 2 * hkv, D), F16, 1).cuda()
    kc, vc = (torch.zeros(N, hkv, 16, D, dtype=F16, device="cuda") for _ in range(2))
    table, _ = fa.fa_rope_table(D)
    at = torch.zeros(N, dtype=torch.int32, device="cuda")
    good = dict(q=x[:, :hq], k=x[:, hq:hq + hkv], v=x[:, hq + hkv:], qo=torch.empty(N, hq, D, dtype=F16, device="cuda"),
                kc=kc, vc=vc, at=at, table=table, w=None)

    def call(**kw):
        a = {**good, **kw}
        fa.fa_rope_append_kv(a["q"], a["k"], a["v"], a["qo"], a["kc"], a["vc"], None, None, None, a["at"], a["table"],
                             q_weight=a["w"])

    call()
    for kw in (dict(q=x[:2, :hq]), dict(q=x[:, :hq].float()), dict(k=x[:, hq:hq + hkv].transpose(1, 2)),
               dict(v=x[:, hq:hq + 1]), dict(qo=None), dict(qo=torch.empty(N, hq, D, device="cuda")), dict(kc=kc[:2]),
               dict(vc=vc.float()), dict(at=at.long()), dict(table=table.float()), dict(w=table),
               dict(k=x[:, ::2][:, :hkv]), dict(v=x[:, hq + hkv:].cpu()), dict(q=x[0])):
        with pytest.raises(ValueError):
            call(**kw)
    out = torch.empty(N, hq, D, dtype=F16, device="cuda")
    for a, b in ((x[:, :hq], out[:2]), (x[:, :hq].int(), out), (x[:, :hq].cpu(), out)):
        with pytest.raises(ValueError):
            fa.fa_rope(a, at, table, b)
    with pytest.raises(fa.FaDecodeError) as e:
        fa.fa_rope(x[:, :hq], at, table, x[:, 1:hq + 1])       # a shifted overlap
    assert e.value.code == -7
    torch.cuda.synchronize()
