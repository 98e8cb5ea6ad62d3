"""Chunk attention over so many keys that a sum which drops bits at every addition would show."""
import pytest
import torch

import decode_step_kv_gb300 as fa
from decode_step_kv_gb300 import binding

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attend(q, k, v, vs, n, L, hq, D, window=None, sink=0):
    out = torch.empty(n, hq, D, dtype=torch.float16, device="cuda")
    fa.fa_prefill(q, k, v, vs, None, ints([0, n]), ints([L]), hq, 1, D, D ** -0.5, window, out, n_sink=sink,
                  workspace=fa.alloc_workspace_prefill(1, n, hq, 1, D, L))
    assert binding.fa_decode_device_status() == 0
    return out


def codes(v):
    """V as int8 codes and scales, and their values."""
    blk = v.float().unflatten(-1, (-1, 32))
    s = (blk.abs().amax(-1, keepdim=True) / 127).half()
    c = torch.round(blk / s.float()).clamp(-127, 127)
    return c.flatten(-2).to(torch.int8), s.squeeze(-1), (c * s.float()).flatten(-2)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("L,n,hq", [(524288, 4096, 8), (100000, 4096, 8), (300000, 3, 4), (40000, 9000, 1)])
def test_values_that_do_not_change_along_the_keys(D, int8, L, n, hq):
    """Every key has the same V row, so that row is the result, whatever the weights: the units are long, taken
    whole or cut.  32-bit sums whose additions drop up to a step (2^-23) lose 2^-13 over the 1024 additions of
    16384 keys.  The weights' roundings, 2^-11 each at most, fall on both sides: of a mean over this many keys
    they leave under 2^-14.  int8 V is rounded by 2^-11, and so is the output."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(n, hq, D, device="cuda", generator=g).half()
    k = torch.randn(1, 1, L, D, device="cuda", generator=g).half()
    row = (torch.rand(D, device="cuda", generator=g) + 0.5).half()
    v, vs, val = row.expand(1, 1, L, D).contiguous(), None, row.float()
    if int8:
        c, s, val = codes(row)
        v, vs = c.expand(1, 1, L, D).contiguous(), s.expand(1, 1, L, D // 32).contiguous()
    out = attend(q, k, v, vs, n, L, hq, D)
    rel = (out.float() / val - 1).abs().amax().item()
    assert rel <= 2.0 ** -13 + 2.0 ** -14 + 2.0 ** -11 * (2 if int8 else 1), rel


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("grow", [False, True])
def test_against_64_bits(D, grow):
    """Rows over 2^19 keys by the norm of their error: a rounding of each weight and of the output, in
    quadrature (see the bounds of shorter contexts), and 2^-13 of what the sums drop.  `grow`: scores that rise
    along the keys, so that what was summed before is scaled down again and again."""
    L, n, hq = 524288, 2048, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(n, hq, D, device="cuda", generator=g).half()
    k = torch.randn(1, 1, L, D, device="cuda", generator=g).half()
    if grow:
        q[..., 0] = 4.0
        k[0, 0, :, 0] = torch.linspace(0, 40 * D ** 0.5 / 16, L, device="cuda").half()
    v = (torch.randn(1, 1, L, D, device="cuda", generator=g) + 0.5).half()
    out = attend(q, k, v, None, n, L, hq, D)
    for i in (0, 777, n - 1):
        end = L - n + i + 1
        p = torch.softmax(q[i].double() @ k[0, 0, :end].double().T * D ** -0.5, dim=-1)
        want = p @ v[0, 0, :end].double()
        spread = (p.square() @ v[0, 0, :end].double().square().sum(-1)).sqrt()
        err = (out[i].double() - want).norm(dim=-1)
        most = 2 * 2.0 ** -11 * spread + (2.0 ** -11 + 2.0 ** -13 + 2.0 ** -16) * want.norm(dim=-1)
        assert bool((err <= most).all()), float((err / most).max())


@pytest.mark.parametrize("D", [128, 256])
def test_windows_of_many_tiles(D):
    """A window and sinks beyond one stretch of keys: rows of a unit begin and end at different tiles."""
    L, n, hq, window, sink = 60000, 300, 8, 40000, 700
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(n, hq, D, device="cuda", generator=g).half()
    k = torch.randn(1, 1, L, D, device="cuda", generator=g).half()
    v = (torch.randn(1, 1, L, D, device="cuda", generator=g) + 0.5).half()
    k[0, 0, sink:L - n - window + 1] = float("nan")
    v[0, 0, sink:L - n - window + 1] = float("nan")
    out = attend(q, k, v, None, n, L, hq, D, ints([window]), sink)
    for i in (0, 150, n - 1):
        at = L - n + i
        t = torch.cat([torch.arange(sink, device="cuda"), torch.arange(at - window + 1, at + 1, device="cuda")])
        p = torch.softmax(q[i].double() @ k[0, 0, t].double().T * D ** -0.5, dim=-1)
        want = p @ v[0, 0, t].double()
        spread = (p.square() @ v[0, 0, t].double().square().sum(-1)).sqrt()
        err = (out[i].double() - want).norm(dim=-1)
        most = 2 * 2.0 ** -11 * spread + (2.0 ** -11 + 2.0 ** -13 + 2.0 ** -16) * want.norm(dim=-1)
        assert bool((err <= most).all()), float((err / most).max())
