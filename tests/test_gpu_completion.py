"""What is queued behind a decode call finds all of its rows written, also where no row has
partials to merge: one worker per unit, one tile per unit, or empty sequences beside long ones."""
import numpy as np
import pytest
import torch

from decode_step_kv_gb300 import binding as fa

pytestmark = pytest.mark.gpu


def step(kind, B, Hkv, length, D=128, G=2, empty=0):
    """A call of `kind` over one sequence's pages, which all block tables name."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    blocks = -(-length // 16)
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
    lens[B - empty:] = 0
    q = torch.randn(B, Hkv * G, D, generator=gen, device="cuda").half()
    rows = (blocks, Hkv, 16)
    acc = torch.zeros(rows, device="cuda")
    if kind.startswith("int4"):
        c = [torch.randint(0, 255, (*rows, D // 2), generator=gen, device="cuda", dtype=torch.uint8),
             torch.rand(*rows, D // 32, generator=gen, device="cuda").half()]
        c += [x.clone() for x in c]
        wt = kind == "int4 weights"
        out = torch.empty(B, Hkv * G, D, dtype=torch.float16, device="cuda")
        ws = fa.alloc_workspace_int4(B, 1, Hkv * G, Hkv, D, blocks * 16, weights=wt)
        return out, lambda: fa.fa_decode_int4(q, *c, table, lens, Hkv * G, Hkv, D, 0.05, None, out,
                                              acc=acc if wt else None, workspace=ws)
    k, v = (torch.randn(*rows, D, generator=gen, device="cuda").half() for _ in range(2))
    if kind == "weights":
        out = torch.empty(B, Hkv * G, D, dtype=torch.float16, device="cuda")
        ws = fa.alloc_workspace_weights(B, 1, Hkv * G, Hkv, D, blocks * 16)
        return out, lambda: fa.fa_decode_weights(q, k, v, None, table, lens, Hkv * G, Hkv, D, 0.05, None,
                                                 out, acc, workspace=ws)
    out = torch.empty(B, Hkv * G, D, dtype=torch.float32, device="cuda")
    if kind == "invariant":
        n = fa.fa_decode_batch_invariant_workspace_size(B, Hkv * G, Hkv, D, blocks * 16, 256)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        return out, lambda: fa.fa_decode_batch_invariant(q, k, v, None, table, lens, Hkv * G, Hkv, D, 0.05,
                                                         None, out, split_tokens=256, workspace=ws)
    ws = fa.alloc_workspace(B, Hkv * G, Hkv, D, blocks * 16)
    return out, lambda: fa.fa_decode(q, k, v, None, table, lens, Hkv * G, Hkv, D, 0.05, None, out, workspace=ws)


@pytest.mark.parametrize("kind", ["int4", "int4 weights", "weights", "decode", "invariant"])
@pytest.mark.parametrize("B,Hkv,length,empty", [(32, 8, 16, 0), (100, 2, 7, 40),    # one tile per unit
                                                (114, 16, 2048, 0), (76, 16, 2048, 0),   # a worker per unit
                                                (120, 16, 4000, 119)])
def test_rows_are_there_for_the_next_kernel(kind, B, Hkv, length, empty):
    if kind == "invariant" and length > 256:
        length = 256                                    # one split per unit: nothing to merge
    out, call = step(kind, B, Hkv, length, empty=empty)
    call()
    torch.cuda.synchronize()
    want = out.clone()
    assert torch.all(torch.isfinite(want)) and not want[B - empty:].any()
    copies = [torch.empty_like(out) for _ in range(20)]
    torch.cuda.synchronize()
    for c in copies:
        out.fill_(float("nan"))
        call()
        c.copy_(out)
    torch.cuda.synchronize()
    for c in copies:
        assert torch.equal(c, want)
    assert fa.fa_decode_device_status() == 0


def test_rows_are_there_inside_a_graph():
    out, call = step("int4", 114, 16, 2048)
    call()
    torch.cuda.synchronize()
    want, seen = out.clone(), torch.empty_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out.fill_(float("nan"))
        call()
        seen.copy_(out)
    for _ in range(20):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(seen, want)
