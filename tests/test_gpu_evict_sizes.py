"""Eviction with budgets whose index arithmetic passes 32 bits."""
import pytest
import torch

from decode_step_kv_gb300 import binding as fa

pytestmark = pytest.mark.gpu


def cache(tokens, D=128):
    """A contiguous 4-bit cache of one sequence and one KV head (~148 bytes per token)."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randint(0, 256, (1, 1, tokens, D // 2), dtype=torch.uint8, device="cuda", generator=gen)
    ks = torch.rand(1, 1, tokens, D // 32, dtype=torch.float16, device="cuda", generator=gen)
    acc = torch.rand(1, 1, tokens, device="cuda", generator=gen)
    return k, ks, k.flip(-1), ks.flip(-1).contiguous(), acc


def test_tens_of_millions_of_tokens():
    """The totals behind the budget start again from zero, and no others do."""
    n, budget, sink, recent = 86_000_000, 66_000_000, 4, 1000
    k, ks, v, vs, acc = cache(n)
    old_k, old_vs, old_acc = k.clone(), vs.clone(), acc.clone()
    lens, new_lens = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (n, 0))
    kept = torch.empty(1, 1, budget, dtype=torch.int32, device="cuda")
    fa.fa_decode_device_status()
    fa.fa_evict_kv(k, v, acc, None, lens, new_lens, budget=budget, n_sink=sink, n_recent=recent,
                   kept=kept, k_scales=ks, v_scales=vs)
    assert fa.fa_decode_device_status() == 0 and int(new_lens[0]) == budget
    mid = old_acc[0, 0, sink:n - recent].sort(descending=True, stable=True).indices
    mid = mid[:budget - sink - recent].sort().values + sink
    want = torch.cat([torch.arange(sink, device="cuda"), mid, torch.arange(n - recent, n, device="cuda")])
    assert torch.equal(kept[0, 0].long(), want)
    assert torch.equal(acc[0, 0, :budget], old_acc[0, 0, want])
    assert not acc[0, 0, budget:].any()
    for new, old in ((k, old_k), (vs, old_vs)):
        assert torch.equal(new[0, 0, budget:], old[0, 0, budget:])
        some = torch.arange(0, budget, 997, device="cuda")
        assert torch.equal(new[0, 0, some], old[0, 0, want[some]])


def test_the_largest_budget():
    """More than any sequence holds: nothing moves, and kept is written to its end."""
    budget = 2 ** 31 - 1
    k, ks, v, vs, acc = cache(1024)
    before = [x.clone() for x in (k, ks, v, vs, acc)]
    lens, new_lens = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (777, 0))
    kept = torch.zeros(1, 1, budget, dtype=torch.int32, device="cuda")
    fa.fa_evict_kv(k, v, acc, None, lens, new_lens, budget=budget, n_sink=4, n_recent=9, kept=kept,
                   k_scales=ks, v_scales=vs)
    assert int(new_lens[0]) == 777
    assert torch.equal(kept[0, 0, :777], torch.arange(777, dtype=torch.int32, device="cuda"))
    assert torch.all(kept[0, 0, 777:] == -1)
    for x, y in zip((k, ks, v, vs, acc), before):
        assert torch.equal(x, y)
