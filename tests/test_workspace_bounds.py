"""A workspace sized for a server's largest step serves its smaller ones (host only)."""
import functools
import itertools

import pytest

from decode_step_kv_gb300 import binding as fa

BATCH = [1, 4, 16, 32, 64, 200]
CAPACITY = [16, 100, 512, 1040, 2048, 8192, 32768, 131072]
QUERIES = [1, 2, 3, 4, 6, 8, 12, 13, 16, 17, 25, 32, 48, 49, 100, 256]


def steps(sizes):
    """Pairs (smaller, larger) of neighbouring sizes along one axis."""
    for at in itertools.product(*(range(len(x)) for x in sizes)):
        for axis in range(len(sizes)):
            if at[axis]:
                less = list(at)
                less[axis] -= 1
                yield tuple(x[i] for x, i in zip(sizes, less)), tuple(x[i] for x, i in zip(sizes, at))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("Hkv,G", [(2, 1), (8, 3), (1, 4), (4, 8)])
@pytest.mark.parametrize("sms", [152, 148])
def test_int4_workspace_grows_with_every_size(D, Hkv, G, sms):
    @functools.cache
    def size(b, cap, tq, weights):
        return fa.fa_decode_int4_workspace_size(b, tq, G * Hkv, Hkv, D, cap, weights, sms)
    for less, more in steps([BATCH, CAPACITY, QUERIES]):
        assert 0 < size(*less, False) <= size(*more, False), (less, more)
        assert size(*less, True) <= size(*more, True), (less, more)
        assert size(*more, False) <= size(*more, True), more


def test_a_longer_caches_workspace_serves_a_shorter_one():
    """The plan of 512 tokens has more partial slots than that of 1024."""
    assert (fa.fa_decode_int4_workspace_size(64, 3, 24, 8, 128, 512, False, 152)
            <= fa.fa_decode_int4_workspace_size(64, 3, 24, 8, 128, 1024, False, 152))


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("Hkv,G", [(2, 1), (8, 3), (4, 8)])
def test_weights_workspace_grows_with_every_size(D, Hkv, G):
    @functools.cache
    def size(b, cap, tq):
        return fa.fa_decode_weights_workspace_size(b, tq, G * Hkv, Hkv, D, cap, 152)
    for less, more in steps([BATCH, CAPACITY, QUERIES]):
        assert 0 < size(*less) <= size(*more), (less, more)
