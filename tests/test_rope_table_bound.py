"""The rotation table against 60 digits (no GPU needed)."""
import numpy as np
import pytest

import decode_step_kv_gb300 as fa

mp = pytest.importorskip("mpmath")


@pytest.mark.parametrize("rot", [16, 128, 256])
@pytest.mark.parametrize("base", [2.0, 10000.0, 500000.0])
@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 13.0), ("ntk", 8.0), ("yarn", 8.0)])
def test_every_rate_is_within_2_to_the_minus_54_turns(rot, base, scaling, factor):
    """A rate is a power of at most 1 radian, within a step (2^-53 of it), over 2 pi: 2^-55.6 turns.  The quotient
    adds half a step, 2^-56, and 2 pi as a 64-bit float 2^-57; where YaRN slows a pair or NTK raises the base
    the rates are smaller by more than their operations add."""
    table, _ = fa.fa_rope_table(rot, base, scaling=scaling, factor=factor, original_len=8192, device="cpu")
    got = table.numpy().view(np.uint64)
    with mp.workdps(60):
        b, f = mp.mpf(base), mp.mpf(factor)
        if scaling == "ntk":
            b *= f ** (mp.mpf(rot) / (rot - 2))
        pair = [rot * mp.log(8192 / (turns * 2 * mp.pi)) / (2 * mp.log(b)) for turns in (32, 1)]
        lo, hi = max(mp.floor(pair[0]), 0), min(mp.ceil(pair[1]), rot - 1)
        for j in range(rot // 2):
            rate = b ** (mp.mpf(-2 * j) / rot)
            if scaling == "linear":
                rate /= f
            if scaling == "yarn":
                slow = min(max((j - lo) / max(hi - lo, mp.mpf("0.001")), 0), 1)
                rate = rate * (1 - slow) + rate / f * slow
            assert abs(mp.mpf(int(got[j])) / mp.mpf(2) ** 64 - rate / (2 * mp.pi)) < mp.mpf(2) ** -54
