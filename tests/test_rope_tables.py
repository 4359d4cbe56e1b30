"""Frequency tables of rope_append for trained lengths of any size: which pairs yarn slows."""
import math

import numpy as np
import pytest

from compressed_sparse_kv_fp32_b200 import adamas


@pytest.mark.parametrize("rot,base", [(128, 10000.0), (64, 10000.0), (128, 500000.0), (96, 1000.0), (6, 10000.0)])
@pytest.mark.parametrize("length", [512, 4096, 32768, 63000, 65536, 131072, 1 << 20, 1 << 30])
def test_yarn_slows_pairs_by_their_own_turns(rot, base, length):
    factor = 16.0
    plain = adamas.rope_frequencies(rot, base, device="cpu")[0].double().numpy()
    yarn = adamas.rope_frequencies(rot, base, scaling="yarn", factor=factor, original_len=length, device="cpu")[0].double().numpy()
    turns = length * base ** (-np.arange(0, rot, 2) / rot) / (2 * math.pi)
    # pair number j turns 32 (once) at this place: base^(-2j / rot) length / 2 pi = 32 (1)
    fast, slow = (rot * math.log(length / (2 * math.pi * t), base) / 2 for t in (32.0, 1.0))
    lo, hi = max(0, math.floor(fast)), math.ceil(slow)
    assert hi > lo and hi <= 2 * rot     # the ramp may end behind the last pair
    slowed = np.clip((np.arange(rot // 2) - lo) / (min(hi, rot - 1) - lo), 0, 1) if min(hi, rot - 1) > lo else np.zeros(rot // 2)
    # 2^-50: the powers' rounding; a unit of the table is 2^-64 turns
    assert np.allclose(yarn, plain * (1 - slowed) + plain / factor * slowed, rtol=2.0 ** -48, atol=2.0)
    # as the function says: the fast ones as trained, only those below one turn by the whole factor
    ratio = yarn / plain
    assert np.allclose(ratio[turns > 33 * base ** (2 / rot)], 1.0, rtol=1e-9)
    assert (ratio[turns >= 1.0] > 1.0 / factor + 1e-9).all()


def test_yarn_at_a_trained_length_of_131072():
    """The last of 64 pairs turns 2.41 times: the ramp, from pair 45 to 70, has it at 18 / 25."""
    plain = adamas.rope_frequencies(128, device="cpu")[0].double().numpy()
    yarn = adamas.rope_frequencies(128, scaling="yarn", factor=32.0, original_len=131072, device="cpu")[0].double().numpy()
    assert np.isclose(yarn[63] / plain[63], 7 / 25 + 18 / 25 / 32, rtol=1e-9)
    assert np.allclose(yarn[:46] / plain[:46], 1.0, rtol=1e-9) and (np.diff(yarn[45:] / plain[45:]) < 0).all()
