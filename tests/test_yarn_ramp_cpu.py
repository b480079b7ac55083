"""YaRN tables for long trained contexts: the ramp of Peng et al. ("YaRN: Efficient Context Window Extension of Large
Language Models") written out pair by pair, where its upper end lies behind the last pair."""
import math

import numpy as np
import pytest

from compressed_kv_sparse_gb300 import lib
from oracle import kv
from test_abi_cpu import L  # noqa: F401  (the library fixture)

CASES = [  # n_rot, base, trained positions, factor, beta_fast, beta_slow
    (64, 1e4, 65536, 4.0, 32.0, 1.0), (64, 1e4, 131072, 8.0, 32.0, 1.0), (20, 1e4, 32768, 4.0, 32.0, 1.0),
    (128, 1e4, 1 << 20, 2.0, 32.0, 1.0), (16, 100.0, 1 << 20, 16.0, 32.0, 1.0), (64, 1e4, 131072, 8.0, 16.0, 2.0),
    (2, 1e4, 4096, 16.0, 32.0, 1.0), (4, 1e4, 4096, 16.0, 32.0, 1.0), (6, 1e4, 1 << 18, 40.0, 32.0, 1.0),
    (64, 5e5, 8192, 8.0, 32.0, 1.0), (128, 1e4, 4096, 16.0, 32.0, 1.0),
]


def angles(n_rot, base, orig, factor, fast, slow):
    """Pairs that turn more than `fast` times over the trained positions keep their angle, those that turn less than
    `slow` times get 1 / factor of it, in between it changes linearly with the pair; the ends are whole pairs, at most
    the head's dims."""
    pair = lambda turns: n_rot / 2 * math.log(orig / (2 * math.pi * turns)) / math.log(base)  # noqa: E731
    low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), n_rot - 1)
    out = []
    for i in range(n_rot // 2):
        t = base ** (-2.0 * i / n_rot)
        mixed = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        out.append((1 - mixed) * t + mixed * t / factor)
    return np.array(out)


@pytest.mark.parametrize("n_rot,base,orig,factor,fast,slow", CASES)
def test_ramp(L, n_rot, base, orig, factor, fast, slow):  # noqa: F811
    want, n = angles(n_rot, base, orig, factor, fast, slow), 200
    c, s = np.empty((n, n_rot // 2), np.float32), np.empty((n, n_rot // 2), np.float32)
    args = (base, factor, float(orig), fast, slow, 1.0)
    assert L.ds4a_rope_table_scaled(lib.SCALINGS["yarn"], *args, n_rot, n, c.ctypes.data, s.ctypes.data) == 0
    a = np.arange(n)[:, None] * want
    # (one rounding to fp32 of values up to 1; the angles, below 200, differ by 2^-50 of themselves)
    assert np.abs(c - np.cos(a)).max() <= 2.0 ** -24 + 1e-11 and np.abs(s - np.sin(a)).max() <= 2.0 ** -24 + 1e-11
    th, _ = kv.theta(n_rot, base, kind="yarn", factor=factor, orig_len=float(orig), beta_fast=fast, beta_slow=slow)
    assert np.allclose(th, want, rtol=1e-12, atol=0)


def test_a_pair_that_turns_more_than_beta_slow_times_is_not_interpolated_whole():
    n_rot, base, orig = 64, 1e4, 131072
    th = base ** (-2.0 * np.arange(32) / n_rot)
    turns = orig * th / (2 * np.pi)
    got, _ = kv.theta(n_rot, base, kind="yarn", factor=8.0, orig_len=float(orig))
    assert turns[-1] > 2 and (got[turns > 1] > th[turns > 1] / 8 * (1 + 1e-9)).all()
