"""ds4a_kv_append refuses queries that would be rotated into keys or values that other threads still read (CPU: the
check is made on the host; what it lets through is not launched without a GPU)."""
import ctypes

import pytest

from test_abi_cpu import L  # noqa: F401  (the library fixture)
from test_kv_abi_cpu import FAKE, cache

BIG, KV, Q = 1 << 24, 512, 512            # rows of 4 heads of 128 bf16 elements: 1,024 bytes


def call(L, k, v, q_out, n=3, ks=KV, vs=KV):
    return L.ds4a_kv_append(ctypes.byref(cache()), n, FAKE, FAKE, k, ks, v, vs, BIG // 2, Q, 4, q_out, None)


@pytest.mark.parametrize("at", [0, 2, -2, 3 * 1024 - 2, -(3 * 1024 - 2), 1024])
def test_queries_into_keys_or_values(L, at):  # noqa: F811
    far = BIG + (1 << 20)
    assert call(L, BIG, far, BIG + at) == -1 and call(L, far, BIG, BIG + at) == -1


def test_queries_into_strided_rows(L):  # noqa: F811
    far = BIG + (1 << 20)
    for at in (0, 1022, 6000, 2 * 6000 + 1022, -(3 * 1024 - 2), 1024 + 6000 - 3 * 1024 - 1024 + 2):
        assert call(L, BIG, far, BIG + at, ks=3000) == -1, at
        assert call(L, far, BIG, BIG + at, vs=3000) == -1, at
    # one token: rows side by side in a projection's output
    assert call(L, BIG + 1024, BIG + 2048, BIG + 2, n=1) == -1 and call(L, BIG + 1024, BIG + 2048, BIG + 2046, n=1) == -1


def test_queries_beside_them_are_not_refused(L):  # noqa: F811
    """Behind the last row, before the first, in a gap that holds them all. (Without a GPU the launch fails: -6.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the call would launch on addresses that are none")
    far = BIG + (1 << 20)
    for at, ks in ((3 * 1024, KV), (-3 * 1024, KV), (2 * 6000 + 1024, 3000), (1024, 2048), (4096 + 1024, 2048)):
        assert call(L, BIG, far, BIG + at, ks=ks) not in (0, -1, -2, -5), (at, ks)
    assert call(L, BIG + 1024, BIG + 2048, BIG, n=1) not in (0, -1, -2, -5)
