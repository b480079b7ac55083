"""What the calls refuse or accept on the host, by the returned status only (nothing is
launched: every case ends at a check)."""
import ctypes

from compressed_kv_sparse_gb300 import lib
from test_abi_cpu import L, _fake_cache  # noqa: F401  (L: the library fixture)

FAKE = 0x1000


def cache(**kw):
    c = _fake_cache()
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def append(L, c):
    return L.ds4a_compress_append(ctypes.byref(c), 9, 1, *([FAKE] * 9), None, None)


def test_the_flag_for_ready_queries(L):
    assert append(L, cache(qat=lib.Q_READY)) == -4       # past the cache's checks (position)
    assert append(L, cache(qat=lib.Q_READY | lib.Q_ROTATED | lib.FP4_ROWS)) == -4
    assert append(L, cache(qat=lib.Q_READY << 1)) == -1
