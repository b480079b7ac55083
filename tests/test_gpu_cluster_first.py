"""ds4a_decode_cluster_size as the first call of a process: it answers, and the decode calls
behind it use, what they use in a process that has launched before."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import sys; sys.path.insert(0, '.')
import torch
from compressed_kv_sparse_gb300 import lib
lib.load()


def sizes():
    out = []
    for B in (1, 2, 3, 8, 32):
        for fp4 in (0, lib.FP4_ROWS):
            for n in (20000, 131072, 300000):
                c = lib.LayerCache(ratio=128, head_dim=512, n_rot=64, batch=B, comp_cap=n // 128,
                                   base=160000.0, dtype='bf16', rope_max_pos=8, qat=fp4)
                c.n_tokens = n
                out.append(lib.ds4a_decode_cluster_size(c, 64, 1))
    return out


first = sizes() if sys.argv[1] == 'first' else None
for fp4 in (0, lib.FP4_ROWS):
    c = lib.LayerCache(ratio=128, head_dim=512, n_rot=64, batch=2, comp_cap=16, base=160000.0,
                       dtype='bf16', rope_max_pos=2048, qat=fp4)
    c.n_tokens = 2000
    q = torch.zeros((2, 64, 512), dtype=torch.bfloat16, device='cuda')
    ws = lib.workspace(c.workspace_bytes(lib.CALL_ATTN_DECODE, 1, 64, 1))
    lib.ds4a_sparse_attn_decode(c, 1999, q, 64, None, 1, 0.1, torch.empty_like(q), ws)
torch.cuda.synchronize()
print('sizes', first or sizes())
"""


def test_asked_before_the_first_launch():
    out = []
    for when in ("first", "later"):
        r = subprocess.run([sys.executable, "-c", CODE, when], capture_output=True, text=True, timeout=180)
        assert r.returncode == 0, r.stderr[-2000:]
        out.append(r.stdout.split("sizes")[1])
    assert out[0] == out[1]
