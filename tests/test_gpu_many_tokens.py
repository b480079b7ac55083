"""ds4a_paged_attn_decode on packed tokens whose rows (token times heads) pass 2^32."""
import pytest
import torch

from kv_step import Step, check
from test_gpu_paged_attn import run
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype,D", [("bf16", 8), ("f32", 2)])
def test_rows_beyond_32_bits(dtype, D):
    """The first sequence brings more tokens than max_new, of which the first one alone is computed; the rows of the
    others, whole in one block and divided, lie behind 2^32."""
    lib, H, K, first = lib_(), 1024, 32, 1 << 22
    step = Step(lib, 31, [100, 3000], [1, 1], H, K, D, dtype)
    c, cu = step.on_gpu()
    check(step, *run(step, c, cu), 1 / D ** 0.5)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < (first + 2) * H * (2 * D * step.q.element_size() + 4) + (4 << 30):
        pytest.skip("queries and outputs do not fit")
    q = torch.empty((first + 2, H, D), dtype=step.q.dtype, device=DEV)
    out, lse = torch.empty_like(q), torch.empty((first + 2, H), device=DEV)
    q[first:] = step.q.to(DEV)
    q[:2], out[:2], out[first:], lse[:2] = 1.0, 77.0, 77.0, 77.0
    wide = lib.KvCache(head_dim=D, n_kv_heads=K, batch=3, block_table=torch.cat([c.block_table[1:], c.block_table]),
                       n_blocks=step.nb, dtype=dtype, k=c.k, v=c.v)
    wide.set_seq_pos(torch.tensor([5, 100, 3000], dtype=torch.int32, device=DEV))
    ws = lib.workspace(wide.attn_workspace_bytes(H), DEV)
    cu = torch.tensor([0, first, first + 1, first + 2], dtype=torch.int32, device=DEV)
    lib.ds4a_paged_attn_decode(wide, q, out, ws, cu_len=cu, lse=lse)
    assert lib.ds4a_workspace_status(ws) == 0
    assert (out[1] == 77).all() and (lse[1] == 77).all() and not (out[0] == 77).any()
    check(step, out[first:], lse[first:], 1 / D ** 0.5)
    del q, out, lse
    torch.cuda.empty_cache()
