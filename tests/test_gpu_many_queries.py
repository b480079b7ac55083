"""Chunks of more than 65,535 queries in a call (a grid's second and third dimension end there), on
the kernels that take a block per query: the last sequences' results are those of a smaller call."""
import pytest
import torch

from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(ratio, B, T, H, D, dt, p0):
    lib = lib_()
    c = lib.LayerCache(ratio=ratio, head_dim=D, n_rot=8, batch=B, comp_cap=(p0 + T) // 4 + 1 if ratio else 0,
                       dtype="f32" if dt is torch.float32 else "bf16", base=10000.0, rope_max_pos=p0 + T,
                       index_dim=32, index_rot=8, cap_raw=4, device=DEV)
    c.n_tokens = p0 + T
    return c


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ratio", [0, 4])
def test_attention(ratio, dt):
    lib = lib_()
    B, T, H, D, p0, k = 17, 4000, 3, 16, 8, 4
    g = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=g).to(DEV, dt)  # noqa: E731
    q, chunk, ring, rows = rn(B, T, H, D), rn(B, T, D), rn(B, 4, D), rn(B, (p0 + T) // 4 + 1, D)
    tk = torch.randint(-1, 2, (B, T, k), generator=g, dtype=torch.int32).to(DEV)

    def run(b0, b1):
        c = make(ratio, b1 - b0, T, H, D, dt, p0)
        c.raw_kv.copy_(ring[b0:b1])
        if ratio:
            c.attn_comp_kv.copy_(rows[b0:b1])
        out = torch.full((b1 - b0, T, H, D), 9.0, dtype=dt, device=DEV)
        ws = lib.workspace(c.workspace_bytes(lib.CALL_ATTN_PREFILL, T, H, k))
        lib.ds4a_sparse_attn_prefill_chunk(c, p0, T, q[b0:b1], H, chunk[b0:b1], tk[b0:b1] if ratio else None,
                                           k, 0.25, out, ws)
        torch.cuda.synchronize()
        return out

    whole = run(0, B)
    assert B * T > 65535
    for b0, b1 in ((0, 2), (15, 17)):
        assert torch.equal(whole[b0:b1], run(b0, b1))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_top_k(dt):
    lib = lib_()
    B, T, H, p0, k = 17, 4000, 2, 600, 8
    g = torch.Generator().manual_seed(2)
    rn = lambda *s: torch.randn(s, generator=g).to(DEV, dt)  # noqa: E731
    q, w, keys = rn(B, T, H, 32), rn(B, T, H), rn(B, (p0 + T) // 4 + 1, 32)

    def run(b0, b1):
        c = make(4, b1 - b0, T, H, 16, dt, p0)
        c.index_comp_kv.copy_(keys[b0:b1])
        lib.ds4a_index_norms(c)
        out = torch.full((b1 - b0, T, k), -7, dtype=torch.int32, device=DEV)
        ws = lib.workspace(c.workspace_bytes(lib.CALL_INDEX_TOPK, T, H, k))
        lib.ds4a_index_topk(c, p0, T, q[b0:b1], w[b0:b1], H, k, out, ws)
        torch.cuda.synchronize()
        return out

    whole = run(0, B)
    assert (whole >= 0).all()
    for b0, b1 in ((0, 2), (15, 17)):
        assert torch.equal(whole[b0:b1], run(b0, b1))
