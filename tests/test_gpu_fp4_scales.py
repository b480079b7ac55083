"""4-bit rows at the ends of their scales on the tensor-core attention: scale bytes 0 (subnormal
values), far above 128 (the tile loader's two products), 253 (the largest) and 255 (NaN).
Answers and bounds are test_gpu_fp4_attention.py's."""
import numpy as np
import pytest
import torch

from helpers import np_
from test_gpu_fp4_attention import DEV, Case
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
NOPE = 448
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def set_rows(c, x):
    """x [B][cap][512] packed into the case's cache; the scale bytes of every row."""
    lib, (B, cap, D) = lib_(), x.shape
    x = torch.tensor(x).bfloat16().to(DEV).reshape(B * cap, D).contiguous()
    slots = c.c.slots(cap).reshape(-1)
    lib.ds4a_pack_rows(c.c, x, slots)
    back = torch.empty_like(x)
    lib.ds4a_unpack_rows(c.c, back, slots)
    c.rows = np_(back).astype(np.float64).reshape(B, cap, D)
    packed = np_(c.c.attn_comp_kv.view(-1, 384)[slots.long()]).astype(np.uint8)
    # (seven blocks: word 7 of lanes 2 q holds blocks 0 .. 3 of dims 16 q .., of 2 q + 1 blocks 4 .. 6)
    word = lambda lane: packed[:, 128 + 16 * lane + 12:128 + 16 * lane + 16]  # noqa: E731
    return np.concatenate([np.concatenate([word(2 * q), word(2 * q + 1)[:, :3]], 1) for q in range(4)], 1)


@pytest.mark.parametrize("T,cluster", [(1, 1), (1, 0), (9, 0)])
def test_far_above_and_below_the_quick_path(T, cluster):
    lib = lib_()
    c = Case(4, 2, T, 2000, 64, top_k=200, rot_q=True, q_std=2.0 ** -40)
    x = np.random.default_rng(2).standard_normal(c.rows.shape)
    x[:, ::2] *= 2.0 ** 40
    x[:, 1::4] *= 2.0 ** -40
    x[:, 7::8, :NOPE:32] *= 2.0 ** 30          # (both kinds in one row)
    sb = set_rows(c, x)
    assert sb.max() > 160 and sb.min() < 100 and ((sb > 128).any(1) & (sb <= 128).any(1)).any()
    lib.ds4a_set_decode_cluster(cluster)
    try:
        c.run()
        c.check([(0, 0), (1, T - 1)])
    finally:
        lib.ds4a_set_decode_cluster(0)


@pytest.mark.parametrize("ratio,T", [(4, 1), (4, 9), (128, 1)])
def test_subnormal_rows(ratio, T):
    """Values E2M1 * 2^-127 (scale byte 0) against queries around 2^125: scores of a few, which the
    rotated dims' outputs tell."""
    pos = 2000 if ratio == 4 else 9000
    c = Case(ratio, 2, T, pos, 64, top_k=150, rot_q=True)
    rng = np.random.default_rng(3)

    def tiny(*s):
        v = rng.standard_normal(s + (512,))
        v[..., :NOPE] = (E2M1[rng.integers(0, 8, s + (NOPE,))] * rng.choice([-1, 1], s + (NOPE,))) * 2.0 ** -127
        return v

    x = tiny(*c.rows.shape[:2])
    sb = set_rows(c, x)
    assert (sb == 0).all() and np.array_equal(c.rows[..., :NOPE], x[..., :NOPE])
    bf = lambda v: torch.tensor(v).bfloat16().to(DEV)  # noqa: E731
    q = rng.standard_normal(c.q.shape) * 2.0 ** 125
    q[..., NOPE:] = 0
    c.q.copy_(bf(q))
    c.ring.copy_(bf(tiny(2, 128)))
    c.chunk.copy_(bf(tiny(2, T)))
    if T == 1:
        for b in range(2):
            c.ring[b, pos % 128] = c.chunk[b, 0]
    c.c.raw_kv.copy_(c.ring)
    c.run()
    c.check([(0, 0), (1, T - 1)])
    # (the scores matter: without them the outputs would be plain means)
    o = np_(c.out).astype(np.float64)[..., NOPE:]
    assert np.abs(o - o.mean(2, keepdims=True)).max() > 0.1


@pytest.mark.parametrize("top,byte", [(3.0, 252), (3.75, 253)])   # 3 * 2^126 = 6 * 2^125
@pytest.mark.parametrize("T", [1, 2])
def test_the_largest_scales(T, top, byte):
    """Rows that reach 3 * 2^126, the largest value there is: one among the window's."""
    c = Case(4, 2, T, 3, 64, top_k=4, rot_q=True, q_std=0.0)
    x = np.random.default_rng(4).standard_normal(c.rows.shape) * 2.0 ** 126
    x[..., NOPE:] *= 2.0 ** -126
    x[:, 0, :NOPE:16] = top * 2.0 ** 126
    x = np.clip(x, -top * 2.0 ** 126, top * 2.0 ** 126)
    sb = set_rows(c, x)
    assert (sb[[0, c.rows.shape[1]]] == byte).all() and c.rows[:, 0].max() == 3.0 * 2.0 ** 126
    c.run()
    c.check()


@pytest.mark.parametrize("T", [1, 12])
@pytest.mark.parametrize("cluster", [1, 3])
def test_a_row_of_nan(T, cluster):
    """One block of one row holds a NaN (scale byte 255): NaN for the query that lists the row,
    nothing for the others."""
    lib = lib_()
    c = Case(4, 2, T, 2000, 64, top_k=200, rot_q=True)
    t = T // 2
    row = int(c.topk_np[1, t, 140])
    for b in range(2):
        for s in range(T):
            if (b, s) != (1, t):
                c.topk_np[b, s][c.topk_np[b, s] == row] = -1
    c.topk.copy_(torch.tensor(c.topk_np))
    x = np.random.default_rng(5).standard_normal(c.rows.shape)
    x[:, row, 100] = np.nan
    sb = set_rows(c, x)
    assert (sb == 255).sum() == 2
    lib.ds4a_set_decode_cluster(cluster)
    try:
        c.run()
        c.check([(b, s) for b in range(2) for s in range(T) if (b, s) != (1, t)])
    finally:
        lib.ds4a_set_decode_cluster(0)
    assert c.out[1, t].isnan().all()
