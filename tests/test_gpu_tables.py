"""ds4a_block_tables against oracle/serving.py, exactly: random steps one after the other
on one pool (requests growing, ending, rolled back, the pool running out), and the sizes at
which its work split changes."""
import numpy as np
import pytest
import torch

from oracle import serving
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOK = ("tok_seq", "tok_pos", "raw_slot", "comp_slot4", "comp_slot128")


def host(pool):
    return {k: getattr(pool, k).cpu().numpy().astype(np.int64)
            for k in ("table", "held", "free_list", "state")}


def step(pool, ctx, new, cap_raw, max_tokens):
    """One call, and the oracle's from the same state; both compared whole."""
    lib = lib_()
    st = lib.StepTables(pool.rows, max_tokens, device=DEV)
    want_pool = host(pool)
    want = serving.block_tables(want_pool, ctx, new, cap_raw, max_tokens)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    lib.ds4a_block_tables(pool, t(ctx), t(new), cap_raw, st)
    torch.cuda.synchronize()
    got = host(pool)
    for k in want_pool:
        assert np.array_equal(got[k], want_pool[k]), k
    for k in ("seq_pos", "cu_len") + TOK:
        assert np.array_equal(getattr(st, k).cpu().numpy(), want[k]), k
    return st


@pytest.mark.parametrize("B,M,n_blocks,cap_raw", [(1, 4, 4, 128), (5, 6, 30, 128), (16, 9, 60, 7), (17, 9, 60, 7), (33, 9, 120, 7),
                                                  (300, 5, 1700, 1024), (1024, 3, 3300, 5),
                                                  (1025, 3, 3300, 128), (2040, 2, 3000, 128), (2048, 3, 6500, 128),
                                                  (8192, 2, 9000, 128)])
def test_steps_on_one_pool(B, M, n_blocks, cap_raw):
    lib = lib_()
    rng = np.random.default_rng(B)
    pool = lib.BlockPool(B, M, n_blocks, device=DEV)
    ctx = np.zeros(B, np.int64)
    for it in range(6 if B < 1000 else 3):
        new = rng.choice([0, 1, 1, 2, 5, 200 if B < 1000 else 9, 300 if B < 1000 else 3], B)
        ctx = ctx + new
        if it == 2:                                    # rolled back, some to the very block edge
            ctx = np.where(rng.random(B) < 0.3, np.maximum(ctx - 300, 0) // 256 * 256, ctx)
        ctx = np.where(rng.random(B) < 0.1, 0, ctx)    # ended
        ctx = np.minimum(ctx, (M + 1) * 256)           # (a few beyond the table)
        total = int(np.minimum(new, ctx).sum())
        step(pool, ctx, new, cap_raw, total + 3 if it % 2 else max(1, total - 2))
    st = pool.state.cpu().numpy()
    assert st[1] + int(pool.held.sum()) <= n_blocks and st[3] == 0
    step(pool, np.zeros(B, int), np.zeros(B, int), cap_raw, 2)       # everything given back
    assert int(pool.held.sum()) == 0 and int(pool.state[1]) == n_blocks
    assert sorted(pool.free_list.tolist()) == list(range(n_blocks))


@pytest.mark.parametrize("n_tok", [1, 3, 511, 512, 513, 1023, 1024, 1025, 70000, 400001])
def test_token_counts(n_tok):
    lib = lib_()
    M = n_tok // 256 + 2
    pool = lib.BlockPool(3, M, 2 * M, device=DEV)
    step(pool, [n_tok // 2, 0, n_tok - n_tok // 2], [n_tok // 2, 5, n_tok - n_tok // 2], 128, n_tok)
    step(pool, [n_tok // 2 + 1, 1, n_tok - n_tok // 2], [1, 1, 0], 128, 2)


def test_outputs_not_asked_for_and_full_table_of_new_tokens():
    lib = lib_()
    pool = lib.BlockPool(2, 3, 8, device=DEV)
    st = lib.StepTables(2, 8, device=DEV)
    st.tok_pos.fill_(77)
    st.c.seq_pos = st.c.cu_len = st.c.tok_seq = st.c.tok_pos = st.c.comp_slot128 = None
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    lib.ds4a_block_tables(pool, t([300, 4]), t([4, 4]), 128, st)
    torch.cuda.synchronize()
    assert pool.table.tolist() == [[0, 1, -1], [2, -1, -1]]
    assert (st.tok_pos == 77).all() and (st.tok_seq == -1).all() and st.seq_pos.tolist() == [0, 0]
    assert st.raw_slot.tolist() == [296 % 128, 297 % 128, 298 % 128, 299 % 128, 128, 129, 130, 131]
    assert st.comp_slot4.tolist() == [-1, -1, -1, 64 + 10, -1, -1, -1, 128]


def test_replayed_graph_advances_the_pool():
    """A captured step finds the lengths of each replay and carries the pool on."""
    lib = lib_()
    B, M = 16, 8
    pool = lib.BlockPool(B, M, B * M, device=DEV)
    want = lib.BlockPool(B, M, B * M, device=DEV)
    ctx = torch.zeros(B, dtype=torch.int32, device=DEV)
    new = torch.ones(B, dtype=torch.int32, device=DEV)
    st, sw = lib.StepTables(B, B, device=DEV), lib.StepTables(B, B, device=DEV)
    lib.ds4a_block_tables(pool, ctx, new, 128, st)     # (nothing to take yet)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.ds4a_block_tables(pool, ctx, new, 128, st)
    for it in range(5):
        ctx += torch.arange(B, dtype=torch.int32, device=DEV) * 23 + 1
        g.replay()
        lib.ds4a_block_tables(want, ctx, new, 128, sw)
        torch.cuda.synchronize()
        for k in ("table", "held", "free_list", "state"):
            assert torch.equal(getattr(pool, k), getattr(want, k)), (it, k)
        for k in ("seq_pos", "cu_len") + TOK:
            assert torch.equal(getattr(st, k), getattr(sw, k)), (it, k)
