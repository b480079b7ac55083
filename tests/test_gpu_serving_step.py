"""The serving operators as a step runs them: tables from request lengths, norms with the
insert, append of the compressor lanes into 4-bit rows, top-k, attention.

A paged cache with 4-bit rows is compared with a contiguous cache in the layer's own type
that goes through the same steps: the 4-bit rows must be the quantised fp32 rows of the
compressor, and the attention the one over the values that they stand for."""
import numpy as np
import pytest
import torch

import synth
from helpers import np_
from oracle import serving
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV = "cuda"
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def rows_close(got, pre, rot, dtype):
    """got: values read back; pre: the compressor's rows rounded to the type [n][D]. Where
    the row is exact in the type (fp32) the codes are those of the row, but for values whose
    fp32 differs in the last places between two compilations of the pooling; for bf16 the
    row was rounded first, half a step, so a code may be the neighbouring one."""
    nope = got.shape[1] - rot
    x = pre.astype(np.float64)
    blk = np.abs(x[:, :nope]).reshape(len(x), -1, 16).max(-1)
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20
    # in units of 2^k the block's largest value a is above 3. A value x in [4, 6] is off by
    # min(x - 4, 6 - x) <= x / 5 <= a / 5 (equal at x = 5); one below 4 by at most 1/2 < a / 6
    tol = np.repeat(blk, 16, -1) * (1 / 5 + 2 * u) * (1 + 4 * u)
    assert (np.abs(got[:, :nope] - x[:, :nope]) <= tol + 1e-30).all()
    same = serving.quantise_row(x, rot, "f32")[:, :nope]
    assert (got[:, :nope] != same).mean() <= (0.05 if dtype == "bf16" else 1e-3)
    assert np.abs(got[:, nope:] - x[:, nope:]).max() <= 2 * u * np.abs(x[:, nope:]).max()


@pytest.mark.parametrize("ratio,D,dtype", [(4, 512, "bf16"), (128, 512, "bf16"), (4, 128, "f32"),
                                           (128, 1024, "f32"), (4, 512, "f32")])
@pytest.mark.parametrize("T", [1, 150])
def test_append_emits_4_bit_rows(ratio, D, dtype, T):
    lib = lib_()
    shape = synth.LayerShape(ratio=ratio, head_dim=D, index_dim=32, index_heads=2, n_heads=4, top_k=8,
                             dtype=dtype)
    B, p0 = 3, 1023 if T == 1 else 500
    cap = (p0 + T) // ratio + 2
    cap = -(-cap // (256 // ratio)) * (256 // ratio)
    wl = synth.Workload("fp4a", 5, B, (shape,), p0, "decode" if T == 1 else "prefill")
    hist = synth.cache_history(wl, 0, p0, comp_cap=cap)
    inp = {k: v.to(DEV).contiguous() for k, v in synth.step_inputs(wl, 0, p0, T).items()}
    caches = []
    mb = cap // (256 // ratio)
    table = torch.randperm(B * mb + 2, generator=torch.Generator().manual_seed(1))[:B * mb]
    table = table.int().view(B, mb).to(DEV)
    for kw in (dict(qat=0), dict(qat=lib.FP4_ROWS), dict(qat=lib.FP4_ROWS, block_table=table,
                                                         n_blocks=B * mb + 2)):
        c = lib.LayerCache(ratio=ratio, head_dim=D, n_rot=64, batch=B, comp_cap=cap, dtype=dtype,
                           base=shape.rope_base, rope_max_pos=p0 + T + 1, index_dim=32, index_rot=32,
                           device=DEV, **kw)
        c.load_state({k: v.to(DEV) for k, v in hist.items()}, p0)
        chunk = None if T == 1 else torch.empty((B, T, D), dtype=TD[dtype], device=DEV)
        lib.ds4a_compress_append(c, p0, T, inp, raw_chunk_out=chunk)
        caches.append(c)
    torch.cuda.synchronize()
    n0, n1 = p0 // ratio, (p0 + T) // ratio
    assert n1 > n0
    vals = []
    for c in caches[1:]:
        v = torch.empty((B * n1, D), dtype=TD[dtype], device=DEV)
        lib.ds4a_unpack_rows(c, v, c.slots(n1).reshape(-1))
        vals.append(np_(v).astype(np.float64).reshape(B, n1, D))
    assert np.array_equal(vals[0], vals[1])
    old = np_(hist["attn_comp_kv"])[:, :n0].reshape(-1, D)
    assert np.array_equal(vals[0][:, :n0].reshape(-1, D), serving.quantise_row(old, 64, dtype))
    rows_close(vals[0][:, n0:].reshape(-1, D), np_(caches[0].attn_comp_kv)[:, n0:n1].reshape(-1, D), 64,
               dtype)
    for name in ("raw_kv", "attn_state_kv", "attn_state_score", "index_comp_kv", "index_state_kv",
                 "index_state_score", "index_norm_max"):
        a = getattr(caches[0], name)
        if a is not None:
            assert torch.equal(a, getattr(caches[1], name)), name


@pytest.mark.parametrize("captured", [False, True])
def test_decode_steps_of_a_serving_loop(captured):
    """Steps of a ragged c4a batch that lives in a pool: requests of other lengths,
    one that starts, blocks taken as they are needed; every step's attention against
    fp64 over what the caches hold. Captured: one graph, replayed for every step."""
    from oracle.attention import comp_row_ids
    from oracle.rope import rope_tail
    lib = lib_()
    B, H, D, k, steps, base = 4, 64, 512, 64, 12, 160000.0
    start = [250, 0, 1000, 511]
    maxp, M = 1100, 5
    pool = lib.BlockPool(B, M, 18, device=DEV)
    st = lib.StepTables(B, B, device=DEV)
    c = lib.LayerCache(ratio=4, head_dim=D, n_rot=64, batch=B, comp_cap=M * 64, dtype="bf16", base=base,
                       rope_max_pos=maxp, index_dim=128, index_rot=64, device=DEV,
                       qat=lib.FP4_ROWS | lib.Q_ROTATED, block_table=pool.table, n_blocks=18)
    c.set_seq_pos(st.seq_pos)
    ctx = torch.tensor(start, dtype=torch.int32, device=DEV)
    one = torch.ones(B, dtype=torch.int32, device=DEV)
    lib.ds4a_block_tables(pool, ctx, torch.zeros_like(one), 128, st)   # blocks of the histories
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g).to(DEV).bfloat16()  # noqa: E731
    n = max(start) // 4
    lib.ds4a_pack_rows(c, rn(B * n, D), c.slots(n).reshape(-1))        # (unheld entries: dropped)
    c.raw_kv.copy_(rn(B, 128, D))
    c.index_comp_kv.copy_(rn(*c.index_comp_kv.shape))
    c.n_tokens = max(start)
    lib.ds4a_index_norms(c)
    w = {"ape_attn": rn(8, D), "gamma_attn": rn(D), "ape_idx": rn(8, 128), "gamma_idx": rn(128)}
    x = {"attn_cand": rn(B, 1, D), "attn_score": rn(B, 1, D), "idx_cand": rn(B, 1, 128),
         "idx_score": rn(B, 1, 128), **w}
    proj, gq, gk = rn(B, (H + 1) * D), rn(D), rn(D)
    q_idx, wi = rn(B, 1, 64, 128), rn(B, 1, 64)
    q = torch.empty((B, H, D), dtype=torch.bfloat16, device=DEV)
    topk = torch.empty((B, k), dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    c.n_tokens = maxp - 1                       # host bound of every position of the loop
    wk = lib.workspace(c.workspace_bytes(lib.CALL_INDEX_TOPK, 1, 64, k))
    wa = lib.workspace(c.workspace_bytes(lib.CALL_ATTN_DECODE, 1, H, k))

    def step():
        lib.ds4a_block_tables(pool, ctx, one, 128, st)
        lib.ds4a_norm_rope(c, st.tok_pos, q=proj[:, :H * D].view(B, H, D), gamma_q=gq, q_out=q,
                           kv=proj[:, H * D:], gamma_kv=gk, slots=st.raw_slot, rot_q=True)
        c.n_tokens = maxp - 1
        lib.ds4a_compress_append_lanes(c, maxp - 1, 1, lib.LANE_ATTN | lib.LANE_INDEX, x)
        c.n_tokens = maxp
        lib.ds4a_index_topk(c, maxp - 1, 1, q_idx, wi, 64, k, topk, wk)
        lib.ds4a_sparse_attn_decode(c, maxp - 1, q, H, topk, k, lib.default_scale(D), out, wa)

    graph = None
    for it in range(steps):
        ctx += 1
        for t in (proj, q_idx, *(x[m] for m in ("attn_cand", "attn_score", "idx_cand", "idx_score"))):
            t.copy_(rn(*t.shape))
        torch.cuda.synchronize()
        if captured and graph is None:
            keep = [t.clone() for t in (pool.table, pool.held, pool.free_list, pool.state)]
            s = torch.cuda.Stream()             # (first calls set attributes: outside the capture)
            with torch.cuda.stream(s):
                step()
            s.synchronize()
            for t, v in zip((pool.table, pool.held, pool.free_list, pool.state), keep):
                t.copy_(v)
            c.attn_state_score.fill_(float("-inf"))
            c.index_state_score.fill_(float("-inf"))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if captured:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        pos = np.array(start) + it
        assert st.tok_pos.tolist() == pos.tolist() and st.seq_pos.tolist() == pos.tolist()
        assert pool.held.tolist() == [-(-(int(p) + 1) // 256) for p in pos]
        # the norms
        xq = np_(proj).astype(np.float64).reshape(B, H + 1, D)
        qr = serving.norm_rope(xq[:, :H], np_(gq), pos, base, 64, True)
        assert np.abs(np_(q) - qr).max() <= 2.0 ** -8 * np.abs(qr).max()
        kr = serving.norm_rope(xq[:, H], np_(gk), pos, base, 64, True)
        ring = np_(c.raw_kv).astype(np.float64)
        for b in range(B):
            assert np.abs(ring[b, pos[b] % 128] - kr[b]).max() <= 2.0 ** -8 * np.abs(kr[b]).max()
        # the attention, over what the caches hold now
        vals = torch.empty((18 * 64, D), dtype=torch.bfloat16, device=DEV)
        lib.ds4a_unpack_rows(c, vals)
        vals, tb = np_(vals).astype(np.float64), pool.table.cpu().numpy()
        got, lists = np_(out).astype(np.float64), topk.cpu().numpy()
        for b in range(B):
            p = int(pos[b])
            ids = comp_row_ids(4, p, maxp // 4, lists[b])
            assert len(ids) == min(k, (p + 1) // 4)
            rows = [vals[tb[b, i // 64] * 64 + i % 64] for i in ids]
            win = [ring[b, s % 128] for s in range(max(0, p - 127), p + 1)]
            K = np.array(win + rows)
            s = np_(q[b]).astype(np.float64) @ K.T / np.sqrt(D)
            e = np.exp(s - s.max(-1, keepdims=True))
            o = rope_tail(e / e.sum(-1, keepdims=True) @ K, p, base, 64, inverse=True)
            assert np.linalg.norm(got[b] - o) <= 6e-3 * np.linalg.norm(o), (it, b)
