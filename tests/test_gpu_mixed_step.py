"""A step whose rows have different numbers of new tokens: tables and norms over all of them, the
other calls for the decoding rows and for the chunk's row on caches of these rows alone, at once on
two streams. Every row is compared with the same step on a contiguous cache of its own."""
import numpy as np
import pytest
import torch

from helpers import np_, rel_l2
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("chunk_first", [False, True])
@pytest.mark.parametrize("T", [2, 40, 200])
def test_decoding_rows_beside_a_chunk(T, chunk_first):
    lib = lib_()
    H, D, k, base, maxp, M, nb = 64, 512, 64, 160000.0, 1100, 5, 18
    old, new = ([150, 700, 301], [T, 1, 1]) if chunk_first else ([700, 301, 150], [1, 1, T])
    ic, d0 = (0, 1) if chunk_first else (2, 0)      # the chunk's row, the first decoding one
    g = torch.Generator().manual_seed(T)
    rn = lambda *s: torch.randn(s, generator=g).to(DEV).bfloat16()  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    pool, st = lib.BlockPool(3, M, nb, device=DEV), lib.StepTables(3, sum(new) + 3, device=DEV)
    kw = dict(ratio=4, head_dim=D, n_rot=64, dtype="bf16", base=base, rope_max_pos=maxp, index_dim=128,
              index_rot=64, device=DEV, qat=lib.FP4_ROWS | lib.Q_ROTATED, comp_cap=M * 64)
    c = lib.LayerCache(batch=3, block_table=pool.table, n_blocks=nb, **kw)
    c.set_seq_pos(st.seq_pos)
    lib.ds4a_block_tables(pool, i32(old), i32([0, 0, 0]), 128, st)
    lib.ds4a_pack_rows(c, rn(nb * 64, D))
    c.index_comp_kv.copy_(rn(*c.index_comp_kv.shape))
    for t in (c.raw_kv, c.attn_state_kv, c.attn_state_score, c.index_state_kv, c.index_state_score):
        t.copy_(rn(*t.shape))
    c.n_tokens = max(old)
    lib.ds4a_index_norms(c)

    # every row as a cache of its own, before the step
    alone = []
    for b in range(3):
        r, n = lib.LayerCache(batch=1, **kw), old[b] // 4
        at = c.slots(n)[b].long()
        r.attn_comp_kv[0, :n] = c.attn_comp_kv.view(-1, c.attn_comp_kv.shape[-1])[at]
        r.index_comp_kv[0, :n] = c.index_comp_kv.view(-1, 128)[at]
        for m in ("raw_kv", "attn_state_kv", "attn_state_score", "index_state_kv", "index_state_score"):
            getattr(r, m).copy_(getattr(c, m)[b:b + 1])
        r.n_tokens = old[b]
        lib.ds4a_index_norms(r)
        alone.append(r)

    w = {"ape_attn": rn(8, D), "gamma_attn": rn(D), "ape_idx": rn(8, 128), "gamma_idx": rn(128)}
    x = {"attn_cand": rn(sum(new), D), "attn_score": rn(sum(new), D), "idx_cand": rn(sum(new), 128),
         "idx_score": rn(sum(new), 128)}
    proj, gq, gk = rn(sum(new), (H + 1) * D), rn(D), rn(D)
    q_idx, wi = rn(sum(new), 64, 128), rn(sum(new), 64)

    def run(cache, tok, B, pos, slots, chunk, stream, whole):
        """Norms (slots number the rows of the cache `whole`), append, top-k and attention of
        tokens `tok` (B rows, as many each)."""
        n, T = tok.stop - tok.start, (tok.stop - tok.start) // B
        q = torch.empty((n, H, D), dtype=torch.bfloat16, device=DEV)
        out, topk = torch.empty_like(q), torch.empty((n, k), dtype=torch.int32, device=DEV)
        p = proj[tok]
        call = lib.CALL_ATTN_DECODE if chunk is None else lib.CALL_ATTN_PREFILL
        ws = [lib.workspace(cache.workspace_bytes(a, T, 64, k)) for a in (lib.CALL_INDEX_TOPK, call)]
        last = cache.n_tokens + T
        with torch.cuda.stream(stream):
            lib.ds4a_norm_rope(whole, pos, q=p[:, :H * D].view(n, H, D), gamma_q=gq, q_out=q,
                               kv=p[:, H * D:], gamma_kv=gk, kv_out=chunk,
                               slots=slots if chunk is None else None, rot_q=True)
            lib.ds4a_compress_append_lanes(cache, last - T, T, lib.LANE_ATTN | lib.LANE_INDEX,
                                           {**w, **{m: t[tok].view(B, T, -1) for m, t in x.items()}})
            cache.n_tokens = last
            lib.ds4a_index_topk(cache, last - T, T, q_idx[tok], wi[tok], 64, k, topk, ws[0])
            if chunk is None:
                lib.ds4a_sparse_attn_decode(cache, last - 1, q, H, topk, k, lib.default_scale(D), out, ws[1])
            else:
                lib.ds4a_sparse_attn_prefill_chunk(cache, last - T, T, q, H, chunk, topk, k,
                                                   lib.default_scale(D), out, ws[1])
        return out, topk, ws

    ctx = [a + b for a, b in zip(old, new)]
    lib.ds4a_block_tables(pool, i32(ctx), i32(new), 128, st)
    cu = st.cu_len.tolist()
    assert st.tok_pos[:2 + T].tolist() == sum([list(range(a, a + b)) for a, b in zip(old, new)], [])
    chunk = torch.empty((T, D), dtype=torch.bfloat16, device=DEV)
    dec, pre = c.rows(d0, d0 + 2), c.rows(ic, ic + 1)
    dec.n_tokens, pre.n_tokens = 700, 150
    td, tc = slice(cu[d0], cu[d0 + 2]), slice(cu[ic], cu[ic + 1])
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    a = run(dec, td, 2, st.tok_pos[td], st.raw_slot[td], None, streams[0], c)
    b = run(pre, tc, 1, st.tok_pos[tc], None, chunk, streams[1], pre)
    torch.cuda.synchronize()

    for i, r in enumerate(alone):
        tok, n = slice(cu[i], cu[i + 1]), new[i]
        pos = torch.arange(old[i], old[i] + n, dtype=torch.int32, device=DEV)
        ch = None if n == 1 else torch.empty((n, D), dtype=torch.bfloat16, device=DEV)
        out, topk, _ = run(r, tok, 1, pos, pos % 128 if n == 1 else None, ch, streams[0], r)
        torch.cuda.synchronize()
        got = (b[0], b[1]) if i == ic else (a[0][i - d0:i - d0 + 1], a[1][i - d0:i - d0 + 1])
        assert torch.equal(got[1], topk), i
        assert rel_l2(np_(got[0]), np_(out)) <= 2 ** -7, i     # (other cluster sizes)
        for m in ("raw_kv", "attn_state_kv", "attn_state_score", "index_state_kv", "index_state_score"):
            assert torch.equal(getattr(c, m)[i], getattr(r, m)[0]), (i, m)
        rows = ctx[i] // 4
        at = c.slots(rows)[i].long()
        vals = [torch.empty((rows, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        lib.ds4a_unpack_rows(c, vals[0], at.int())
        lib.ds4a_unpack_rows(r, vals[1])
        assert torch.equal(*vals) and np.isfinite(np_(vals[0])).all()
        assert torch.equal(c.index_comp_kv.view(-1, 128)[at], r.index_comp_kv[0, :rows])
