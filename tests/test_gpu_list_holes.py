"""Attention over bf16 rows where a tile's usual source is not the one: lists that hold
no row for whole tiles (the rows behind the hole are attended all the same, on every
cluster size), a chunk of one token (its row is not in the ring yet)."""
import numpy as np
import pytest
import torch

import synth
from helpers import TOL, gpu_cache, np_, oracle_cache, rel_l2, to_dev, to_np
from oracle import layer as olayer
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cluster", [1, 2, 3, 0])
def test_rows_behind_a_hole(cluster):
    lib = lib_()
    shape = synth.LayerShape(ratio=4)
    p, cap = 9000, 2251
    wl = synth.Workload("holes", 7, 2, (shape,), p, "decode")
    hist = synth.cache_history(wl, 0, p + 1, comp_cap=cap)
    # scores around -450: every row close to -20 times the queries' common part
    big = torch.randn((512,), generator=torch.Generator().manual_seed(5))
    rows = 0.1 * torch.randn(hist["attn_comp_kv"].shape) - 20 * big
    hist["attn_comp_kv"] = rows.bfloat16()
    hist["raw_kv"] = (-21 * big).bfloat16().expand_as(hist["raw_kv"]).contiguous()
    q = (0.05 * torch.randn((2, 1, 64, 512)) + big).bfloat16()
    tk = torch.full((2, 1, 512), -1, dtype=torch.int32)
    rng = np.random.default_rng(1)
    for b in range(2):
        tk[b, 0, 400:] = torch.tensor(np.sort(rng.choice((p + 1) // 4, 112, replace=False)))
    gc = gpu_cache(shape, 2, cap, p + 2, hist, p + 1)
    out = torch.empty((2, 64, 512), dtype=torch.bfloat16, device="cuda")
    ws = lib.workspace(gc.workspace_bytes(lib.CALL_ATTN_DECODE, 1, 64, 512))
    lib.ds4a_set_decode_cluster(cluster)
    try:
        lib.ds4a_sparse_attn_decode(gc, p, q[:, 0].cuda().contiguous(), 64, tk[:, 0].cuda().contiguous(),
                                    512, lib.default_scale(512), out, ws)
        torch.cuda.synchronize()
    finally:
        lib.ds4a_set_decode_cluster(0)
    want = olayer.attention(oracle_cache(shape, hist, p + 1), p, np_(q), np_(tk).astype(np.int32))
    assert rel_l2(np_(out), want[:, 0]) <= TOL["bf16"]


@pytest.mark.parametrize("ratio", [0, 4, 128])
def test_chunk_of_one_token(ratio):
    """A prefill chunk of one token behind a full window: its row is in the chunk alone."""
    lib = lib_()
    shape = synth.LayerShape(ratio=ratio)
    p0 = 20000
    wl = synth.Workload("one", 3, 2, (shape,), p0, "prefill", chunk=1)
    cap = p0 // ratio + 1 if ratio else 0
    hist = synth.cache_history(wl, 0, p0, comp_cap=cap)
    inp = synth.step_inputs(wl, 0, p0, 1)
    gc = gpu_cache(shape, 2, cap, p0 + 1, hist, p0)
    d = to_dev(inp)
    chunk = torch.empty((2, 1, 512), dtype=torch.bfloat16, device="cuda")
    lib.ds4a_compress_append(gc, p0, 1, d, raw_chunk_out=chunk)
    topk, k = None, 512
    if ratio == 4:
        topk = torch.empty((2, 1, k), dtype=torch.int32, device="cuda")
        ws = lib.workspace(gc.workspace_bytes(lib.CALL_INDEX_TOPK, 1, shape.index_heads, k))
        lib.ds4a_index_topk(gc, p0, 1, d["q_idx"], d["w"], shape.index_heads, k, topk, ws)
    out = torch.empty((2, 1, 64, 512), dtype=torch.bfloat16, device="cuda")
    ws = lib.workspace(gc.workspace_bytes(lib.CALL_ATTN_PREFILL, 1, 64, k))
    lib.ds4a_sparse_attn_prefill_chunk(gc, p0, 1, d["q"], 64, chunk, topk, k,
                                       lib.default_scale(512), out, ws)
    torch.cuda.synchronize()
    want = olayer.prefill_chunk(oracle_cache(shape, hist, p0), p0, to_np(inp), k)[0]
    assert rel_l2(np_(out), want) <= TOL["bf16"]
