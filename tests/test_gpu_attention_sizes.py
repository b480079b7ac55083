"""Attention at head sizes whose shared-memory tiles hold an odd number of rows (D 192 and
others): fp32 layers on the CUDA-core path against the oracle."""
import pytest
import torch

import synth
from helpers import TOL, gpu_cache, np_, oracle_cache, rel_l2, to_dev, to_np
from oracle import layer as olayer
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,H,T", [(192, 5, 1), (192, 5, 9), (148, 3, 1), (600, 1, 3)])
def test_attention_of_odd_tiles(D, H, T):
    lib = lib_()
    shape = synth.LayerShape(ratio=128, head_dim=D, n_heads=H, dtype="f32")
    p0 = 900
    wl = synth.Workload("odd", D, 2, (shape,), p0, "decode" if T == 1 else "prefill")
    cap = (p0 + T) // 128 + 1
    hist = synth.cache_history(wl, 0, p0, comp_cap=cap)
    inp = synth.step_inputs(wl, 0, p0, T)
    gc, d = gpu_cache(shape, 2, cap, p0 + T + 1, hist, p0), to_dev(inp)
    out = torch.empty((2, T, H, D), device="cuda")
    call = lib.CALL_ATTN_DECODE if T == 1 else lib.CALL_ATTN_PREFILL
    ws = lib.workspace(gc.workspace_bytes(call, T, H, 1))
    scale = lib.default_scale(D)
    if T == 1:
        lib.ds4a_compress_append(gc, p0, T, d)
        lib.ds4a_sparse_attn_decode(gc, p0, d["q"], H, None, 1, scale, out, ws)
        want = olayer.decode_step(oracle_cache(shape, hist, p0), p0, to_np(inp), 1)[0][:, None]
    else:
        chunk = torch.empty((2, T, D), device="cuda")
        lib.ds4a_compress_append(gc, p0, T, d, raw_chunk_out=chunk)
        lib.ds4a_sparse_attn_prefill_chunk(gc, p0, T, d["q"], H, chunk, None, 1, scale, out, ws)
        want = olayer.prefill_chunk(oracle_cache(shape, hist, p0), p0, to_np(inp), 1)[0]
    torch.cuda.synchronize()
    assert rel_l2(np_(out), want) <= TOL["f32"]
