"""What the Python calls refuse before the library is called: tensors of another device, type or
size, on a binding whose checks stay under `python -O`. No GPU: a cache's tensors stand on the
CPU, and a device that is not there is played by its number."""
import subprocess
import sys

import pytest
import torch

from compressed_kv_sparse_gb300 import lib
from test_abi_cpu import L  # noqa: F401  (the library fixture)

BF, I32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)


def cache(ratio=128, **kw):
    a = dict(ratio=ratio, comp_cap=6, head_dim=512, n_rot=64, batch=2, dtype="bf16", base=160000.0,
             rope_max_pos=16, device="cpu", qat=lib.FP4_ROWS)
    return lib.LayerCache(**{**a, **kw})


def calls(c, dev="cpu"):
    """Every call that launches, with tensors that suit it but for their device."""
    t = lambda *s, **k: torch.zeros(s, device=dev, **(k or BF))  # noqa: E731
    x = {"raw_kv_in": t(2, 1, 512), "attn_cand": t(2, 1, 512), "attn_score": t(2, 1, 512),
         "ape_attn": t(128, 512), "gamma_attn": t(512)}
    pos, q, kv, ws = t(3, **I32), t(3, 4, 512), t(3, 512), t(1 << 16, dtype=torch.uint8)
    step, pool = lib.StepTables(2, 4, device=dev), lib.BlockPool(2, 4, 8, device=dev)
    return {
        "reset": lambda **k: lib.ds4a_cache_reset(c, **k),
        "norms": lambda **k: lib.ds4a_index_norms(c, **k),
        "append": lambda **k: lib.ds4a_compress_append(c, 0, 1, x, **k),
        "lanes": lambda **k: lib.ds4a_compress_append_lanes(c, 0, 1, lib.LANE_ATTN, x, **k),
        "topk": lambda **k: lib.ds4a_index_topk(c, 0, 1, q, kv, 4, 8, pos, ws, **k),
        "noalloc": lambda **k: lib.ds4a_index_topk_noalloc(c, 0, 1, q, kv, 4, 8, pos, **k),
        "decode": lambda **k: lib.ds4a_sparse_attn_decode(c, 0, q, 4, None, 1, 0.1, q, ws, **k),
        "chunk": lambda **k: lib.ds4a_sparse_attn_prefill_chunk(c, 0, 1, q, 4, kv, None, 1, 0.1, q, ws, **k),
        "pack": lambda **k: lib.ds4a_pack_rows(c, kv, **k),
        "unpack": lambda **k: lib.ds4a_unpack_rows(c, kv, pos, **k),
        "rope": lambda **k: lib.ds4a_norm_rope(c, pos, q=q, q_out=q, kv=kv, kv_out=kv, **k),
        "tables": lambda **k: lib.ds4a_block_tables(pool, t(2, **I32), t(2, **I32), 128, step, **k),
        "clear": lambda **k: lib.ds4a_workspace_clear_status(ws, **k),
        "selftest": lambda **k: lib.ds4a_wait_selftest(ws, 1000, **k),
    }


NAMES = list(calls(cache()))


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_the_cpu(L, name):
    for stream in (None, 0):
        with pytest.raises(lib.ArgumentError, match="not on a GPU"):
            calls(cache())[name](stream=stream)


@pytest.mark.parametrize("name", [n for n in NAMES if n not in ("reset", "norms", "tables", "clear", "selftest")])
def test_tensors_of_another_device_than_the_cache(L, name):
    """The cache on (what says it is) a GPU, the tensors on the CPU."""
    c = cache()
    c.dev = 0
    with pytest.raises(lib.ArgumentError, match="device|on cpu"):
        calls(c)[name](stream=0)


def test_a_device_that_is_not_the_current_one(L, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(lib.ArgumentError, match="cuda:1, which is not the current"):
        lib._stream(None, 1)

    class Stream:
        cuda_stream, device_index = 0x77, 1

    with pytest.raises(lib.ArgumentError, match="a stream of cuda:1"):
        lib._stream(Stream(), 0)
    Stream.device_index = 0
    assert lib._stream(Stream(), 0) == 0x77 and lib._stream(5, 0) == 5


def test_caches_and_positions(L):
    c = cache(batch=3)
    for bad in (torch.zeros(3, dtype=torch.int64), torch.zeros(2, **I32), torch.zeros(6, **I32)[::2]):
        with pytest.raises(lib.ArgumentError):
            c.set_seq_pos(bad)
        assert not c.c.seq_pos
    c.set_seq_pos(torch.zeros(3, **I32))
    assert c.c.seq_pos
    c.set_seq_pos(None)
    assert not c.c.seq_pos
    for table in (torch.zeros((2, 3)), torch.zeros((3, 3), **I32)):
        with pytest.raises(lib.ArgumentError):
            cache(block_table=table, n_blocks=4)
    with pytest.raises(lib.ArgumentError):
        cache(block_table=torch.zeros((2, 4), **I32), n_blocks=4)
    pool, other = lib.BlockPool(2, 4, 8, device="cpu"), lib.StepTables(3, 4, device="cpu")
    with pytest.raises(lib.ArgumentError):
        lib.ds4a_block_tables(pool, torch.zeros(2, **I32), torch.zeros(2, **I32), 128, other, stream=0)


def test_checks_stay_without_assertions(L):
    code = """
import sys; sys.path[:0] = ['.', 'tests']
import torch
from compressed_kv_sparse_gb300 import lib
from test_binding_checks_cpu import cache
assert False          # (not run: python -O)
c, n = cache(), 0
rows = torch.zeros((3, 512))
for bad in ((rows, None), (rows.bfloat16()[:, :256], None), (rows.bfloat16(), torch.zeros(3, dtype=torch.int64)),
            (rows.bfloat16(), None)):
    try:
        lib.ds4a_pack_rows(c, *bad)
    except lib.ArgumentError:
        n += 1
try:
    lib.ds4a_norm_rope(c, torch.zeros(3, dtype=torch.int64), kv=rows, kv_out=rows)
except lib.ArgumentError:
    n += 1
print('refused', n)
"""
    r = subprocess.run([sys.executable, "-O", "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "refused 5" in r.stdout, (r.stdout, r.stderr[-2000:])


@pytest.mark.parametrize("paged", [False, True])
def test_rows_of_a_cache(L, paged):
    """Sequences of a cache as a cache of their own: the same memory, its own count."""
    kw = dict(block_table=torch.arange(8, **I32).view(4, 2), n_blocks=9) if paged else {}
    c = cache(ratio=4, batch=4, comp_cap=128, index_dim=128, index_rot=64, **kw)
    c.set_seq_pos(torch.arange(4, **I32))
    c.n_tokens = 12
    v = c.rows(1, 3)
    assert v.batch == v.c.batch == 2 and c.c.batch == 4 and v.n_tokens == 12
    v.n_tokens = 13
    assert c.n_tokens == 12 and v.ref()._obj.n_tokens == 13 and c.ref()._obj.n_tokens == 12
    per = ["raw_kv", "attn_state_kv", "attn_state_score", "index_state_kv", "index_state_score",
           "index_norm_max", "seq_pos"]
    pool = ["attn_comp_kv", "index_comp_kv", "index_norm"]
    for n in per + (["block_table"] if paged else pool):
        assert getattr(v.c, n) == getattr(c, n)[1:].data_ptr() and getattr(v, n).shape[0] == 2, n
    for n in (pool if paged else []) + ["rope_cos", "rope_sin", "index_rope_cos"]:
        assert getattr(v.c, n) == getattr(c, n).data_ptr(), n
    assert v.slots(2).tolist() == (c.slots(2)[1:3].tolist() if paged else [[0, 1], [128, 129]])
    for bad in ((0, 0), (2, 1), (0, 5), (-1, 2)):
        with pytest.raises(lib.ArgumentError):
            c.rows(*bad)
