"""First calls of a process from several host threads at once, sizes that differ from thread to
thread: every one of them launches and gives what the same call gives alone."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import sys; sys.path.insert(0, 'tests'); sys.path.insert(0, '.')
import threading
import torch
from compressed_kv_sparse_gb300 import lib
lib.load()
ROWS = (1900, 8192, 2500, 5000, 3000, 7000)
HEADS = (64, 5, 64, 8, 64, 3)
jobs, bad = [], []
for t, (rows, H) in enumerate(zip(ROWS, HEADS)):
    g = torch.Generator().manual_seed(t)
    D, dt = (512, torch.bfloat16) if t % 2 == 0 else (256, torch.float32)
    c = lib.LayerCache(ratio=128, head_dim=D, n_rot=64, batch=2, comp_cap=8, base=160000.0,
                       dtype='bf16' if t % 2 == 0 else 'f32', rope_max_pos=1024,
                       qat=lib.FP4_ROWS if t in (2, 3) else 0)
    c.raw_kv.copy_(torch.randn(c.raw_kv.shape, generator=g))
    if not c.fp4_rows:
        c.attn_comp_kv.copy_(torch.randn(c.attn_comp_kv.shape, generator=g))
    c.n_tokens = 1000
    q = torch.randn((2, H, D), generator=g).to('cuda', dt)
    ws = lib.workspace(c.workspace_bytes(lib.CALL_ATTN_DECODE, 1, H, 1))
    ctx = torch.randint(0, 1500, (rows,), generator=g, dtype=torch.int32).cuda()
    jobs.append((rows, H, c, q, ws, ctx, torch.cuda.Stream()))
torch.cuda.synchronize()
gate = threading.Barrier(len(jobs))


def one(job, out, wait):
    rows, H, c, q, ws, ctx, s = job
    pool, step = lib.BlockPool(rows, 8, rows * 6), lib.StepTables(rows, rows)
    o = torch.empty_like(q)
    torch.cuda.synchronize()
    wait()
    with torch.cuda.stream(s):
        lib.ds4a_block_tables(pool, ctx, torch.ones_like(ctx), 128, step)
        lib.ds4a_sparse_attn_decode(c, 999, q, H, None, 1, lib.default_scale(q.shape[2]), o, ws)
    s.synchronize()
    out.append((pool.table, step.raw_slot, o))


def thread(job, out):
    try:
        one(job, out, gate.wait)
    except BaseException as e:
        bad.append(repr(e))
        gate.abort()


got = [[] for _ in jobs]
th = [threading.Thread(target=thread, args=a) for a in zip(jobs, got)]
for x in th:
    x.start()
for x in th:
    x.join()
assert not bad, bad
for job, out in zip(jobs, got):
    one(job, out, lambda: None)
    for a, b in zip(*out):
        assert torch.equal(a, b)
print('threads done')
"""


def test_first_calls_from_many_threads():
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=180)
    assert r.returncode == 0 and "threads done" in r.stdout, r.stderr[-2000:]
