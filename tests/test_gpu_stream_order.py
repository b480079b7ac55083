"""The attention reads its queries, positions and workspace in stream order: whatever writes
them may be the launch directly before. Every call is compared bit for bit with the same call
behind a synchronisation."""
import pytest
import torch

from test_gpu_fp4_attention import BASE, DEV
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
H, D, POS, B = 64, 512, 3000, 6
SCALE = 0.2          # sharp weights: another query gives another output


def layer(ratio, fp4, T=1, more=0):
    lib = lib_()
    cap = 768 if ratio == 4 else 24 if ratio else 0
    c = lib.LayerCache(ratio=ratio, head_dim=D, n_rot=64, batch=B, comp_cap=cap, dtype="bf16", base=BASE,
                       rope_max_pos=POS + T, index_dim=32, index_rot=32, device=DEV,
                       qat=(lib.FP4_ROWS if fp4 else 0) | more)
    g = torch.Generator().manual_seed(ratio + fp4)
    rn = lambda *s: torch.randn(s, generator=g).bfloat16().to(DEV)  # noqa: E731
    c.raw_kv.copy_(rn(B, 128, D))
    if fp4:
        lib.ds4a_pack_rows(c, rn(B * cap, D))
    elif ratio:
        c.attn_comp_kv.copy_(rn(B, cap, D))
    c.n_tokens = POS + T
    c.tk = None
    if ratio == 4:
        c.tk = torch.stack([torch.randperm(700, generator=g)[:256].sort()[0] for _ in range(B * T)])
        c.tk = c.tk.int().view(B, T, 256).to(DEV)
    call = lib.CALL_ATTN_DECODE if T == 1 else lib.CALL_ATTN_PREFILL
    c.ws = lib.workspace(c.workspace_bytes(call, T, H, 256))
    c.chunk = rn(B, T, D)
    return c, rn


def attend(c, T, q, out):
    lib = lib_()
    if T == 1:
        lib.ds4a_sparse_attn_decode(c, POS, q, H, c.tk, 256, SCALE, out, c.ws)
    else:
        lib.ds4a_sparse_attn_prefill_chunk(c, POS, T, q, H, c.chunk, c.tk, 256, SCALE, out, c.ws)


def both(run, n, like):
    """run(i, out, sync) for every i, with a wait after every launch and without."""
    want, got = [torch.empty_like(like) for _ in range(n)], [torch.empty_like(like) for _ in range(n)]
    for i in range(n):
        run(i, want[i], torch.cuda.synchronize)
        torch.cuda.synchronize()
    for _ in range(2):
        for i in range(n):
            run(i, got[i], lambda: None)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert not torch.equal(want[0], want[1])


@pytest.mark.parametrize("ratio,fp4", [(0, False), (4, False), (128, False), (4, True), (128, True)])
def test_one_attention_writes_the_queries_of_the_next(ratio, fp4):
    c, rn = layer(ratio, fp4)
    x = [rn(B, H, D) for _ in range(20)]
    mid = torch.empty_like(x[0])

    def run(i, out, sync):
        attend(c, 1, x[i], mid)
        sync()
        attend(c, 1, mid, out)

    both(run, len(x), mid)


def test_one_chunk_writes_the_queries_of_the_next():
    T = 8
    c, rn = layer(4, True, T)
    ring = c.raw_kv.clone()
    x = [rn(B, T, H, D) for _ in range(12)]
    mid = torch.empty_like(x[0])

    def run(i, out, sync):
        c.raw_kv.copy_(ring)
        sync()
        attend(c, T, x[i], mid)
        sync()
        c.raw_kv.copy_(ring)
        sync()
        attend(c, T, mid, out)

    both(run, len(x), mid)


@pytest.mark.parametrize("fp4", [False, True])
def test_positions_written_by_the_launch_before(fp4):
    c, rn = layer(4, fp4)
    q = rn(B, H, D)
    seq = torch.zeros(B, dtype=torch.int32, device=DEV)
    c.set_seq_pos(seq)
    pos = [torch.randint(0, POS + 1, (B,), dtype=torch.int32).to(DEV) for _ in range(20)]

    def run(i, out, sync):
        torch.add(pos[i], 0, out=seq)
        sync()
        attend(c, 1, q, out)

    both(run, len(pos), q)


def test_a_status_word_written_by_the_launch_before():
    """The workspace's first word changes between calls: no call takes it for a wait that gave up."""
    lib = lib_()
    c, rn = layer(4, False)
    x = [rn(B, H, D) for _ in range(20)]
    word = c.ws[:4].view(torch.int32)

    def run(i, out, sync):
        word.fill_(i % 3)
        sync()
        attend(c, 1, x[i], out)

    both(run, len(x), x[0])
    lib.ds4a_workspace_clear_status(c.ws)
    torch.cuda.synchronize()
    assert lib.ds4a_workspace_status(c.ws) == 0


@pytest.mark.parametrize("ratio,fp4", [(0, False), (4, False), (128, False), (4, True), (128, True)])
@pytest.mark.parametrize("T", [1, 8])
def test_queries_that_are_ready(ratio, fp4, T):
    """DS4A_Q_READY changes no result: another call of the library stands between what
    writes the queries and the attention."""
    lib = lib_()
    outs = []
    for more in (0, lib.Q_READY):
        c, rn = layer(ratio, fp4, T, more)
        x = [rn(B, T, H, D) for _ in range(6)]
        got, q, kv = [], torch.empty_like(x[0]), rn(B * T, D)
        row, p = torch.empty_like(kv), torch.full((B * T,), 7, dtype=torch.int32, device=DEV)
        ring = c.raw_kv.clone()
        for xi in x:
            c.raw_kv.copy_(ring)
            q.copy_(xi)
            lib.ds4a_norm_rope(c, p, kv=kv, kv_out=row)
            out = torch.empty_like(q)
            attend(c, T, q, out)
            got.append(out)
        torch.cuda.synchronize()
        outs.append(got)
    for a, b in zip(*outs):
        assert torch.equal(a, b)
