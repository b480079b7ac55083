"""ds4a_paged_attn_decode against oracle/kv.py. Every row of the pools that no token may see holds NaN."""
import numpy as np
import pytest
import torch

from helpers import np_
from kv_step import Step, check
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV = "cuda"

CASES = [  # old lengths, new tokens, H, K, D, window, dtype, kv_dtype
    ([0], [1], 1, 1, 128, 0, "bf16", "bf16"),
    ([127, 128, 0, 255, 256, 511], [1] * 6, 16, 2, 128, 0, "bf16", "bf16"),
    ([1500, 3, 700], [1, 1, 1], 64, 8, 128, 0, "bf16", "bf16"),
    ([1500, 3, 700], [1, 1, 1], 64, 8, 128, 0, "bf16", "e4m3"),
    ([600, 126, 254, 0], [5, 3, 4, 2], 8, 1, 128, 0, "bf16", "bf16"),
    ([600, 126, 254, 0], [5, 3, 4, 2], 8, 1, 128, 0, "bf16", "e4m3"),
    ([300, 10, 900], [2, 0, 1], 5, 5, 64, 0, "bf16", "bf16"),
    ([300, 10, 900], [2, 0, 1], 10, 5, 64, 0, "bf16", "e4m3"),
    ([777, 64], [1, 8], 32, 2, 256, 0, "bf16", "bf16"),
    ([777, 64], [1, 8], 32, 2, 256, 0, "bf16", "e4m3"),
    ([400, 33], [1, 3], 6, 2, 96, 0, "bf16", "bf16"),
    ([400, 33], [1, 3], 6, 2, 96, 0, "bf16", "e4m3"),
    ([400, 33], [2, 1], 14, 2, 80, 0, "bf16", "bf16"),
    ([500, 33], [2, 1], 4, 2, 192, 0, "bf16", "bf16"),
    ([1000, 40, 128], [3, 2, 1], 16, 2, 128, 100, "bf16", "bf16"),
    ([1000, 40, 128], [3, 2, 1], 16, 2, 128, 129, "bf16", "e4m3"),
    ([1000, 40], [4, 2], 8, 2, 64, 1, "bf16", "bf16"),
    ([512, 5], [40, 20], 16, 2, 128, 0, "bf16", "bf16"),      # more rows than one group takes
    ([512, 5], [40, 20], 16, 2, 128, 30, "bf16", "e4m3"),
    ([300, 2], [1, 2], 4, 4, 10, 0, "bf16", "bf16"),          # CUDA cores
    ([300, 2], [1, 2], 4, 2, 20, 0, "bf16", "e4m3"),
    ([900, 0, 255], [2, 1, 3], 10, 2, 80, 0, "f32", "f32"),
    ([900, 0, 255], [2, 1, 3], 10, 2, 80, 64, "f32", "e4m3"),
    ([1300], [20], 6, 1, 256, 0, "f32", "f32"),
    ([100, 7], [1, 1], 128, 128, 2, 0, "f32", "f32"),
]


def run(step, c, cu, max_new=None, scale=None, ws=None, q=None, **kw):
    lib, H = step.lib, step.H
    max_new = max_new or max(int(step.new.max()), 1)
    q = step.q.to(DEV) if q is None else q
    out = torch.full((step.n, H, step.D), 77.0, dtype=q.dtype, device=DEV)
    lse = torch.full((step.n, H), 77.0, device=DEV)
    if ws is None:
        ws = lib.workspace(c.attn_workspace_bytes(H, max_new), DEV)
        ws[256:] = 255          # (what lies in a workspace is nobody's)
    lib.ds4a_paged_attn_decode(c, q, out, ws, max_new=max_new, cu_len=cu, lse=lse, window=step.window, scale=scale, **kw)
    assert lib.ds4a_workspace_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("old,new,H,K,D,window,dtype,kvd", CASES)
def test_attention(old, new, H, K, D, window, dtype, kvd):
    step = Step(lib_(), sum(old) + H + D, old, new, H, K, D, dtype, kvd, window)
    c, cu = step.on_gpu()
    out, lse = run(step, c, cu)
    check(step, out, lse, 1 / np.sqrt(D))
    again = run(step, c, cu)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("kvd", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [16, 64, 80, 112, 128, 176, 192, 240, 256])
@pytest.mark.parametrize("T,G", [(1, 3), (2, 7), (4, 8), (5, 8), (7, 16)])
def test_every_row_count_and_width(T, G, D, kvd):
    """Each number of rows a block takes, on each width of keys and values."""
    step = Step(lib_(), T * G + D, [200, 31, 3], [T, max(1, T - 2), T], 2 * G, 2, D, "bf16", kvd)
    c, cu = step.on_gpu()
    check(step, *run(step, c, cu), 1 / np.sqrt(D))


@pytest.mark.parametrize("dtype,kvd", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales_and_a_window_wider_than_the_context(dtype, kvd, scale):
    step = Step(lib_(), 21, [290, 7], [2, 1], 8, 2, 64, dtype, kvd, window=5000)
    c, cu = step.on_gpu()
    check(step, *run(step, c, cu, scale=scale), scale)


@pytest.mark.parametrize("dtype,kvd", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
def test_many_sequences_some_of_them_free(dtype, kvd):
    """More sequences than blocks, most of them short; free rows in between and at the ends."""
    rng = np.random.default_rng(5)
    B = 700
    old, new = rng.integers(0, 40, B), rng.integers(0, 3, B)
    old[350], new[350], new[:3], new[-40:] = 1500, 2, 0, 0
    old[new == 0] = 0
    step = Step(lib_(), 22, list(old), list(new), 4, 2, 32, dtype, kvd)
    c, cu = step.on_gpu()
    check(step, *run(step, c, cu), 1 / np.sqrt(32))


@pytest.mark.parametrize("kvd", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [1, 40])
def test_long_and_many(B, kvd):
    """One sequence shared among all SMs, and a ragged batch that several share."""
    rng = np.random.default_rng(B)
    old = [20000] if B == 1 else list(rng.integers(0, 3000, B))
    step = Step(lib_(), B, old, [1] * B, 8, 2 if B == 1 else 4, 128, "bf16", kvd)
    c, cu = step.on_gpu()
    check(step, *run(step, c, cu), 1 / np.sqrt(128))


@pytest.mark.parametrize("std", [0.02, 12.0])
@pytest.mark.parametrize("kvd", ["bf16", "e4m3"])
def test_flat_and_peaked_scores(kvd, std):
    """Scores that are all alike, and ones that spread over hundreds (the maximum keeps growing)."""
    step = Step(lib_(), 3, [1900, 600], [2, 1], 16, 2, 128, "bf16", kvd, std=std)
    c, cu = step.on_gpu()
    check(step, *run(step, c, cu), 1 / np.sqrt(128))


@pytest.mark.parametrize("dtype,kvd", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
def test_rising_scores(dtype, kvd):
    """Each tile's keys beat the ones before by far, then fall: every rescaling on the way."""
    step = Step(lib_(), 8, [1535], [1], 8, 1, 128, dtype, kvd, std=0.05)
    level = torch.arange(1536).div(64, rounding_mode="floor").float()
    level = torch.where(level < 16, level * 3, 60 - level)
    for i, blk in enumerate(step.table[0]):
        x = level[256 * i:256 * (i + 1)]
        if kvd == "e4m3":
            x = x / step.k_scale[0]
        step.pk[blk, 0, :, 0] = x.clamp(-448, 448).to(step.pk.dtype)
    step.q[:, :, 0] = 3.0
    c, cu = step.on_gpu()
    check(step, *run(step, c, cu, scale=1.0), 1.0)


@pytest.mark.parametrize("dtype,kvd", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
def test_blocks_that_are_not_there(dtype, kvd):
    """Their keys take no part; a token all of whose keys are missing gets zeros."""
    step = Step(lib_(), 4, [600, 300, 100, 700], [2, 1, 3, 1], 8, 2, 64, dtype, kvd,
                hole=[(0, 1), (2, 0), (3, 0), (3, 1), (3, 2)])
    c, cu = step.on_gpu()
    out, lse = run(step, c, cu)
    check(step, out, lse, 1 / 8.0)
    assert (out[3:6] == 0).all() and (out[6] == 0).all() and torch.isneginf(lse[3:]).all()
    c.block_table[0, 1], c.block_table[2, 0] = step.nb, 1 << 30     # outside the pool: the same
    again = run(step, c, cu)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype,kvd", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
@pytest.mark.parametrize("window", [0, 40])
def test_what_one_token_sees_and_another_does_not(dtype, kvd, window):
    """NaN and infinities in rows that only some of a sequence's tokens see reach those alone."""
    step = Step(lib_(), 5, [300], [4], 8, 2, 64, dtype, kvd, window)
    inf = float("nan") if kvd == "e4m3" else float("inf")
    at = lambda p: (step.table[0, p // 256], p % 256)  # noqa: E731
    blk, r = at(303)                       # the last token's own row
    step.pv[blk, 1, r, 7], step.pv[blk, 1, r, 9] = float("nan"), inf
    step.pk[blk, 0, r, 3] = float("nan")
    if window:                             # the first token's oldest row
        blk, r = at(261)
        step.pv[blk, 0, r, 20] = inf
    c, cu = step.on_gpu()
    out, lse = run(step, c, cu)
    ok = torch.ones((4, 8, 64), dtype=torch.bool)
    ok[3, :4], ok[3, 4:, 7], ok[3, 4:, 9] = False, False, False
    if window:
        ok[0, :4, 20] = False
    bad = ~torch.isfinite(out.cpu().float())
    assert (bad == ~ok).all()
    assert torch.isfinite(lse[:3]).all() and torch.isfinite(lse[3, 4:]).all() and torch.isnan(lse[3, :4]).all()
    # the others' values: those of a step without the rows
    clean = Step(lib_(), 5, [300], [4], 8, 2, 64, dtype, kvd, window)
    want, _, mag, flat = clean.oracle(1 / 8.0)
    tol, _ = clean.tolerance(want, mag, flat, 1 / 8.0)
    err = np.abs(np_(out).astype(np.float64) - want)
    assert (err[ok.numpy()] <= tol[ok.numpy()]).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 32)])
def test_more_tokens_than_max_new_and_rows_behind_the_last(dtype, D):
    step = Step(lib_(), 6, [200, 90], [5, 2], 4, 2, D, dtype)
    c, cu = step.on_gpu()
    out, lse = run(step, c, cu, max_new=3)
    check(step, out, lse, 1 / np.sqrt(D), max_new=3)
    assert (out[3:5] == 77).all() and (lse[3:5] == 77).all()
    # packed tokens: what follows the last one stays
    big = torch.full((step.n + 3, 4, D), 77.0, dtype=out.dtype, device=DEV)
    q = torch.zeros_like(big)
    q[:step.n] = step.q.to(DEV)
    ws = step.lib.workspace(c.attn_workspace_bytes(4, 5), DEV)
    step.lib.ds4a_paged_attn_decode(c, q, big, ws, max_new=5, cu_len=cu)
    assert (big[step.n:] == 77).all()


@pytest.mark.parametrize("D,shift", [(128, 0), (128, 1), (96, 5)])
def test_strided_and_unaligned_queries_and_no_lengths(D, shift):
    """Queries inside a projection's output, off 16 bytes; cu_len None: as many tokens each; no lse."""
    for kvd in ("bf16", "e4m3"):
        step = Step(lib_(), 7, [333, 41], [2, 2], 8, 2, D, "bf16", kvd)
        c, cu = step.on_gpu()
        want = run(step, c, cu)
        wide = torch.zeros(4 * (8 * D + 24) + shift, dtype=torch.bfloat16, device=DEV)[shift:].view(4, -1)
        q = wide[:, :8 * D].view(4, 8, D)
        q.copy_(step.q)
        got = run(step, c, None, max_new=2, q=q)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        out = torch.empty_like(got[0])
        step.lib.ds4a_paged_attn_decode(c, q, out, step.lib.workspace(c.attn_workspace_bytes(8, 2), DEV), max_new=2)
        assert torch.equal(out, want[0])


def test_two_streams_and_a_graph():
    """Calls on two streams with a workspace each; a captured call replayed with other lengths."""
    lib = lib_()
    a = Step(lib, 9, [900, 20], [1, 1], 16, 2, 128, "bf16")
    b = Step(lib, 10, [50, 1200, 3], [2, 1, 2], 8, 2, 64, "bf16", "e4m3")
    (ca, cua), (cb, cub) = a.on_gpu(), b.on_gpu()
    wa, wb = run(a, ca, cua), run(b, cb, cub)
    qa, qb = a.q.to(DEV), b.q.to(DEV)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    for i in range(10):
        with torch.cuda.stream(s1):
            x = run(a, ca, cua, q=qa)[0]
        with torch.cuda.stream(s2):
            y = run(b, cb, cub, q=qb)[0]
        outs.append((x, y))
    torch.cuda.synchronize()
    assert all(torch.equal(x, wa[0]) and torch.equal(y, wb[0]) for x, y in outs)

    ws, out = lib.workspace(ca.attn_workspace_bytes(16, 1), DEV), torch.empty_like(wa[0])
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        lib.ds4a_paged_attn_decode(ca, qa, out, ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            lib.ds4a_paged_attn_decode(ca, qa, out, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, wa[0])
    ca.seq_pos.copy_(torch.tensor([400, 0], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    a.old = np.array([400, 0])
    a.pk, a.pv = a.pk.float(), a.pv.float()
    want, _, mag, flat = a.oracle(1 / np.sqrt(128))
    tol, _ = a.tolerance(want, mag, flat, 1 / np.sqrt(128))
    assert (np.abs(np_(out) - want) <= tol).all()


def test_offsets_beyond_32_bits():
    """Blocks whose rows start beyond 2^32 bytes and 2^31 elements of the pools."""
    lib = lib_()
    K, D = 2, 256
    nb = (1 << 31) // (K * 256 * D) + 40
    step = Step(lib, 11, [700], [1], 8, K, D, "bf16")
    c, cu = step.on_gpu()
    want = run(step, c, cu)
    pk = torch.empty((nb, K, 256, D), dtype=torch.bfloat16, device=DEV)
    pv = torch.empty_like(pk)
    far = torch.arange(nb - step.nb, nb, device=DEV)
    pk[far], pv[far] = c.k, c.v
    big = lib.KvCache(head_dim=D, n_kv_heads=K, batch=1, block_table=c.block_table + (nb - step.nb), n_blocks=nb,
                      k=pk, v=pv, device=DEV)
    big.set_seq_pos(c.seq_pos)
    got = run(step, big, cu)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    k, v = (torch.randn((1, K, D), device=DEV).bfloat16() for _ in range(2))
    lib.ds4a_kv_append(big, i32([0]), i32([5]), k, v)
    blk = int(big.block_table[0, 0])
    assert torch.equal(pk[blk, :, 5], k[0]) and torch.equal(pv[blk, :, 5], v[0])




@pytest.mark.parametrize("kvd", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("T,G", [(1, 3), (2, 7), (4, 8), (5, 8), (40, 5)])
def test_every_row_count_and_width_divided(T, G, D, kvd):
    """The same with sequences whose tiles several blocks share; groups that start inside a token."""
    step = Step(lib_(), T * G + D + 1, [1500, 700, 3], [T, max(1, T - 2), T], G, 1, D, "bf16", kvd)
    c, cu = step.on_gpu()
    check(step, *run(step, c, cu), 1 / np.sqrt(D))


@pytest.mark.parametrize("dtype,kvd", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
@pytest.mark.parametrize("window", [1, 128, 378, 381, 384, 500])
def test_windows_around_the_longest_undivided_sequence(window, dtype, kvd):
    step = Step(lib_(), window, [1023, 895, 130, 640], [3, 2, 3, 1], 8, 2, 64, dtype, kvd, window=window)
    c, cu = step.on_gpu()
    check(step, *run(step, c, cu), 1 / 8)


@pytest.mark.parametrize("kvd", ["bf16", "e4m3"])
def test_more_undivided_sequences_than_blocks(kvd):
    rng = np.random.default_rng(9)
    B = 500
    old, new = rng.integers(0, 500, B), rng.integers(0, 4, B)
    old[new == 0] = 0
    step = Step(lib_(), 23, list(old), list(new), 6, 2, 16, "bf16", kvd)
    c, cu = step.on_gpu()
    check(step, *run(step, c, cu), 0.25)


@pytest.mark.parametrize("old", [[200, 30], [900, 30]])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("D", [64, 144, 256])
def test_unaligned_queries_over_8_bits(D, shift, old):
    """Rows that do not start on 16 bytes give what aligned ones give, bit for bit."""
    step = Step(lib_(), D + shift, old, [3, 2], 10, 2, D, "bf16", "e4m3")
    c, cu = step.on_gpu()
    want = run(step, c, cu)
    check(step, *want, 1 / np.sqrt(D))
    wide = torch.zeros(step.n * (10 * D + 3) + 8, dtype=torch.bfloat16, device=DEV)
    q = wide.as_strided((step.n, 10, D), (10 * D + 3, D, 1), shift)
    q.copy_(step.q)
    got = run(step, c, cu, q=q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
