"""Attention over compressed rows held in 4 bits, decode and chunk, against a plain fp64
softmax over the values that the rows stand for.

Tolerance per output element, from the arithmetic (u: half a step of the type, 2^-8 for
bf16): the probabilities and, in a cluster, the partial outputs are rounded to the type, which
with the sums taken over the rounded probabilities moves an output by at most 3 u A, A = sum_i
p_i |v_i|; a rotated query is rounded to the type again, which moves a score by at most d =
scale * sum over the tail of u |q'| |k|, and fp32 sums of D products add D 2^-24 scale sum
|q'| |k|; both move the output by 2 d A; the tail is turned back, which adds the bounds of a pair;
and the result is rounded: u |o|. For fp32 the same with u = 2^-24 and 2^-19 for the
exponentials and long sums."""
import numpy as np
import pytest
import torch

from helpers import np_
from oracle.attention import comp_row_ids
from oracle.rope import rope_tail
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV = "cuda"
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
BASE = 160000.0


class Case:
    """A cache with 4-bit rows, its queries and lists, and the fp64 answer."""

    def __init__(self, ratio, B, T, pos, H, D=512, top_k=512, dtype="bf16", ragged=None, paged=False,
                 rot_q=False, seed=0, q_std=2.0, cap_raw=128, n_rot=64, lists=None):
        lib = lib_()
        self.__dict__.update(ratio=ratio, B=B, T=T, pos=pos, H=H, D=D, k=top_k, dtype=dtype,
                             rot_q=rot_q, cap_raw=cap_raw, n_rot=n_rot)
        g = torch.Generator().manual_seed(seed + 7 * pos + H)
        rn = lambda *s: torch.randn(s, generator=g).to(DEV, TD[dtype])  # noqa: E731
        self.p0 = np.full(B, pos) if ragged is None else np.array(ragged)
        assert self.p0.max() <= pos and len(self.p0) == B
        rpb, mb = 256 // ratio, -(-(pos + T) // 256)
        cap = mb * rpb
        kw = {}
        if paged:
            n_blocks = B * mb + 3
            table = torch.randperm(n_blocks, generator=g)[:B * mb].int().view(B, mb).to(DEV)
            kw = dict(block_table=table, n_blocks=n_blocks)
        qat = lib.FP4_ROWS | (lib.Q_ROTATED if rot_q else 0)
        self.c = lib.LayerCache(ratio=ratio, head_dim=D, n_rot=n_rot, batch=B, comp_cap=cap,
                                dtype=dtype, base=BASE, rope_max_pos=pos + T, index_dim=32,
                                index_rot=32, cap_raw=cap_raw, qat=qat, device=DEV, **kw)
        rows = rn(B * cap, D)
        lib.ds4a_pack_rows(self.c, rows, self.c.slots(cap).reshape(-1))
        self.rows = torch.empty_like(rows)
        lib.ds4a_unpack_rows(self.c, self.rows, self.c.slots(cap).reshape(-1))
        self.rows = np_(self.rows).reshape(B, cap, D).astype(np.float64)
        self.c.n_tokens = pos + T
        if ragged is not None:
            self.c.set_seq_pos(torch.tensor(self.p0, dtype=torch.int32, device=DEV))
        self.q = (q_std * torch.randn((B, T, H, D), generator=g)).to(DEV, TD[dtype])
        self.chunk = rn(B, T, D)
        self.ring = rn(B, cap_raw, D)
        if T == 1:
            for b in range(B):
                self.ring[b, int(self.p0[b]) % cap_raw] = self.chunk[b, 0]
        # slots of positions that never were must not matter
        for b in range(B):
            n = int(self.p0[b]) + (1 if T == 1 else 0)
            if n < cap_raw:
                self.ring[b, n:] = float("nan")
        self.c.raw_kv.copy_(self.ring)
        self.topk = None
        if ratio == 4:
            tk = np.full((B, T, top_k), -1, np.int32)
            rng = np.random.default_rng(seed)
            for b in range(B):
                for t in range(T):
                    vis = (int(self.p0[b]) + t + 1) // 4
                    m = min(vis, top_k)
                    tk[b, t, :m] = np.sort(rng.choice(vis, m, replace=False)) if vis else []
                    if lists is not None:
                        lists(rng, tk[b, t], vis)
            self.topk_np = tk
            self.topk = torch.tensor(tk, device=DEV)
        self.scale = lib.default_scale(D)
        self.out = torch.full((B, T, H, D), 55.0, dtype=TD[dtype], device=DEV)
        call = lib.CALL_ATTN_DECODE if T == 1 else lib.CALL_ATTN_PREFILL
        self.ws = lib.workspace(self.c.workspace_bytes(call, T, H, top_k))

    def run(self, stream=None):
        lib = lib_()
        if self.T == 1:
            lib.ds4a_sparse_attn_decode(self.c, self.pos, self.q, self.H, self.topk, self.k,
                                        self.scale, self.out, self.ws, stream=stream)
        else:
            lib.ds4a_sparse_attn_prefill_chunk(self.c, self.pos, self.T, self.q, self.H, self.chunk,
                                               self.topk, self.k, self.scale, self.out, self.ws,
                                               stream=stream)

    def want(self, b, t):
        """fp64 output [H][D] and its tolerance."""
        p0, u = int(self.p0[b]), torch.finfo(TD[self.dtype]).eps / 2
        p = p0 + t
        win = []
        for s in range(max(0, p - self.cap_raw + 1), p + 1):
            win.append(np_(self.chunk[b, s - p0] if s >= p0 else self.ring[b, s % self.cap_raw]))
        n_comp = (self.pos + self.T) // self.ratio
        ids = comp_row_ids(self.ratio, p, n_comp, None if self.topk is None else self.topk_np[b, t])
        K = np.concatenate([np.array(win, np.float64).reshape(-1, self.D), self.rows[b, ids]])
        q = np_(self.q[b, t]).astype(np.float64)
        if not self.rot_q:
            q = rope_tail(q, p, BASE, self.n_rot)
        s = q @ K.T * self.scale
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        o = rope_tail(w @ K, p, BASE, self.n_rot, inverse=True)
        A = w @ np.abs(K)
        nope, mag = self.D - self.n_rot, np.abs(q) @ np.abs(K).T * self.scale
        d = self.D * 2.0 ** -24 * mag
        if not self.rot_q and self.dtype == "bf16":
            d = d + u * (np.abs(q[:, nope:]) @ np.abs(K[:, nope:]).T) * self.scale
        base = (3 * u if self.dtype == "bf16" else 2.0 ** -19) + 2 * d.max(-1, keepdims=True)
        tol = base * A
        tail = tol[:, nope:]
        tol[:, nope:] = np.repeat(tail[:, 0::2] + tail[:, 1::2], 2, -1)
        return o, tol + u * np.abs(o) + 1e-30

    def check(self, queries=None):
        torch.cuda.synchronize()
        got = np_(self.out).astype(np.float64)
        todo = queries or [(b, t) for b in range(self.B) for t in range(self.T)]
        num = den = 0.0
        for b, t in todo:
            o, tol = self.want(b, t)
            err = np.abs(got[b, t] - o)
            assert (err <= tol).all(), (b, t, float((err / tol).max()))
            num, den = num + (err ** 2).sum(), den + (o ** 2).sum()
        assert np.sqrt(num / den) <= (6e-3 if self.dtype == "bf16" else 2e-6)
        if self.T > 1:      # the window now holds the chunk's last rows
            for b in range(self.B):
                for t in range(max(0, self.T - self.cap_raw), self.T):
                    slot = (int(self.p0[b]) + t) % self.cap_raw
                    assert torch.equal(self.c.raw_kv[b, slot], self.chunk[b, t])


def few(rng, row, vis):
    """Holes in the list, nothing left of every third one."""
    row[rng.random(len(row)) < 0.4] = -1
    if rng.random() < 0.35:
        row[:] = -1


def ends_early(rng, row, vis):
    """An entry that is not visible ends the list; what follows it does not count."""
    m = int((row >= 0).sum())
    if m > 2:
        row[m // 2] = vis + 3
    elif m < len(row):
        row[m] = vis


def late(rng, row, vis):
    """Nothing in the first 400 places, so that whole tiles have no row."""
    m = int((row >= 0).sum())
    keep = row[:m].copy()
    row[:] = -1
    row[400:] = np.sort(rng.choice(keep, len(row) - 400, replace=False))


DECODE = [  # ratio, B, pos, H, dtype, ragged, paged, rot_q, top_k
    (4, 1, 0, 64, "bf16", None, False, True, 512),
    (4, 2, 2, 64, "bf16", None, True, False, 512),
    (4, 3, 126, 64, "bf16", None, False, False, 512),
    (4, 3, 127, 64, "bf16", None, False, True, 512),
    (4, 5, 9000, 64, "bf16", [0, 3, 127, 600, 9000], True, False, 512),
    (4, 2, 5000, 5, "bf16", None, True, True, 77),
    (4, 2, 5000, 128, "bf16", [5000, 131], False, True, 129),
    (4, 1, 20000, 33, "bf16", None, False, False, 2048),
    (4, 7, 3000, 1, "bf16", None, True, True, 1),
    (128, 1, 0, 64, "bf16", None, True, True, 1),
    (128, 2, 127, 64, "bf16", None, False, True, 1),
    (128, 2, 16511, 64, "bf16", None, False, False, 1),
    (128, 3, 70000, 64, "bf16", [70000, 40, 20479], True, True, 1),
    (128, 2, 70001, 24, "bf16", [70001, 0], False, False, 1),
    (128, 40, 33000, 64, "bf16", None, True, True, 1),
    (4, 2, 4099, 5, "f32", [4099, 1], True, False, 64),
    (128, 2, 3000, 4, "f32", None, False, True, 1),
]


@pytest.mark.parametrize("ratio,B,pos,H,dtype,ragged,paged,rot_q,top_k", DECODE)
def test_decode(ratio, B, pos, H, dtype, ragged, paged, rot_q, top_k):
    c = Case(ratio, B, 1, pos, H, D=512 if dtype == "bf16" else 128, top_k=top_k, dtype=dtype,
             ragged=ragged, paged=paged, rot_q=rot_q)
    c.run()
    c.check()


CHUNK = [  # ratio, B, T, p0, H, dtype, ragged, paged, rot_q, top_k
    (4, 1, 2, 0, 64, "bf16", None, False, True, 512),
    (4, 1, 200, 0, 64, "bf16", None, False, False, 512),
    (4, 2, 130, 1000, 64, "bf16", [1000, 61], True, True, 300),
    (4, 1, 40, 5001, 128, "bf16", None, True, False, 77),
    (4, 2, 33, 400, 5, "bf16", None, False, True, 64),
    (128, 1, 300, 100, 64, "bf16", None, False, True, 1),
    (128, 2, 70, 33000, 24, "bf16", [33000, 0], True, False, 1),
    (4, 2, 9, 300, 5, "f32", [300, 2], True, True, 16),
    (128, 1, 50, 1000, 8, "f32", None, False, False, 1),
]


@pytest.mark.parametrize("ratio,B,T,p0,H,dtype,ragged,paged,rot_q,top_k", CHUNK)
def test_chunk(ratio, B, T, p0, H, dtype, ragged, paged, rot_q, top_k):
    c = Case(ratio, B, T, p0, H, D=512 if dtype == "bf16" else 192, top_k=top_k, dtype=dtype,
             ragged=ragged, paged=paged, rot_q=rot_q)
    c.run()
    pick = [(b, t) for b in range(B) for t in sorted({*range(0, T, max(1, T // 23)), T - 1})]
    c.check(pick)


@pytest.mark.parametrize("T", [1, 60])
@pytest.mark.parametrize("lists", [few, ends_early])
def test_lists_with_holes_and_early_ends(T, lists):
    c = Case(4, 3, T, 3000, 64, top_k=200, lists=lists, ragged=[3000, 5, 900])
    c.run()
    c.check([(b, t) for b in range(3) for t in range(0, T, 7)])


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("ratio", [4, 128])
def test_rows_that_are_not_attended_do_not_matter(T, ratio):
    """NaN rows behind the visible ones, in unlisted places and in other pages."""
    c = Case(ratio, 2, T, 4000, 64, top_k=64, paged=True, rot_q=True)
    c.run()
    c.check([(0, 0), (1, T - 1)])
    want, rpb = c.out.clone(), 256 // ratio
    last = [(int(c.p0[b]) + T) // ratio for b in range(2)]
    bad = torch.ones((c.c.n_blocks * rpb,), dtype=torch.bool, device=DEV)
    for b in range(2):
        rows = np.arange(last[b]) if ratio == 128 else np.unique(c.topk_np[b][c.topk_np[b] >= 0])
        bad[c.c.slots(c.rows.shape[1])[b].long()[torch.tensor(rows, device=DEV)]] = False
    c.c.attn_comp_kv.view(-1, 384)[bad] = 0xFF
    c.c.raw_kv.copy_(c.ring)
    c.out.fill_(3)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)


def test_large_scales_and_scores():
    """Rows of magnitude 2^40 and 2^-40 (scales beyond the quick path of the tile loader),
    and scores that differ by hundreds."""
    lib = lib_()
    for T in (1, 10):
        c = Case(4, 2, T, 2000, 64, top_k=100, rot_q=True, q_std=1e-3)
        cap = c.rows.shape[1]
        x = torch.randn((2 * cap, 512), device=DEV)
        x[::2] *= 2.0 ** 12
        x[1::4] *= 2.0 ** -40
        lib.ds4a_pack_rows(c.c, x.bfloat16(), c.c.slots(cap).reshape(-1))
        back = torch.empty_like(x.bfloat16())
        lib.ds4a_unpack_rows(c.c, back, c.c.slots(cap).reshape(-1))
        c.rows = np_(back).reshape(2, cap, 512).astype(np.float64)
        c.run()
        c.check([(0, 0), (1, T - 1)])


def test_odd_window_sizes_and_heads_of_other_sizes():
    for cap_raw in (1, 7, 200):
        c = Case(4, 2, 1, 700, 64, top_k=30, cap_raw=cap_raw, rot_q=True)
        c.run()
        c.check()
        c = Case(128, 1, 9, 700, 64, cap_raw=cap_raw)
        c.run()
        c.check()
    c = Case(4, 2, 1, 700, 7, D=1024, n_rot=16, top_k=30)
    c.run()
    c.check()
    c = Case(128, 2, 5, 700, 3, D=84, n_rot=4, dtype="f32")
    c.run()
    c.check()


def test_replayed_graph_and_other_stream():
    c = Case(4, 4, 1, 5000, 64, ragged=[5000, 100, 2, 4000], paged=True, rot_q=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    want = c.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for _ in range(3):
        c.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)
    c.check()


def test_decode_is_repeatable_on_one_workspace():
    """Calls of other sizes in between leave nothing behind in the workspace."""
    a = Case(128, 3, 1, 70000, 64, paged=True, rot_q=True)
    b = Case(4, 2, 1, 700, 24, top_k=50)
    a.run()
    torch.cuda.synchronize()
    want = a.out.clone()
    b.ws = a.ws if a.ws is not None and b.ws is not None and a.ws.numel() >= b.ws.numel() else b.ws
    for _ in range(4):
        b.run()
        a.run()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want)
    b.check()


@pytest.mark.parametrize("cluster", [1, 2, 3, 5, 0])
@pytest.mark.parametrize("T", [1, 5])
def test_tiles_without_a_row_before_ones_with_rows(T, cluster):
    """The first rows that a block meets may come tiles after its first tile: scores
    far below zero must not be lost against a maximum that no row had."""
    lib = lib_()
    c = Case(4, 2, T, 9000, 64, top_k=512, lists=late, rot_q=True, q_std=0.05)
    # every row close to -20 times the queries' mean: scores around -450
    big = torch.randn((1, 512), generator=torch.Generator().manual_seed(5)).to(DEV)
    cap = c.rows.shape[1]
    x = (0.1 * torch.randn((2 * cap, 512), device=DEV) - 20 * big).bfloat16()
    lib.ds4a_pack_rows(c.c, x, c.c.slots(cap).reshape(-1))
    back = torch.empty_like(x)
    lib.ds4a_unpack_rows(c.c, back, c.c.slots(cap).reshape(-1))
    c.rows = np_(back).reshape(2, cap, 512).astype(np.float64)
    c.q = (c.q.float() + big).bfloat16()
    c.ring.copy_((-21 * big).bfloat16().expand_as(c.ring))
    c.chunk.copy_((-21 * big).bfloat16().expand_as(c.chunk))
    c.c.raw_kv.copy_(c.ring)
    lib.ds4a_set_decode_cluster(cluster)
    try:
        c.run()
        c.check()
    finally:
        lib.ds4a_set_decode_cluster(0)


@pytest.mark.parametrize("ratio,pos", [(4, 9000), (128, 60000)])
def test_every_cluster_size(ratio, pos):
    lib = lib_()
    c = Case(ratio, 2, 1, pos, 40, top_k=1500, paged=True, rot_q=True)
    try:
        for C in range(1, 17):
            lib.ds4a_set_decode_cluster(C)
            c.out.fill_(9)
            c.run()
            c.check()
    finally:
        lib.ds4a_set_decode_cluster(0)


def test_chunk_with_lists_of_2048():
    c = Case(4, 1, 12, 12000, 64, top_k=2048, paged=True)
    c.run()
    c.check()


@pytest.mark.parametrize("ratio", [0, 128])
def test_queries_and_rows_written_by_the_launch_before(ratio):
    """ds4a_norm_rope, then the attention at once, again and again with other inputs: the
    results are those of the same calls with a wait between them."""
    lib = lib_()
    B, H, D, pos = 8, 64, 512, 3000
    qat = lib.Q_ROTATED | (lib.FP4_ROWS if ratio else 0)
    c = lib.LayerCache(ratio=ratio, head_dim=D, n_rot=64, batch=B, comp_cap=24 if ratio else 0,
                       dtype="bf16", base=BASE, rope_max_pos=pos + 1, qat=qat, device=DEV)
    c.n_tokens = pos + 1
    c.raw_kv.normal_()
    if ratio:
        lib.ds4a_pack_rows(c, torch.randn((B * 24, D), device=DEV).bfloat16())
    p = torch.full((B,), pos, dtype=torch.int32, device=DEV)
    slots = (torch.arange(B, device=DEV) * 128 + pos % 128).int()
    x = [torch.randn((B, (H + 1) * D), device=DEV).bfloat16() for _ in range(40)]
    q = torch.empty((B, H, D), dtype=torch.bfloat16, device=DEV)
    ws = lib.workspace(c.workspace_bytes(lib.CALL_ATTN_DECODE, 1, H, 1))
    got = [torch.empty_like(q) for _ in x]
    want = [torch.empty_like(q) for _ in x]
    for out, wait in ((want, True), (got, False), (got, False)):
        for xi, o in zip(x, out):
            lib.ds4a_norm_rope(c, p, q=xi[:, :H * D].view(B, H, D), q_out=q, kv=xi[:, H * D:],
                               slots=slots, rot_q=True)
            if wait:
                torch.cuda.synchronize()
            lib.ds4a_sparse_attn_decode(c, pos, q, H, None, 1, lib.default_scale(D), o, ws)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_first_call_inside_a_capture():
    """In a process of its own: nothing of the library ran before the capture."""
    import subprocess
    import sys
    code = """
import sys; sys.path.insert(0, 'tests'); sys.path.insert(0, '.')
import torch, test_gpu_fp4_attention as t
from compressed_kv_sparse_gb300 import lib
c = t.Case(4, 2, 1, 700, 64, top_k=50, rot_q=True)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c.run()
g.replay()
c.check()
print('captured')
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("ratio,p0", [(4, 0), (4, 127), (4, 3001), (128, 130), (128, 20479)])
def test_chunk_of_one_token(ratio, p0):
    """The token's row is in the chunk alone, its slot of the ring still holds position
    p - 128's."""
    c = Case(ratio, 2, 1, p0, 64, top_k=300, rot_q=True)
    call = lib_().CALL_ATTN_PREFILL
    c.ws = lib_().workspace(c.c.workspace_bytes(call, 1, 64, 300))
    c.c.raw_kv[:, p0 % 128] = -3.0
    lib_().ds4a_sparse_attn_prefill_chunk(c.c, p0, 1, c.q, 64, c.chunk, c.topk, c.k, c.scale, c.out,
                                          c.ws)
    c.check()
    assert torch.equal(c.c.raw_kv[:, p0 % 128], c.chunk[:, 0])


@pytest.mark.parametrize("T", [1, 30])
def test_rows_behind_as_many_places_as_are_visible(T):
    """A list with fewer visible rows than places, all of them in its last places (entries
    below 0 are skipped wherever they are)."""
    def last(rng, row, vis):
        m = int((row >= 0).sum())
        row[:] = np.concatenate([row[m:], row[:m]])

    c = Case(4, 3, T, 900, 64, top_k=512, lists=last, ragged=[900, 13, 300])
    c.run()
    c.check([(b, t) for b in range(3) for t in range(0, T, 7)])


@pytest.mark.parametrize("ratio,T,dtype", [(4, 1, "bf16"), (4, 9, "bf16"), (128, 1, "bf16"),
                                           (4, 1, "f32")])
def test_pool_offsets_pass_32_bits(ratio, T, dtype):
    """The same rows at the far end of a pool of more than 4 GiB: the same output."""
    lib = lib_()
    D = 512 if dtype == "bf16" else 128
    c = Case(ratio, 2, T, 5000, 64 if dtype == "bf16" else 5, D=D, top_k=100, dtype=dtype, paged=True)
    c.run()
    c.check()
    rpb, near = 256 // ratio, c.c.n_blocks
    far = (1 << 32) // (384 * rpb) + 1
    table = torch.where(c.c.block_table >= 0, c.c.block_table + far, -1).int()
    big = lib.LayerCache(ratio=ratio, head_dim=D, n_rot=64, batch=2, comp_cap=c.rows.shape[1],
                         dtype=dtype, base=BASE, rope_max_pos=5000 + T, index_dim=32, index_rot=32,
                         qat=lib.FP4_ROWS, device=DEV, block_table=table, n_blocks=far + near)
    big.attn_comp_kv[far:] = c.c.attn_comp_kv
    big.raw_kv.copy_(c.ring)
    big.n_tokens = 5000 + T
    want, c.c = c.out.clone(), big
    c.out.fill_(7)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)


def test_two_calls_at_once():
    """Calls on two streams, a workspace each."""
    a = Case(128, 3, 1, 70000, 64, paged=True, rot_q=True)
    b = Case(4, 2, 40, 700, 64, top_k=200)
    cases, streams = (a, b), (torch.cuda.Stream(), torch.cuda.Stream())
    for c in cases:
        c.run()
    torch.cuda.synchronize()
    want = [c.out.clone() for c in cases]
    b.c.raw_kv.copy_(b.ring)
    for _ in range(5):
        for c, s in zip(cases, streams):
            c.out.zero_()
            s.wait_stream(torch.cuda.current_stream())
            c.run(stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(c.out, w) for c, w in zip(cases, want))
        b.c.raw_kv.copy_(b.ring)
