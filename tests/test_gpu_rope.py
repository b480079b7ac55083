"""ds4a_rope and ds4a_kv_append against oracle/kv.py, and bit for bit against the fp32 arithmetic
that ds4a.h states.

Tolerance, from the arithmetic, u = 2^-24: a coefficient is off by u of the magnitude, a product by u and the
sum by u: 3 u (|a| + |b|) mag for a pair (a, b), plus half a step of the stored type; the angle (fp64) adds
p 2^-52 at most."""
import numpy as np
import pytest
import torch

from helpers import np_
from kv_step import BLOCK, TD, bits, rand, table_for
from oracle import kv
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV, MAXP, BASE = "cuda", 9000, 10000.0
SCALED = {"none": {}, "linear": dict(factor=8.0), "ntk": dict(factor=8.0),
          "yarn": dict(factor=16.0, orig_len=1024.0)}


def make_rope(rot, rot_at=0, half=False, kind="none", max_pos=MAXP):
    return lib_().Rope(n_rot=rot, max_pos=max_pos, base=BASE, rot_at=rot_at, half=half, scaling=kind,
                       device=DEV, **SCALED[kind])


def recipe(x, pos, rope, inverse=False):
    """The stated fp32 arithmetic on the library's tables (fp32 result)."""
    x = np_(x).astype(np.float32).copy()
    c, s = (np_(t)[np.asarray(pos)][:, None] for t in (rope.cos, rope.sin))
    s = -s if inverse else s
    r = x[..., rope.rot_at:rope.rot_at + rope.n_rot]
    h = rope.n_rot // 2
    a, b = (slice(0, h), slice(h, None)) if rope.half else (slice(0, None, 2), slice(1, None, 2))
    y = r.copy()
    y[..., a], y[..., b] = r[..., a] * c - r[..., b] * s, r[..., a] * s + r[..., b] * c
    x[..., rope.rot_at:rope.rot_at + rope.n_rot] = y
    return x


def near(got, x, pos, rope, kind, dtype, inverse=False):
    x = np_(x).astype(np.float64)
    kw = dict(kind=kind, **SCALED[kind])
    want = kv.rotate(x, pos, rope.n_rot, BASE, rope.rot_at, rope.half, inverse, **kw)
    mag = kv.theta(rope.n_rot, BASE, **kw)[1]
    both = np.zeros_like(x)
    r = np.abs(x[..., rope.rot_at:rope.rot_at + rope.n_rot])
    h = rope.n_rot // 2
    p = (r[..., :h] + r[..., h:]) if rope.half else (r[..., 0::2] + r[..., 1::2])
    both[..., rope.rot_at:rope.rot_at + rope.n_rot] = np.concatenate([p, p], -1) if rope.half else np.repeat(p, 2, -1)
    tol = (3 * 2.0 ** -24 + 2.0 ** -36) * mag * both + torch.finfo(TD[dtype]).eps / 2 * np.abs(want) + 1e-38
    err = np.abs(np_(got).astype(np.float64) - want)
    assert (err <= tol).all(), float((err / tol).max())


CASES = [  # n, H, D, rot_at, rot, half, kind, inverse, dtype, extra elements per token
    (1, 1, 128, 0, 128, True, "none", False, "bf16", 0), (8, 64, 128, 0, 128, True, "yarn", False, "bf16", 0),
    (77, 3, 512, 448, 64, False, "linear", False, "bf16", 64), (333, 5, 96, 0, 32, True, "ntk", True, "f32", 0),
    (5, 2, 10, 2, 6, False, "none", False, "f32", 3), (5, 2, 10, 4, 6, True, "none", True, "bf16", 1),
    (19, 7, 80, 16, 40, True, "yarn", False, "bf16", 0), (4, 3, 64, 0, 2, False, "none", False, "f32", 8),
    (2, 1024, 16, 8, 8, False, "none", False, "bf16", 0), (9, 2, 512, 0, 510, True, "none", False, "f32", 0),
    (700, 1, 2, 0, 2, True, "none", False, "bf16", 0), (3, 4, 64, 0, 0, False, "none", False, "bf16", 0),
    (1, 5, 192, 64, 96, False, "ntk", False, "bf16", 16),
]


@pytest.mark.parametrize("n,H,D,rot_at,rot,half,kind,inverse,dtype,extra", CASES)
def test_rope(n, H, D, rot_at, rot, half, kind, inverse, dtype, extra):
    lib = lib_()
    g = torch.Generator().manual_seed(n * H + D)
    rope = make_rope(rot or 2, rot_at, half, kind)
    rope.c.n_rot = rope._back.n_rot = rope.n_rot = rot
    wide = rand(g, n, H * D + extra, dtype=TD[dtype]).to(DEV)
    x = wide[:, :H * D].view(n, H, D)
    pos = torch.randint(0, MAXP, (n,), generator=g, dtype=torch.int32)
    y = torch.full((n, H, D), 7.0, dtype=TD[dtype], device=DEV)
    lib.ds4a_rope(rope, pos.to(DEV), x, y, inverse=inverse)
    if rot:
        near(y, x, pos.numpy(), rope, kind, dtype, inverse)
        want = torch.from_numpy(recipe(x, pos.numpy(), rope, inverse)).to(TD[dtype])
        assert torch.equal(y.cpu(), want)
    else:
        assert torch.equal(y, x)
    before = wide.clone()                               # in place, on the strided tokens
    lib.ds4a_rope(rope, pos.to(DEV), x, x, inverse=inverse)
    assert torch.equal(x, y) and torch.equal(wide[:, H * D:], before[:, H * D:])


def test_rope_skips_positions_out_of_range_and_takes_no_tokens():
    lib = lib_()
    rope = make_rope(32, 0, True, max_pos=50)
    x = torch.randn((4, 2, 64), device=DEV)
    y = torch.full_like(x, 3.0)
    lib.ds4a_rope(rope, torch.tensor([0, -1, 50, 49], dtype=torch.int32, device=DEV), x, y)
    assert (y[1:3] == 3).all() and torch.equal(y[0], x[0]) and not (y[3] == 3).any()
    lib.ds4a_rope(rope, torch.zeros(0, dtype=torch.int32, device=DEV), x[:0], y[:0])


def test_rotation_back_is_the_gradient():
    """d <w, rot(x)> / dx by differences of the linear map, and the round trip."""
    lib = lib_()
    rope = make_rope(24, 4, False, "yarn")
    g = torch.Generator().manual_seed(5)
    x, w = (rand(g, 3, 2, 40).to(DEV) for _ in range(2))
    pos = torch.tensor([0, 77, 8999], dtype=torch.int32, device=DEV)
    gx, y0, y1 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    lib.ds4a_rope(rope, pos, w, gx, inverse=True)
    lib.ds4a_rope(rope, pos, x, y0)
    for d in (0, 4, 5, 17, 27, 28, 39):
        e = x.clone()
        e[:, :, d] += 1.0
        lib.ds4a_rope(rope, pos, e, y1)
        slope = ((y1 - y0).double() * w.double()).sum(-1)
        # both sides' roundings: 3 u of pairs of magnitude <= 6 times |w| <= 5, over two dims and four maps
        assert (slope - gx[:, :, d].double()).abs().max() <= 8 * 3 * 2.0 ** -24 * 2 * 6 * 5


APPEND = [  # old lengths, new tokens, H, K, D, rot, half, dtype, kv_dtype
    ([0], [1], 1, 1, 128, 128, True, "bf16", "bf16"),
    ([255, 256, 0, 511, 30], [1, 1, 1, 1, 1], 16, 2, 128, 64, False, "bf16", "e4m3"),
    ([250, 0], [13, 300], 4, 4, 64, 64, True, "bf16", "bf16"),
    ([7, 0, 300], [5, 0, 2], 3, 1, 80, 32, True, "f32", "f32"),
    ([100], [600], 8, 2, 96, 96, False, "f32", "e4m3"),
    ([3, 9], [2, 3], 6, 3, 10, 6, False, "bf16", "e4m3"),
    ([3, 9], [2, 3], 0, 2, 256, 0, False, "bf16", "bf16"),
]


@pytest.mark.parametrize("old,new,H,K,D,rot,half,dtype,kvd", APPEND)
def test_append(old, new, H, K, D, rot, half, dtype, kvd):
    lib = lib_()
    g = torch.Generator().manual_seed(sum(old) + D)
    old, new = np.array(old), np.array(new)
    table, nb = table_for(g, old + new)
    n = int(new.sum())
    seq = np.repeat(np.arange(len(old)), new)
    pos = np.concatenate([np.arange(o, o + m) for o, m in zip(old, new)]).astype(np.int32)
    order = torch.randperm(n, generator=g).numpy()       # (any order of the tokens)
    seq, pos = seq[order].astype(np.int32), pos[order]
    rope = make_rope(rot, 0, half, "yarn") if rot else None
    qkv = rand(g, n, (H + 2 * K) * D + 3, dtype=TD[dtype], std=2.0)
    if kvd == "e4m3" and n > 2:
        qkv[0, H * D], qkv[1, H * D + 1], qkv[2, -5] = float("nan"), 3e4, float("-inf")
    qkv = qkv.to(DEV)
    cut = lambda a, b: qkv[:, a * D:b * D].view(n, b - a, D)  # noqa: E731
    q, k, v = cut(0, H), cut(H, H + K), cut(H + K, H + 2 * K)
    f8 = kvd == "e4m3"
    ks, vs = (torch.rand(K, generator=g) * 0.02 + 0.01 for _ in range(2))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    c = lib.KvCache(head_dim=D, n_kv_heads=K, batch=len(old), block_table=i32(table), n_blocks=nb, dtype=dtype,
                    kv_dtype=kvd, k_scale=ks.to(DEV) if f8 else None, v_scale=vs.to(DEV) if f8 else None,
                    rope=rope, device=DEV)
    for p in (c.k, c.v):
        bits(p).fill_(0x11 if f8 else 3.0)
    q_out = torch.full((n, H, D), 5.0, dtype=TD[dtype], device=DEV) if H else None
    lib.ds4a_kv_append(c, i32(seq), i32(pos), k, v, q=q if H else None, q_out=q_out)
    turn = (lambda x: recipe(x, pos, rope)) if rot else (lambda x: np_(x).astype(np.float32))
    if H:
        assert torch.equal(q_out.cpu(), torch.from_numpy(turn(q)).to(TD[dtype]))
        if rot:
            near(q_out, q, pos, rope, "yarn", dtype)
    for pool, x, scale in ((c.k, turn(k), ks), (c.v, np_(v).astype(np.float32), vs)):
        if f8:   # bit for bit: the fp32 product with the reciprocal, then the nearest value
            x = kv.to_e4m3(x * (np.float32(1) / scale.numpy())[None, :, None])
            want = np.full((nb, K, BLOCK, D), kv.e4m3_table()[0x11])
            got = kv.e4m3_table()[bits(pool).cpu().numpy()]
        else:
            x = np_(torch.from_numpy(x).to(TD[dtype]))
            want, got = np.full((nb, K, BLOCK, D), 3.0), np_(pool)
        kv.append(want, want.copy(), table, seq, pos, x, x)
        assert np.array_equal(got, want, equal_nan=True)
    if H:                                                # in place
        flat = q.contiguous()
        lib.ds4a_kv_append(c, i32(seq), i32(pos), k, v, q=flat, q_out=flat)
        assert torch.equal(flat, q_out)


def test_append_leaves_out_what_has_no_place():
    """Sequences out of range, positions beyond the tables or the blocks, blocks that are not there."""
    lib = lib_()
    rope = make_rope(16, 0, False, max_pos=600)
    table = torch.tensor([[1, -1, 7], [0, 2, 1]], dtype=torch.int32, device=DEV)
    c = lib.KvCache(head_dim=16, n_kv_heads=1, batch=2, block_table=table, n_blocks=3, dtype="f32", rope=rope, device=DEV)
    seq = [0, 0, 0, 1, 2, -1, 1, 1, 0]
    pos = [3, 256, 520, 300, 5, 5, 600, -1, 768]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    k, v, q = (torch.randn((9, 1, 16), device=DEV) for _ in range(3))
    q_out = torch.full_like(q, 9.0)
    lib.ds4a_kv_append(c, i32(seq), i32(pos), k, v, q=q, q_out=q_out)
    assert torch.equal(c.v[1, 0, 3], v[0, 0]) and torch.equal(c.v[2, 0, 44], v[3, 0])
    c.v[1, 0, 3], c.v[2, 0, 44] = 0, 0
    assert not c.v.any()
    # queries of tokens without a block are rotated; those of skipped tokens stay
    done = (q_out != 9).flatten(1).any(1).tolist()
    assert done == [True, True, True, True, False, False, False, False, False]


@pytest.mark.parametrize("swap", [False, True])
def test_rope_between_columns_of_one_buffer(swap):
    """Out beside in, in the same rows and behind them; what overlaps is refused."""
    lib, n, H, D = lib_(), 9, 3, 64
    rope = make_rope(64, 0, True)
    pos = torch.arange(n, dtype=torch.int32, device=DEV) * 7
    wide = torch.randn((2 * n, 2 * H * D + 8), device=DEV)
    cols = [wide[:n, :H * D].view(n, H, D), wide[:n, H * D:2 * H * D].view(n, H, D)]
    x, y = cols[::-1] if swap else cols
    want = torch.empty((n, H, D), device=DEV)
    lib.ds4a_rope(rope, pos, x, want)
    lib.ds4a_rope(rope, pos, x, y)
    assert torch.equal(y, want)
    below = wide[n:, :H * D].view(n, H, D)
    lib.ds4a_rope(rope, pos, x, below)
    assert torch.equal(below, want)
    before = wide.clone()
    for other in (wide[1:n + 1, :H * D].view(n, H, D), wide[:n, 8:8 + H * D].view(n, H, D),
                  wide.view(-1)[:n * H * D].view(n, H, D)):
        with pytest.raises(lib.Ds4aError):
            lib.ds4a_rope(rope, pos, cols[0], other)
    assert torch.equal(wide, before)
