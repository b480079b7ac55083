"""Argument checks of the calls around a paged cache of keys and values (CPU: every check is made
on the host before any launch), their structs and tables."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

from compressed_kv_sparse_gb300 import lib
from oracle import kv
from test_abi_cpu import HEADER, L  # noqa: F401  (L: the library fixture)

FAKE = 0x1000


def spec(**kw):
    return lib.RopeSpecC(**{**dict(rot_at=0, n_rot=64, max_pos=100, flags=0, cos=FAKE, sin=FAKE), **kw})


def cache(rope=None, **kw):
    a = dict(head_dim=128, n_kv_heads=4, batch=2, max_blocks=3, n_blocks=7, dtype=lib.DS4A_BF16,
             kv_dtype=lib.DS4A_BF16, k=FAKE, v=FAKE, k_scale=None, v_scale=None, block_table=FAKE, seq_pos=FAKE)
    return lib.KvCacheC(**{**a, **kw}, rope=rope or spec())


def test_structs_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    fields = {"ds4a_rope_spec": lib.RopeSpecC, "ds4a_kv_cache": lib.KvCacheC}
    body = "".join(f'printf("%zu ", offsetof({n}, {f[0]}));' for n, c in fields.items() for f in c._fields_)
    body += "".join(f'printf("%zu ", sizeof({n}));' for n in fields)
    src.write_text(f'#include <stdio.h>\n#include "{HEADER}"\nint main(){{{body}return 0;}}')
    exe = tmp_path / "s"
    subprocess.check_call(["gcc", str(src), "-o", str(exe)])
    want = [getattr(c, f[0]).offset for c in fields.values() for f in c._fields_] + [ctypes.sizeof(c) for c in fields.values()]
    assert [int(x) for x in subprocess.check_output([str(exe)]).split()] == want


@pytest.mark.parametrize("kind", ["none", "linear", "ntk", "yarn"])
def test_scaled_tables(L, kind):
    n_rot, n_pos = 64, 3000
    c, s = np.empty((n_pos, 32), np.float32), np.empty((n_pos, 32), np.float32)
    args = (1e4, 8.0, 512.0, 32.0, 1.0, 0.0)
    assert L.ds4a_rope_table_scaled(lib.SCALINGS[kind], *args, n_rot, n_pos, c.ctypes.data, s.ctypes.data) == 0
    th, mag = kv.theta(n_rot, 1e4, kind=kind, factor=8.0, orig_len=512.0)
    a = np.arange(n_pos)[:, None] * th
    # (one rounding of values up to mag; the angles' fp64 differ by 2^-50 of 3000)
    assert np.abs(c - mag * np.cos(a)).max() <= mag * 2.0 ** -24 + 1e-11
    assert np.abs(s - mag * np.sin(a)).max() <= mag * 2.0 ** -24 + 1e-11
    if kind == "none":
        c0, s0 = np.empty_like(c), np.empty_like(s)
        assert L.ds4a_rope_table(1e4, n_rot, n_pos, c0.ctypes.data, s0.ctypes.data) == 0
        assert np.array_equal(c, c0) and np.array_equal(s, s0)


def test_scaled_table_checks(L):
    buf = np.empty(64, np.float32).ctypes.data
    ok = dict(kind=3, base=1e4, factor=4.0, orig=512.0, fast=32.0, slow=1.0, mag=0.0, n_rot=8, n_pos=2, c=buf, s=buf)
    call = lambda **kw: L.ds4a_rope_table_scaled(*{**ok, **kw}.values())  # noqa: E731
    assert call() == 0 and call(mag=1.0) == 0 and call(n_pos=0) == 0
    inf, nan = float("inf"), float("nan")
    for bad in (dict(kind=4), dict(kind=-1), dict(base=1.0), dict(base=nan), dict(base=inf), dict(factor=0.5),
                dict(factor=nan), dict(factor=inf), dict(orig=0.0), dict(orig=inf), dict(fast=0.0), dict(slow=-1.0), dict(slow=nan),
                dict(mag=-1.0), dict(mag=nan), dict(n_rot=7), dict(n_rot=0), dict(c=None), dict(s=None), dict(kind=2, n_rot=2)):
        assert call(**bad) == -1, bad


def test_rope_checks(L):
    ok = dict(dtype=1, n=0, pos=FAKE, x=FAKE, xs=512, H=4, D=128, y=2 * FAKE, ys=512)

    def call(rope=None, none=False, **kw):
        a = {**ok, **kw}
        r = rope or spec()
        return L.ds4a_rope(None if none else ctypes.byref(r), a["dtype"], a["n"], a["pos"], a["x"], a["xs"], a["H"],
                           a["D"], a["y"], a["ys"], None)

    assert call() == 0 and call(spec(n_rot=0, cos=None, sin=None)) == 0 and call(spec(flags=3)) == 0
    assert call(none=True) == -1 and call(spec(flags=4)) == -1
    assert call(dtype=2) == -5 and call(dtype=-1) == -5
    for bad in (dict(D=0), dict(D=514), dict(D=127), dict(H=0), dict(H=1025, xs=1 << 20, ys=1 << 20), dict(xs=511),
                dict(ys=511), dict(n=1 << 31)):
        assert call(**bad) == -2, bad
    for bad in (dict(n_rot=63), dict(n_rot=130), dict(rot_at=66), dict(rot_at=1), dict(rot_at=0xfffffffe)):
        assert call(spec(**bad)) == -2, bad
    for bad in (dict(cos=None), dict(sin=None), dict(max_pos=0), dict(cos=FAKE + 2)):
        assert call(spec(**bad)) == -1, bad
    for bad in (dict(pos=None), dict(x=None), dict(y=None), dict(pos=FAKE + 2), dict(x=FAKE + 1), dict(y=FAKE + 1),
                dict(y=FAKE, ys=600)):
        assert call(n=1, **bad) == -1, bad


def test_append_checks(L):
    ok = dict(n=0, seq=FAKE, pos=FAKE, k=FAKE, ks=512, v=FAKE, vs=512, q=FAKE, qs=1024, H=8, qo=2 * FAKE)

    def call(c=None, none=False, **kw):
        a = {**ok, **kw}
        c = c or cache()
        return L.ds4a_kv_append(None if none else ctypes.byref(c), a["n"], a["seq"], a["pos"], a["k"], a["ks"], a["v"],
                                a["vs"], a["q"], a["qs"], a["H"], a["qo"], None)

    assert call() == 0 and call(q=None, qo=None, H=0, qs=0) == 0 and call(cache(spec(n_rot=0, cos=None, sin=None))) == 0
    assert call(none=True) == -1
    f8 = dict(kv_dtype=lib.DS4A_E4M3, k_scale=FAKE, v_scale=FAKE)
    assert call(cache(**f8)) == 0
    for bad in (dict(f8, k_scale=None), dict(f8, v_scale=None), dict(k_scale=FAKE), dict(k=None), dict(v=None),
                dict(block_table=None), dict(k=FAKE + 8), dict(v=FAKE + 8), dict(block_table=FAKE + 2), dict(f8, k_scale=FAKE + 2)):
        assert call(cache(**bad)) == -1, bad
    assert call(cache(spec(flags=2))) == -1 and call(cache(spec(n_rot=130))) == -2
    for bad in (dict(dtype=2), dict(dtype=3), dict(kv_dtype=0), dict(kv_dtype=7)):
        assert call(cache(**bad)) == -5, bad
    for bad in (dict(head_dim=0), dict(head_dim=258), dict(head_dim=127), dict(n_kv_heads=0), dict(n_kv_heads=129),
                dict(batch=0), dict(batch=8193), dict(max_blocks=0), dict(max_blocks=(1 << 23) + 1), dict(n_blocks=0),
                dict(n_blocks=(1 << 31) // 1024)):
        assert call(cache(**bad)) == -2, bad
    for bad in (dict(ks=511), dict(vs=511), dict(qs=1023), dict(n=1 << 31), dict(H=1025, qs=1 << 20), dict(H=0)):
        assert call(**bad) == -2, bad
    for bad in (dict(q=None), dict(qo=None), dict(q=FAKE, qo=FAKE, qs=1032)):
        assert call(**bad) == -1, bad
    for bad in (dict(seq=None), dict(pos=None), dict(k=None), dict(v=None), dict(k=FAKE + 1), dict(qo=FAKE + 1),
                dict(seq=FAKE + 2), dict(q=None, qo=None)):
        assert call(n=1, **bad) == -1, bad


def test_attention_checks(L):
    ok = dict(cu=FAKE, new=2, q=FAKE, qs=1024, H=8, win=0, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, wb=1 << 40)

    def call(c=None, none=False, **kw):
        a = {**ok, **kw}
        c = c or cache()
        return L.ds4a_paged_attn_decode(None if none else ctypes.byref(c), a["cu"], a["new"], a["q"], a["qs"], a["H"],
                                        a["win"], a["scale"], a["out"], a["lse"], a["ws"], a["wb"], None)

    assert call(none=True) == -1 and call(cache(dtype=3)) == -5
    for bad in (dict(new=0), dict(new=257), dict(H=0), dict(H=6), dict(H=1028, qs=1 << 20), dict(qs=1023)):
        assert call(**bad) == -2, bad
    for bad in (dict(q=None), dict(out=None), dict(q=FAKE + 1), dict(out=FAKE + 1), dict(cu=FAKE + 2), dict(lse=FAKE + 2),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=FAKE + 8)):
        assert call(**bad) == -1, bad
    assert call(cache(seq_pos=None)) == -1
    need = L.ds4a_paged_attn_ws_bytes(ctypes.byref(cache()), 2, 8)
    assert need >= 256
    assert call(ws=None) == -8 and call(wb=need - 1) == -8
    for c, new, H in ((cache(), 0, 8), (cache(), 2, 6), (cache(head_dim=300), 1, 8), (cache(dtype=5), 1, 8)):
        assert L.ds4a_paged_attn_ws_bytes(ctypes.byref(c), new, H) == 0
    assert L.ds4a_paged_attn_ws_bytes(None, 1, 8) == 0


def test_verify_checks(L):
    ok = dict(dtype=0, B=2, N=3, V=10, cu=FAKE, pos=FAKE, d=FAKE, t=FAKE, ts=10, dp=FAKE, ua=FAKE, us=FAKE, tok=FAKE,
              n=FAKE, ctx=FAKE)
    call = lambda **kw: L.ds4a_verify_drafts(*{**ok, **kw}.values(), None)  # noqa: E731
    assert call(dtype=2) == -5
    for bad in (dict(B=0), dict(B=8193), dict(N=0), dict(N=256), dict(V=0), dict(V=(1 << 20) + 1, ts=1 << 21), dict(ts=9)):
        assert call(**bad) == -2, bad
    for bad in (dict(d=None), dict(t=None), dict(ua=None), dict(us=None), dict(tok=None), dict(n=None), dict(pos=None),
                dict(t=FAKE + 2), dict(dp=FAKE + 2), dict(cu=FAKE + 1), dict(tok=FAKE + 2), dict(ctx=FAKE + 2)):
        assert call(**bad) == -1, bad


# ------------------------------------------------- the binding's own checks

BF, I32, F32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32), dict(dtype=torch.float32)


def py_cache(**kw):
    a = dict(head_dim=16, n_kv_heads=2, batch=2, block_table=torch.zeros((2, 3), **I32), n_blocks=4, device="cpu",
             rope=lib.Rope(n_rot=8, max_pos=20, base=1e4, device="cpu"))
    return lib.KvCache(**{**a, **kw})


def py_calls(dev="cpu"):
    """Every call with tensors that suit it but for their device, and wrong ones for each argument."""
    t = lambda *s, **k: torch.zeros(s, device=dev, **(k or BF))  # noqa: E731
    c = py_cache()
    c.set_seq_pos(torch.zeros(2, **I32))
    rope, n = c.rope, 4
    seq, kk, q = t(n, **I32), t(n, 2, 16), t(n, 4, 16)
    ws, cu = t(1 << 16, dtype=torch.uint8), t(3, **I32)
    tg, dr, ua, us = t(8, 10, **F32), t(2, 3, **I32), t(2, 3, **F32), t(2, **F32)
    return c, {
        "rope": (lib.ds4a_rope, (rope, seq, q, q.clone()), {}, [(1, seq.long()), (1, t(3, **I32)), (2, q.double()), (2, q[:, 0]),
                 (3, q[:2]), (3, q.float()), (2, q.transpose(0, 1).contiguous().transpose(0, 1))]),
        "append": (lib.ds4a_kv_append, (c, seq, seq, kk, kk), dict(q=q, q_out=q.clone()),
                   [(1, seq.long()), (2, t(3, **I32)), (3, kk.float()), (3, kk[:, :1]), (4, kk[:2]), ("q", q.float()),
                    ("q", None), ("q_out", q[:2]), ("q_out", None), ("q", q[:, :, ::2])]),
        "attn": (lib.ds4a_paged_attn_decode, (c, q, q.clone(), ws), dict(max_new=2, cu_len=cu, lse=t(n, 4, **F32)),
                 [(1, q.float()), (1, q[:, 0]), (2, q[:2]), ("lse", t(3, **F32)), ("lse", t(n, 4)), ("cu_len", t(2, **I32)),
                  ("cu_len", cu.long())]),
        "verify": (lib.ds4a_verify_drafts, (tg, dr, ua, us, t(2, 4, **I32), t(2, **I32)),
                   dict(draft_probs=t(2, 3, 10, **F32), cu_len=cu, seq_pos=t(2, **I32), ctx_out=t(2, **I32)),
                   [(0, tg.double()), (0, tg[:, ::2]), (1, dr.long()), (2, ua[:1]), (3, us.double()), (4, t(2, 3, **I32)),
                    (5, us), ("draft_probs", t(2, 3, 10)), ("cu_len", t(2, **I32)), ("seq_pos", us)]),
    }


@pytest.mark.parametrize("name", ["rope", "append", "attn", "verify"])
def test_binding_refuses(L, name):
    c, calls = py_calls()
    fn, args, kw, bad = calls[name]
    with pytest.raises(lib.ArgumentError, match="not on a GPU"):
        fn(*args, **kw)
    for key, value in bad:
        a, k = list(args), dict(kw)
        if isinstance(key, int):
            a[key] = value
        else:
            k[key] = value
        with pytest.raises(lib.ArgumentError) as e:
            fn(*a, **k)
        assert "not on a GPU" not in str(e.value), (name, key)
    if name != "verify":   # the cache (or tables) on what says it is a GPU, the tensors on the CPU
        (c.rope if name == "rope" else c).dev = 0
        with pytest.raises(lib.ArgumentError, match="device|on cpu"):
            fn(*args, **kw, stream=0)


def test_binding_without_tokens(L):
    c, calls = py_calls()
    e = torch.zeros((0, 4, 16), **BF)
    lib.ds4a_rope(c.rope, torch.zeros(0, **I32), e, e)
    lib.ds4a_kv_append(c, torch.zeros(0, **I32), torch.zeros(0, **I32), e[:, :2], e[:, :2])
    lib.ds4a_paged_attn_decode(c, e, e, torch.zeros(8, dtype=torch.uint8), cu_len=torch.zeros(3, **I32))


def test_caches(L):
    for bad in (dict(block_table=torch.zeros((3, 3), **I32)), dict(block_table=torch.zeros((2, 3))), dict(dtype="e4m3"),
                dict(kv_dtype="f32"), dict(kv_dtype="e4m3"), dict(k_scale=torch.ones(2), v_scale=torch.ones(2)),
                dict(k=torch.zeros((4, 2, 256, 8), **BF)), dict(v=torch.zeros((4, 2, 256, 16))),
                dict(kv_dtype="e4m3", k_scale=torch.ones(2), v_scale=torch.ones(3))):
        with pytest.raises(lib.ArgumentError):
            py_cache(**bad)
    c = py_cache(kv_dtype="e4m3", k_scale=torch.ones(2), v_scale=torch.ones(2), rope=None)
    assert c.k.dtype is torch.float8_e4m3fn and c.k.shape == (4, 2, 256, 16) and c.c.rope.n_rot == 0
    with pytest.raises(lib.ArgumentError):
        c.set_seq_pos(torch.zeros(3, **I32))
    with pytest.raises(lib.Ds4aError):
        c.attn_workspace_bytes(3)
    with pytest.raises(lib.ArgumentError):
        lib.Rope(n_rot=8, max_pos=4, base=1e4, scaling="dynamic", device="cpu")
    with pytest.raises(lib.Ds4aError):
        lib.Rope(n_rot=7, max_pos=4, base=1e4, device="cpu")


def test_overlapping_rows_are_refused(L):
    """Out and in may be the same rows, or other columns of one buffer (test_gpu_rope.py); else they race."""
    r, big = spec(), 1 << 20

    def rope(x, xs, y, ys, n=3):   # rows of 512 bf16 elements
        return L.ds4a_rope(ctypes.byref(r), 1, n, FAKE, x, xs, 4, 128, y, ys, None)

    for x, xs, y, ys in [(big, 512, big + 2, 512), (big, 512, big + 1024, 512), (big, 512, big + 256, 512),
                         (big + 256, 512, big, 512), (big, 600, big + 1000, 600), (big, 600, big + 1200, 600),
                         (big, 600, big + 400, 600), (big, 512, big + 1024, 600), (big + 900, 600, big, 512)]:
        assert rope(x, xs, y, ys) == -1, (x, xs, y, ys)
    assert rope(big, 512, big + 1022, 512, n=1) == -1 and rope(big + 1022, 512, big, 512, n=1) == -1


def test_overlapping_queries_are_refused(L):
    c, big = cache(), 1 << 20
    call = lambda q, qs, qo: L.ds4a_kv_append(ctypes.byref(c), 3, FAKE, FAKE, FAKE, 512, FAKE, 512, q, qs, 4, qo, None)  # noqa: E731
    for q, qs, qo in [(big, 512, big + 2), (big, 1536, big + 1024), (big + 1024, 512, big)]:
        assert call(q, qs, qo) == -1, (q, qs, qo)
