"""Argument checks of the serving calls and of a cache with 4-bit rows (CPU: every
check is made on the host before any launch), and their sizes."""
import ctypes

import pytest

from compressed_kv_sparse_gb300 import lib
from oracle import serving
from test_abi_cpu import L, _fake_cache  # noqa: F401  (L: the library fixture)

FAKE = 0x1000


def _fp4(ratio=4, **kw):
    c = _fake_cache(ratio=ratio)
    c.qat = lib.FP4_ROWS
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _append(L, c):
    return L.ds4a_compress_append(ctypes.byref(c), 9, 1, *([FAKE] * 9), None, None)


def test_row_bytes_match_oracle(L):
    for D in (4, 16, 64, 80, 128, 192, 336, 512, 1024, 1028):
        for rot in (0, 2, 16, 32, 64, 128, 512):
            for dt, es in ((lib.DS4A_BF16, 2), (lib.DS4A_F32, 4)):
                ok = rot < D <= 1024 and (D - rot) % 16 == 0
                want = serving.row_layout(D, rot, es)[4] if ok else 0
                assert L.ds4a_row_bytes(D, rot, dt) == want, (D, rot)
    assert L.ds4a_row_bytes(512, 64, lib.DS4A_BF16) == 384
    assert L.ds4a_row_bytes(512, 64, 2) == 0 and L.ds4a_row_bytes(0, 0, 0) == 0
    assert L.ds4a_row_bytes(512, 63, 1) == 0 and L.ds4a_row_bytes(510, 62, 1) == 0
    with pytest.raises(lib.Ds4aError):
        lib.row_bytes(512, 60, "bf16")


def test_fp4_cache_checks(L):
    assert _append(L, _fp4()) == -4                      # past the cache's checks (position)
    assert _append(L, _fp4(qat=lib.FP4_ROWS | lib.Q_ROTATED | lib.QAT_FP4_INDEX)) == -4
    assert _append(L, _fp4(ratio=0)) == -1               # no compressed rows to hold
    assert _append(L, _fp4(qat=lib.FP4_ROWS | lib.QAT_FP8_ATTN)) == -1
    assert _append(L, _fp4(qat=0x40000)) == -1
    assert _append(L, _fp4(n_rot=60)) == -2              # 452 code dims: not in sixteens
    assert _append(L, _fp4(n_rot=512)) == -2             # no code dims at all
    assert _append(L, _fp4(attn_comp_kv=FAKE + 8)) == -1  # rows are read as 16-byte vectors
    assert _append(L, _fp4(comp_cap=(1 << 32) - 1)) == -2   # rows are numbered in 32 bits
    assert _append(L, _fp4(block_table=FAKE, max_blocks=1, comp_cap=64, n_blocks=1 << 26)) == -2
    assert _append(L, _fp4(block_table=FAKE, max_blocks=1, comp_cap=64, n_blocks=1 << 25)) == -4
    ok = _fp4(qat=lib.Q_ROTATED)
    assert _append(L, ok) == -4


def test_rows_calls_check_arguments(L):
    c = _fp4()
    r = ctypes.byref(c)
    for fn in (L.ds4a_pack_rows, L.ds4a_unpack_rows):
        assert fn(r, 0, None, None, None) == 0           # nothing to do
        assert fn(r, 3, None, FAKE, None) == -1
        assert fn(r, 3, FAKE + 1, FAKE, None) == -1
        assert fn(r, c.batch * c.comp_cap + 1, FAKE, None, None) == -3
        assert fn(r, 1 << 31, FAKE, FAKE, None) == -2
        assert fn(None, 3, FAKE, FAKE, None) == -1
        plain = _fake_cache()
        assert fn(ctypes.byref(plain), 3, FAKE, FAKE, None) == -1


def test_norm_rope_checks_arguments(L):
    c = _fake_cache()
    H, D = 64, c.head_dim
    ok = dict(n=4, pos=FAKE, q=FAKE, qs=H * D, H=H, gq=None, qo=2 * FAKE, kv=FAKE, kvs=D, gk=FAKE,
              kvo=4 * FAKE, slots=None, flags=1)

    def call(cache=c, **kw):
        a = {**ok, **kw}
        return L.ds4a_norm_rope(None if cache is None else ctypes.byref(cache), a["n"], a["pos"],
                                a["q"], a["qs"], a["H"], a["gq"], a["qo"], a["kv"], a["kvs"],
                                a["gk"], a["kvo"], a["slots"], a["flags"], None)

    assert call(n=0) == 0                                # nothing to do, after every check
    assert call(cache=None) == -1
    assert call(n=0, flags=2) == -1
    assert call(n=0, q=None, kv=None) == -1
    assert call(n=0, pos=None) == -1
    assert call(n=0, H=0) == -2 and call(n=0, H=129, qs=129 * D) == -2
    assert call(n=0, qo=None) == -1
    assert call(n=0, qs=H * D - 1) == -2 and call(n=0, kvs=D - 1) == -2
    assert call(n=0, qo=FAKE, qs=H * D + 8) == -1        # in place, strided
    assert call(n=0, qo=FAKE) == 0
    assert call(n=0, kvo=FAKE, kvs=D + 8) == -1
    assert call(n=0, kvo=None) == -1                     # neither kv_out nor slots
    assert call(n=0, slots=FAKE) == -1                   # both
    assert call(n=0, kvo=None, slots=FAKE) == 0
    assert call(n=0, q=FAKE + 1) == -1 and call(n=0, gk=FAKE + 1) == -1
    assert call(n=1 << 31) == -2
    assert call(n=0, q=None, H=0, qo=None, qs=0) == 0    # rows only
    assert call(n=0, kv=None, kvo=None, kvs=0) == 0      # queries only


def test_block_tables_checks_arguments(L):
    def pool(**kw):
        a = dict(rows=4, max_blocks=8, n_blocks=16, table=FAKE, held=FAKE, free_list=FAKE,
                 state=FAKE)
        return lib.BlockPoolC(**{**a, **kw})

    def call(p=None, step=None, ctx=FAKE, new=FAKE, cap=128):
        p, step = p or pool(), step or lib.StepTablesC(max_tokens=4)
        return L.ds4a_block_tables(ctypes.byref(p), ctx, new, cap, ctypes.byref(step), None)

    for name in ("table", "held", "free_list", "state"):
        assert call(pool(**{name: None})) == -1
    assert call(ctx=None) == -1 and call(new=None) == -1
    assert L.ds4a_block_tables(None, FAKE, FAKE, 128, None, None) == -1
    for kw in ({"rows": 0}, {"rows": 8193}, {"max_blocks": 0}, {"n_blocks": 0},
               {"n_blocks": (1 << 25) + 1}, {"max_blocks": (1 << 23) + 1}):
        assert call(pool(**kw)) == -2
    assert call(cap=0) == -2 and call(cap=1025) == -2
    assert call(step=lib.StepTablesC(max_tokens=1 << 31)) == -2


def test_fp4_cache_tensors_on_cpu(L):
    """The binding's 4-bit cache: bytes in place of elements, paged or not."""
    import torch
    kw = dict(head_dim=512, n_rot=64, batch=2, dtype="bf16", base=160000.0, rope_max_pos=16,
              device="cpu", qat=lib.FP4_ROWS)
    c = lib.LayerCache(ratio=128, comp_cap=6, **kw)
    assert c.attn_comp_kv.shape == (2, 6, 384) and c.attn_comp_kv.dtype == torch.uint8
    assert c.slots(3).tolist() == [[0, 1, 2], [6, 7, 8]]
    table = torch.tensor([[4, 1, 0], [2, 5, 3]], dtype=torch.int32)
    c = lib.LayerCache(ratio=128, comp_cap=6, block_table=table, n_blocks=7, **kw)
    assert c.attn_comp_kv.shape == (7, 2, 384)
    assert c.slots(5).tolist() == [[8, 9, 2, 3, 0], [4, 5, 10, 11, 6]]


def test_bindings_check_tensors(L):
    """Tensors of another type or size than the call reads are refused before it."""
    import torch
    kw = dict(head_dim=512, n_rot=64, batch=2, dtype="bf16", base=160000.0, rope_max_pos=16,
              device="cpu", qat=lib.FP4_ROWS)
    c = lib.LayerCache(ratio=128, comp_cap=6, **kw)
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    rows = torch.zeros((3, 512), **bf)
    for fn in (lib.ds4a_pack_rows, lib.ds4a_unpack_rows):
        for bad in ((rows.float(), None), (rows[:, :256].contiguous(), None),
                    (rows, torch.zeros(3, dtype=torch.int64)), (rows, torch.zeros(2, **i32))):
            with pytest.raises(AssertionError):
                fn(c, *bad, stream=0)
        fn(c, rows[:0], stream=0)                       # nothing to do
    pos, q, kv = torch.zeros(3, **i32), torch.zeros((3, 4, 512), **bf), torch.zeros((3, 512), **bf)
    ok = dict(q=q, q_out=torch.empty_like(q), kv=kv, kv_out=torch.empty_like(kv), stream=0)
    for bad in (dict(q=q.float()), dict(q_out=q[:2]), dict(kv=kv[:2]), dict(kv_out=kv[:2]),
                dict(gamma_q=q[0, 0].float()), dict(gamma_kv=kv[0, :8]), dict(q=q[:, :, ::2]),
                dict(kv_out=None, slots=pos.long()), dict(kv_out=None, slots=pos[:2]),
                dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(AssertionError):
            lib.ds4a_norm_rope(c, pos, **{**ok, **bad})
    with pytest.raises(AssertionError):
        lib.ds4a_norm_rope(c, pos.long(), **ok)
    lib.ds4a_norm_rope(c, pos[:0], q=q[:0], q_out=q[:0], kv=kv[:0], kv_out=kv[:0], stream=0)
    pool, step = lib.BlockPool(2, 4, 8, device="cpu"), lib.StepTables(2, 16, device="cpu")
    for ctx, new in ((torch.zeros(2, **i32), torch.zeros(3, **i32)),
                     (torch.zeros(2, dtype=torch.int64), torch.zeros(2, **i32))):
        with pytest.raises(AssertionError):
            lib.ds4a_block_tables(pool, ctx, new, 128, step, stream=0)
