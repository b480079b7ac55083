"""What the calls refuse or accept on the host, by the returned status only (nothing is
launched: every case ends at a check)."""
import ctypes

from compressed_kv_sparse_gb300 import lib
from test_abi_cpu import L, _fake_cache  # noqa: F401  (L: the library fixture)

FAKE = 0x1000


def cache(**kw):
    c = _fake_cache()
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def append(L, c):
    return L.ds4a_compress_append(ctypes.byref(c), 9, 1, *([FAKE] * 9), None, None)


def test_the_flag_for_ready_queries(L):
    assert append(L, cache(qat=lib.Q_READY)) == -4       # past the cache's checks (position)
    assert append(L, cache(qat=lib.Q_READY | lib.Q_ROTATED | lib.FP4_ROWS)) == -4
    assert append(L, cache(qat=lib.Q_READY << 1)) == -1


BIG = 1 << 40


def decode(L, c, q=FAKE, topk=FAKE, out=FAKE, ws=FAKE, nbytes=BIG, heads=64):
    return L.ds4a_sparse_attn_decode(ctypes.byref(c), c.n_tokens - 1, q, heads, topk, 512, 0.1, out, ws,
                                     nbytes, None)


def chunk(L, c, q=FAKE, rows=FAKE, topk=FAKE, out=FAKE, ws=FAKE, nbytes=BIG, heads=64):
    return L.ds4a_sparse_attn_prefill_chunk(ctypes.byref(c), c.n_tokens - 2, 2, q, heads, rows, topk, 512,
                                            0.1, out, ws, nbytes, None)


def test_attention_on_the_tensor_cores_wants_16_bytes(L):
    """Rows, queries, output and workspace of the kernels that copy 16 bytes at a time."""
    for qat, heads in ((0, 64), (lib.FP4_ROWS, 64), (lib.FP4_ROWS, 5)):
        kw = dict(qat=qat)
        for call in (decode, chunk):
            assert call(L, cache(**kw), nbytes=8, heads=heads) == -8     # past the checks
            for off in (2, 4, 8):
                for name in ("q", "out", "ws"):
                    assert call(L, cache(**kw), heads=heads, **{name: FAKE + off}) == -1, (name, off)
                for name in ("raw_kv", "attn_comp_kv"):
                    assert call(L, cache(**{name: FAKE + off}, **kw), heads=heads) == -1, (name, off)
                assert chunk(L, cache(**kw), rows=FAKE + off, heads=heads) == -1
            assert call(L, cache(**kw), topk=FAKE + 2, heads=heads) == -1
            assert call(L, cache(seq_pos=FAKE + 2, **kw), heads=heads) == -1


def test_attention_on_the_cuda_cores_wants_whole_elements(L):
    for kw, es, heads in ((dict(dtype=lib.DS4A_F32), 4, 64), (dict(), 2, 8), (dict(head_dim=128), 2, 64)):
        for call in (decode, chunk):
            for name in ("q", "out"):
                assert call(L, cache(**kw), nbytes=8, heads=heads, **{name: FAKE + es}) == -8
                assert call(L, cache(**kw), heads=heads, **{name: FAKE + es // 2}) == -1
            for name in ("raw_kv", "attn_comp_kv"):
                assert call(L, cache(**{name: FAKE + es}, **kw), nbytes=8, heads=heads) == -8
                assert call(L, cache(**{name: FAKE + es // 2}, **kw), heads=heads) == -1
            assert call(L, cache(**kw), ws=FAKE + 8, heads=heads) == -1
    # a row of the window that ds4a_norm_rope may write need not suit the attention
    assert L.ds4a_norm_rope(ctypes.byref(cache(raw_kv=FAKE + 2)), 0, FAKE, None, 0, 0, None, None, FAKE,
                            512, None, None, FAKE, 0, None) == 0
    assert decode(L, cache(raw_kv=FAKE + 2)) == -1


def test_other_calls_check_alignment(L):
    def topk(c, q=FAKE, w=FAKE, out=FAKE, ws=FAKE, nbytes=BIG, heads=64):
        return L.ds4a_index_topk(ctypes.byref(c), 9, 1, q, w, heads, 512, out, ws, nbytes, None)

    assert topk(cache(), q=FAKE + 2, w=FAKE + 2, nbytes=8) == -8         # (any element's place will do)
    assert topk(cache(), q=FAKE + 1) == -1 and topk(cache(), w=FAKE + 1) == -1
    assert topk(cache(), out=FAKE + 2) == -1 and topk(cache(), ws=FAKE + 8) == -1
    assert topk(cache(index_comp_kv=FAKE + 8)) == -1
    assert topk(cache(index_comp_kv=FAKE + 2), heads=8, nbytes=8) == -8
    assert topk(cache(index_comp_kv=FAKE + 1), heads=8) == -1
    assert topk(cache(dtype=lib.DS4A_F32), q=FAKE + 2) == -1

    def app(c, **kw):
        args = [kw.get(f"a{i}", FAKE) for i in range(9)]
        return L.ds4a_compress_append(ctypes.byref(c), 10, 1, *args, None, None)

    for i in range(9):
        assert app(cache(), **{f"a{i}": FAKE + 1}) == -1, i
    assert app(cache(attn_state_kv=FAKE + 4)) == -1 and app(cache(attn_state_score=FAKE + 4)) == -1
    assert app(cache(raw_kv=FAKE + 1)) == -1

    fp4 = cache(qat=lib.FP4_ROWS)
    for fn in (L.ds4a_pack_rows, L.ds4a_unpack_rows):
        assert fn(ctypes.byref(fp4), 3, FAKE, FAKE + 2, None) == -1
        assert fn(ctypes.byref(fp4), 3, FAKE + 1, FAKE, None) == -1

    def norm(**kw):
        a = dict(pos=FAKE, q=FAKE, gq=FAKE, qo=2 * FAKE, kv=FAKE, gk=FAKE, kvo=None, slots=FAKE)
        a.update(kw)
        return L.ds4a_norm_rope(ctypes.byref(cache()), 0, a["pos"], a["q"], 64 * 512, 64, a["gq"], a["qo"],
                                a["kv"], 512, a["gk"], a["kvo"], a["slots"], 0, None)

    assert norm() == 0                                   # (no tokens: nothing to do)
    assert norm(pos=FAKE + 2) == -1 and norm(slots=FAKE + 2) == -1
    for name in ("q", "gq", "qo", "kv", "gk"):
        assert norm(**{name: FAKE + 1}) == -1, name
        assert norm(**{name: FAKE + 2}) == 0, name
    assert norm(kvo=FAKE + 1, slots=None) == -1

    def tables(ctx=FAKE, new=FAKE, pool=(), step=()):
        p = lib.BlockPoolC(**{**dict(rows=4, max_blocks=8, n_blocks=16, table=FAKE, held=FAKE,
                                     free_list=FAKE, state=FAKE), **dict(pool)})
        s = lib.StepTablesC(**{**dict(max_tokens=4), **dict(step)})
        return L.ds4a_block_tables(ctypes.byref(p), ctx, new, 0, ctypes.byref(s), None)

    assert tables() == -2                                # past the pointers (no window)
    assert tables(ctx=FAKE + 2) == -1 and tables(new=FAKE + 1) == -1
    for name in ("table", "held", "free_list", "state"):
        assert tables(pool={name: FAKE + 2}) == -1, name
    for name in ("seq_pos", "cu_len", "tok_seq", "tok_pos", "raw_slot", "comp_slot4", "comp_slot128"):
        assert tables(step={name: FAKE + 2}) == -1, name


SIZES = """
import ctypes, sys
sys.path[:0] = ['.', 'tests']
from compressed_kv_sparse_gb300 import lib
from test_abi_cpu import _fake_cache
L = lib.load()
calls = (lib.CALL_INDEX_TOPK, lib.CALL_ATTN_DECODE, lib.CALL_ATTN_PREFILL)


def ask(c, T=3, H=64, k=512):
    return [L.ds4a_workspace_bytes(w, ctypes.byref(c), T, H, k) for w in calls]


for qat in (0, lib.FP4_ROWS):
    for dtype in (0, 1):
        for ratio in (4, 128):
            def cache(**kw):
                c = _fake_cache(ratio=ratio, dtype=dtype)
                c.qat = qat
                for n, v in kw.items():
                    setattr(c, n, v)
                return c
            assert all(ask(cache())), (qat, dtype, ratio)
            assert ask(cache(raw_kv=None, attn_comp_kv=None, rope_cos=None)) == ask(cache())
            for kw in (dict(T=0), dict(H=0), dict(H=129)):
                assert ask(cache(), **kw) == [0, 0, 0], kw
            for kw in (dict(head_dim=0), dict(head_dim=2000), dict(head_dim=6), dict(batch=0), dict(dtype=9),
                       dict(cap_raw=0), dict(comp_cap=0), dict(ratio=7)):
                assert ask(cache(**kw)) == [0, 0, 0], kw
print('sizes done')
"""


def test_workspace_bytes_of_sizes_that_no_call_takes(L):
    """In a process of its own, which a division by zero would end."""
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", SIZES], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "sizes done" in r.stdout, (r.returncode, r.stderr[-2000:])


def test_a_count_of_tokens_that_the_cache_has_no_room_for(L):
    """n_tokens set by the caller (ds4a_norm_rope and the append by lanes leave it to them)."""
    def topk(c, nbytes=8):
        return L.ds4a_index_topk(ctypes.byref(c), c.n_tokens - 1, 1, FAKE, FAKE, 64, 512, FAKE, FAKE, nbytes,
                                 None)

    small = lambda call: (lambda c: call(c) if call is topk else call(L, c, nbytes=8))  # noqa: E731
    for call in map(small, (decode, chunk, topk)):
        full = cache(n_tokens=64 + 3)                    # 16 rows of 4 tokens, and some
        assert call(full) == -8                          # past the checks: too small a workspace
        assert call(cache(n_tokens=64 + 4)) == -3        # a row more than comp_cap
        assert call(cache(n_tokens=60, rope_max_pos=60)) == -8
        assert call(cache(n_tokens=60, rope_max_pos=59)) == -3
    for call in map(small, (decode, chunk)):
        assert call(cache(ratio=128, n_tokens=17 * 128, rope_max_pos=1 << 20)) == -3
        assert call(cache(ratio=128, n_tokens=17 * 128 - 1, rope_max_pos=1 << 20)) == -8
    for call in (decode, chunk):                         # the raw window alone
        assert call(L, cache(ratio=0, n_tokens=1000), nbytes=8) == -8
        assert call(L, cache(ratio=0, n_tokens=1001), nbytes=8) == -3
    assert L.ds4a_index_norms(ctypes.byref(cache(n_tokens=64 + 4)), None) == -3


def test_every_array_of_a_cache_starts_on_an_element(L):
    for name in ("attn_state_kv", "attn_state_score", "index_state_kv", "index_state_score", "index_norm",
                 "index_norm_max", "rope_cos", "rope_sin", "index_rope_cos", "index_rope_sin", "seq_pos"):
        for off in (1, 2):
            assert L.ds4a_cache_reset(ctypes.byref(cache(**{name: FAKE + off})), None) == -1, name
    for name in ("raw_kv", "attn_comp_kv", "index_comp_kv"):
        assert append(L, cache(**{name: FAKE + 2})) == -4, name          # (bf16: past the cache's checks)
        assert append(L, cache(**{name: FAKE + 1})) == -1, name
        assert append(L, cache(dtype=lib.DS4A_F32, **{name: FAKE + 2})) == -1, name
    # arrays that a layer does not have are not looked at
    assert append(L, cache(ratio=128, index_comp_kv=FAKE + 1, index_norm=FAKE + 1)) == -4
