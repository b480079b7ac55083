"""The operators around a paged, 4-bit cache — TEST INFRASTRUCTURE, part of the
CPU oracle: block tables and slot maps from request lengths, norms of query heads
and K = V rows with the tail rotation, compressed rows held in 4 bits.

vLLM's DeepSeek V4 page gives logical blocks of 256 token positions and names
the fused query norm, KV rotation and insert ("GPU 計算飽和"); neither page gives
formulas or a packed row format. Readings:

* S1 a row of a step's batch that is to hold n tokens holds ceil(n / 256) blocks.
  Blocks are taken from the head of a ring of free blocks, row by row in order, and
  blocks given back go to its tail once every row has taken its own.
* S2 norm: x / sqrt(mean(x^2) + 1e-6) * gamma, then the rotation, in fp64, rounded
  once. The epsilon is the compressor's.
* S3 a 4-bit row: E2M1 codes with a scale 2^k per 16 dims (smallest k >= -127 with
  amax <= 6 * 2^k, as the FP4 round trip has it per 32); the rotated dims keep
  the storage type. Written here dim by dim, from the byte order that ds4a.h states.
"""
import numpy as np

from .numerics import round_store
from .qat import E2M1_MAX, block_scale_exp, e2m1_table, round_to_table
from .rope import rope_tail

BLOCK = 256
SIGN = (15, 12, 14, 13)
MAG = (6, 3, 0, 9)


# ------------------------------------------------------------ 4-bit rows

def row_layout(D: int, n_rot: int, elem_bytes: int):
    """(nb, ns, R, tail offset, row bytes)."""
    nb = -(-(D - n_rot) // 64)
    ns = -(-nb // 8)
    R = -(-(nb + ns) // 4) * 4
    tail = 32 * R
    return nb, ns, R, tail, -(-(tail + n_rot * elem_bytes) // 32) * 32


def _word_at(w, j):
    return 128 * (w // 4) + 16 * j + 4 * (w % 4)


def dim_place(D: int, n_rot: int, d: int, elem_bytes: int):
    """(byte of the half-word, pair index, byte of the scale) of code dim d."""
    nb, ns, _, _, _ = row_layout(D, n_rot, elem_bytes)
    kb, j, i = d // 64, (d % 64) // 8, d % 8
    q, per = (d % 64) // 16, 4 * ns
    scale = _word_at(nb + (kb % per) // 4, 2 * q + kb // per) + kb % 4
    return _word_at(kb, j) + 2 * (i % 2), i // 2, scale


def quantise_row(x, n_rot: int, dtype: str) -> np.ndarray:
    """The values that a 4-bit row stands for (fp64)."""
    x = np.asarray(x, np.float64)
    nope = x.shape[-1] - n_rot
    out = x.copy()
    for b0 in range(0, nope, 16):
        seg = x[..., b0:b0 + 16].reshape(-1, 16)
        res = np.empty_like(seg)
        for r in range(seg.shape[0]):
            if not np.isfinite(seg[r]).all():
                res[r] = np.nan
                continue
            k = block_scale_exp(np.abs(seg[r]).max(), E2M1_MAX)
            v = round_to_table(seg[r] * 2.0 ** -k, e2m1_table())
            if k == 126:
                v = np.clip(v, -3.0, 3.0)
            res[r] = v * 2.0 ** k
        out[..., b0:b0 + 16] = res.reshape(x[..., b0:b0 + 16].shape)
    out[..., nope:] = round_store(x[..., nope:], dtype)
    return out


def read_row(row: np.ndarray, D: int, n_rot: int, dtype: str) -> np.ndarray:
    """Values of one packed row (uint8 bytes), dim by dim."""
    es = 2 if dtype == "bf16" else 4
    _, _, _, tail, _ = row_layout(D, n_rot, es)
    vals, _ = e2m1_table()
    out = np.empty(D, np.float64)
    for d in range(D - n_rot):
        at, t, sc = dim_place(D, n_rot, d, es)
        half = int(row[at]) | int(row[at + 1]) << 8
        sb = int(row[sc])
        v = vals[half >> MAG[t] & 7] * 2.0 ** (sb - 127)
        out[d] = np.nan if sb == 255 else (-v if half >> SIGN[t] & 1 else v)
    raw = np.ascontiguousarray(row[tail:tail + n_rot * es])
    if dtype == "bf16":
        out[D - n_rot:] = (raw.view(np.uint16).astype(np.uint32) << 16).view(np.float32)
    else:
        out[D - n_rot:] = raw.view(np.float32)
    return out


# ----------------------------------------------------------------- norms

def norm_rope(x, gamma, pos, base: float, n_rot: int, rotate: bool) -> np.ndarray:
    """x [n][..., D] normalised over D and (rotate) turned at pos [n]; fp64."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    if not rotate:
        return y
    p = np.asarray(pos).reshape((-1,) + (1,) * (x.ndim - 2))
    return rope_tail(y, p, base, n_rot)


# --------------------------------------------- block tables and slot maps

def block_tables(pool, ctx, new, cap_raw: int, max_tokens: int):
    """pool: dict of table [B][M], held [B], free_list [n], state [4] (numpy), updated in
    place. Returns the step's arrays."""
    table, held, free, state = pool["table"], pool["held"], pool["free_list"], pool["state"]
    B, M = table.shape
    n = len(free)
    head, count, short = int(state[0]), int(state[1]), 0
    tail = (head + count) % n
    room, back = n - count, []
    for b in range(B):
        want = -(-int(ctx[b]) // BLOCK)
        need = min(want, M)
        short += want - need
        had = int(held[b])
        for j in range(had, need):
            if count:
                table[b, j] = free[head]
                head, count = (head + 1) % n, count - 1
                held[b] = j + 1
            else:
                table[b, j] = -1
                short += 1
        for j in range(need, had):
            back.append(int(table[b, j]))
            table[b, j] = -1
        if had > need:
            held[b] = need
    for blk in back[:room]:
        free[tail] = blk
        tail, count = (tail + 1) % n, count + 1
    state[:3] = (head, count, short)
    toks, cu = [], [0]
    for b in range(B):
        nw = min(int(new[b]), int(ctx[b]))
        for p in range(int(ctx[b]) - nw, int(ctx[b])):
            j = p // BLOCK
            blk = int(table[b, j]) if j < M else -1
            ok = 0 <= blk < n
            toks.append((b, p, b * cap_raw + p % cap_raw if p + cap_raw >= int(ctx[b]) else -1,
                         blk * 64 + p % BLOCK // 4 if ok and p % 4 == 3 else -1,
                         blk * 2 + p % BLOCK // 128 if ok and p % 128 == 127 else -1))
        cu.append(len(toks))
    toks = (toks + [(-1,) * 5] * max_tokens)[:max_tokens]
    cols = np.array(toks, np.int64).reshape(max_tokens, 5).T
    first = np.array([int(c) - min(int(w), int(c)) for c, w in zip(ctx, new)])
    return {"seq_pos": first, "cu_len": np.array(cu), "tok_seq": cols[0], "tok_pos": cols[1],
            "raw_slot": cols[2], "comp_slot4": cols[3], "comp_slot128": cols[4]}
