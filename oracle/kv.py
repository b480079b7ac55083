"""The operators around a paged cache of keys and values — TEST INFRASTRUCTURE, part of the CPU
oracle: rotary positions, the append, attention of a step's new tokens, verification of drafts.
fp64 (whole numbers exactly), written from the formulas that ds4a.h states.
"""
from fractions import Fraction

import numpy as np

BLOCK = 256


# -------------------------------------------------------------- rotation

def theta(n_rot, base, kind="none", factor=1.0, orig_len=0.0, beta_fast=32.0, beta_slow=1.0, magnitude=0.0):
    """(angle per position of each pair, factor of cosines and sines)."""
    i = np.arange(n_rot // 2, dtype=np.float64)
    if kind == "ntk":
        base = base * factor ** (n_rot / (n_rot - 2))
    th = base ** (-2 * i / n_rot)
    if kind == "linear":
        return th / factor, 1.0
    if kind != "yarn":
        return th, 1.0
    # pair i turns orig_len * th[i] / (2 pi) times over the trained positions
    at = lambda turns: n_rot / 2 * np.log(orig_len / (2 * np.pi * turns)) / np.log(base)  # noqa: E731
    low, high = max(np.floor(at(beta_fast)), 0), min(np.ceil(at(beta_slow)), n_rot - 1)
    keep = 1 - np.clip((i - low) / max(high - low, 0.001), 0, 1)
    return keep * th + (1 - keep) * th / factor, magnitude or 0.1 * np.log(factor) + 1


def rotate(x, pos, n_rot, base, rot_at=0, half=False, inverse=False, **scaling):
    """x [n][H][D] turned at pos [n]: each pair as a complex number."""
    x = np.array(x, np.float64)
    th, mag = theta(n_rot, base, **scaling)
    w = mag * np.exp(1j * np.asarray(pos, np.float64)[:, None] * th * (-1 if inverse else 1))[:, None]
    r = x[..., rot_at:rot_at + n_rot]
    a, b = (slice(0, n_rot // 2), slice(n_rot // 2, None)) if half else (slice(0, None, 2), slice(1, None, 2))
    z = (r[..., a] + 1j * r[..., b]) * w
    out = r.copy()
    out[..., a], out[..., b] = z.real, z.imag
    x[..., rot_at:rot_at + n_rot] = out
    return x


# ------------------------------------------------------- 8-bit floats, append

def e4m3_table():
    """Value of each of the 256 codes."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def to_e4m3(x):
    """Nearest value, ties to the even code, held to 448."""
    t = e4m3_table()[:127]
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), 448.0)
    bad = np.isnan(x)
    mag = np.where(bad, 0.0, mag)
    hi = np.clip(np.searchsorted(t, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - t[lo], t[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    v = t[code]
    return np.where(bad, np.nan, np.where(np.signbit(x), -v, v))


def append(pool_k, pool_v, table, seq, pos, k, v):
    """k, v [n][K][D] (as they are to be held) into pools [n_blocks][K][256][D] in place."""
    B, M = table.shape
    for i in range(len(seq)):
        s, p = int(seq[i]), int(pos[i])
        if not (0 <= s < B and 0 <= p < M * BLOCK):
            continue
        blk = int(table[s, p // BLOCK])
        if 0 <= blk < len(pool_k):
            pool_k[blk, :, p % BLOCK] = k[i]
            pool_v[blk, :, p % BLOCK] = v[i]


# ------------------------------------------------------------------ attention

def keys_of(table, b, p, window, n_blocks):
    """Positions that the token at p of sequence b sees, and their (block, row)."""
    lo = max(0, p - window + 1) if window else 0
    out = []
    for j in range(lo // BLOCK, min(p // BLOCK + 1, table.shape[1])):
        blk = int(table[b, j])
        if 0 <= blk < n_blocks:
            r0, r1 = max(lo - j * BLOCK, 0), min(p - j * BLOCK, BLOCK - 1) + 1
            out.append((blk, r0, r1))
    return out


def attention(q, pool_k, pool_v, table, seq_pos, cu, scale, window=0, max_new=None):
    """out [n][H][D], lse [n][H], and for tolerances the sums over the keys of weight * |value| and of
    |value| / (sum of weights relative to the largest); rows of tokens beyond max_new are NaN."""
    n, H, D = q.shape
    nb, K = pool_k.shape[:2]
    G = H // K
    out, mag, flat = (np.full((n, H, D), np.nan) for _ in range(3))
    lse = np.full((n, H), np.nan)
    for b in range(len(seq_pos)):
        for t in range(int(cu[b + 1]) - int(cu[b])):
            if max_new is not None and t >= max_new:
                break
            i = int(cu[b]) + t
            parts = keys_of(table, b, int(seq_pos[b]) + t, window, nb)
            if not parts:
                out[i], mag[i], flat[i], lse[i] = 0, 0, 0, -np.inf
                continue
            k = np.concatenate([pool_k[blk, :, r0:r1] for blk, r0, r1 in parts], 1)   # [K][n][D]
            v = np.concatenate([pool_v[blk, :, r0:r1] for blk, r0, r1 in parts], 1)
            s = np.einsum("kgd,knd->kgn", np.asarray(q[i], np.float64).reshape(K, G, D), k) * scale
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(-1, keepdims=True)
            out[i] = np.einsum("kgn,knd->kgd", e / z, v).reshape(H, D)
            mag[i] = np.einsum("kgn,knd->kgd", e / z, np.abs(v)).reshape(H, D)
            flat[i] = (np.abs(v).sum(1)[:, None] / z).reshape(H, D)
            lse[i] = (m + np.log(z))[..., 0].reshape(H)
    return out, lse, mag, flat


# ------------------------------------------------------------ verification

def _whole(p, shift):
    """Probabilities in units of 2^-shift (Python integers)."""
    out = []
    for x in np.asarray(p, np.float64):
        x = min(max(float(x), 0.0), 1.0) if x == x else 0.0
        f = Fraction(x) * (1 << shift)
        n, r = divmod(f.numerator, f.denominator)
        out.append(n + (2 * r > f.denominator or (2 * r == f.denominator and n & 1)))
    return out


def verify(target, drafts, draft_probs, u_accept, u_sample, cnt):
    """One sequence: target [cnt][V], drafts [N], draft_probs [N][V] or None, u_accept [N]. Returns the
    tokens it emits."""
    V = target.shape[1]
    shift = min(45, 62 - max(0, (V - 1).bit_length()))
    m = min(cnt - 1, len(drafts))
    a = 0
    while a < m:
        x = int(drafts[a])
        if not 0 <= x < V:
            break
        p, q = float(target[a, x]), 1.0 if draft_probs is None else float(draft_probs[a, x])
        if not (np.isfinite(q) and (p == np.inf or (np.isfinite(p) and Fraction(float(u_accept[a])) * Fraction(q) < Fraction(p)))):
            break
        a += 1
    P = _whole(target[a], shift)
    w = list(P)
    if a < m:
        if draft_probs is None:
            if 0 <= int(drafts[a]) < V:
                w[int(drafts[a])] = 0
        else:
            w = [max(x - y, 0) for x, y in zip(P, _whole(draft_probs[a], shift))]
        if sum(w) == 0:
            w = P
    total, run, tok = sum(w), 0, V - 1
    thr = Fraction(float(u_sample)) * total
    for i, x in enumerate(w):
        run += x
        if run > thr:
            tok = i
            break
    return [int(x) for x in drafts[:a]] + [tok]
