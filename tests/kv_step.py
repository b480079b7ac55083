"""Shared plumbing of the tests around a paged cache of keys and values: a step's sequences,
blocks and packed tokens on the host, and the cache on the GPU."""
import numpy as np
import torch

from helpers import np_
from oracle import kv

TD = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BLOCK = 256


def rand(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def bits(t):
    """8-bit floats as bytes (indexing and comparing them does not work everywhere)."""
    return t.view(torch.uint8) if t.dtype is torch.float8_e4m3fn else t


def table_for(g, lens, spare=2, hole=None):
    """Random distinct blocks for sequences of these lengths; hole: (b, j) entries left out."""
    held = [-(-int(n) // BLOCK) for n in lens]
    nb = sum(held) + spare
    perm = torch.randperm(nb, generator=g).int().numpy()
    table = np.full((len(lens), max(max(held), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = perm[at:at + n]
        at += n
    for b, j in hole or ():
        table[b, j] = -1
    return table, nb


def values_of(pool, scale, kv_dtype):
    """fp64 values of a pool [n][K][256][D] on the host."""
    if kv_dtype != "e4m3":
        return np_(pool).astype(np.float64)
    v = kv.e4m3_table()[bits(pool).cpu().numpy()]
    return v * np_(scale).astype(np.float64)[None, :, None, None]


class Step:
    """Sequences that hold `old` tokens and get `new` ones; pools of random rows where some token of
    the step may look, NaN everywhere else."""

    def __init__(self, lib, seed, old, new, H, K, D, dtype="bf16", kv_dtype=None, window=0, hole=None, std=1.0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)
        kv_dtype = kv_dtype or dtype
        self.old, self.new, self.H, self.K, self.D = np.array(old), np.array(new), H, K, D
        self.dtype, self.kv_dtype, self.window = dtype, kv_dtype, window
        B = len(old)
        self.cu = np.concatenate([[0], np.cumsum(self.new)])
        self.n = int(self.cu[-1])
        self.table, self.nb = table_for(g, self.old + self.new, hole=hole)
        self.k_scale, self.v_scale = torch.rand(K, generator=g) * 0.02 + 0.01, torch.rand(K, generator=g) * 0.02 + 0.01
        shape = (self.nb, K, BLOCK, D)

        def pool(scale):
            x = torch.randn(shape, generator=g) * std
            if kv_dtype == "e4m3":
                x = (x / scale[None, :, None, None]).clamp(-448, 448)
            return x.to(TD[kv_dtype])

        self.pk, self.pv = pool(self.k_scale), pool(self.v_scale)
        seen = np.zeros((self.nb, BLOCK), bool)
        for b in range(B):
            lo = max(0, self.old[b] + 1 - window) if window else 0
            for p in range(lo, self.old[b] + self.new[b]):
                blk = self.table[b, p // BLOCK]
                if blk >= 0:
                    seen[blk, p % BLOCK] = True
        at = torch.from_numpy(~seen)[:, None, :, None].expand(shape)
        nan = 0x7F if kv_dtype == "e4m3" else float("nan")
        bits(self.pk)[at], bits(self.pv)[at] = nan, nan
        self.q = rand(g, self.n, H, D, dtype=TD[dtype], std=1.5)
        self.lib, self.device = lib, device

    def on_gpu(self, seq_pos=None):
        lib, dev = self.lib, self.device
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)  # noqa: E731
        f8 = self.kv_dtype == "e4m3"
        c = lib.KvCache(head_dim=self.D, n_kv_heads=self.K, batch=len(self.old), block_table=i32(self.table),
                        n_blocks=self.nb, dtype=self.dtype, kv_dtype=self.kv_dtype, k=self.pk.to(dev), v=self.pv.to(dev),
                        k_scale=self.k_scale.to(dev) if f8 else None, v_scale=self.v_scale.to(dev) if f8 else None,
                        device=dev)
        c.set_seq_pos(i32(self.old if seq_pos is None else seq_pos))
        return c, i32(self.cu)

    def oracle(self, scale, max_new=None):
        return kv.attention(np_(self.q), values_of(self.pk, self.k_scale, self.kv_dtype),
                            values_of(self.pv, self.v_scale, self.kv_dtype), self.table, self.old, self.cu, scale,
                            self.window, max_new)

    def tolerance(self, want, mag, flat, scale):
        """Elementwise bound of the output and of lse, from the arithmetic.

        A score is a sum of D products: (D + 4) steps of 2^-23 of the sum of their magnitudes (at
        most |q| |k|, Cauchy). A weight's relative error is twice the largest score's (its own and the
        sum's), plus 2^-21 for the exponential; sums over n keys add n 2^-23. bf16 weights are held
        in two parts (2^-17). Over an 8-bit cache queries too are two 8-bit parts: off by 2^-18 of
        the row's largest, over D dims; weights by 2^-8 relative or 2^-14 of the largest."""
        q = np.abs(np_(self.q)).astype(np.float64)
        k = values_of(self.pk, self.k_scale, self.kv_dtype)
        kn = np.sqrt(np.nansum(k * k, -1).max())
        n = int((self.old + self.new).max())
        ds = (self.D + 4) * 2.0 ** -23 * (np.sqrt((q * q).sum(-1)) * kn).max() * abs(scale)
        w = 2.0 ** -17
        if self.kv_dtype == "e4m3":
            ds += q.max() * 2.0 ** -18 * np.sqrt(self.D) * kn * abs(scale)
            w = 2.0 ** -8
        rel = 2 * ds + 2.0 ** -21 + w + n * 2.0 ** -23
        tol = rel * mag + torch.finfo(TD[self.dtype]).eps / 2 * np.abs(want) + 1e-30
        if self.kv_dtype == "e4m3":
            tol = tol + 2.0 ** -14 * flat
        return tol, 2 * ds + 2.0 ** -21 + n * 2.0 ** -23 + 2.0 ** -20


def check(step, out, lse, scale, max_new=None):
    want, wl, mag, flat = step.oracle(scale, max_new)
    tol, tl = step.tolerance(want, mag, flat, scale)
    live = ~np.isnan(wl[:, 0])
    err = np.abs(np_(out).astype(np.float64)[live] - want[live])
    assert np.isfinite(err).all()
    assert (err <= tol[live]).all(), float((err / tol[live]).max())
    got = np_(lse).astype(np.float64)[live]
    empty = np.isneginf(wl[live])
    assert (np.isneginf(got) == empty).all()
    d = np.abs(got[~empty] - wl[live][~empty])
    assert (d <= tl + 2.0 ** -22 * np.abs(got[~empty])).all(), float(d.max())
