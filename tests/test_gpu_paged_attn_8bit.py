"""Weights over an 8-bit cache (tensor cores): long tails of small ones behind a key that holds most of
the weight, and levels that fall and rise from tile to tile, against oracle/kv.py."""
import numpy as np
import pytest
import torch

from helpers import np_
from kv_step import BLOCK, bits
from oracle import kv
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV, TILE, LN2 = "cuda", 128, np.log(2.0)
K_SCALE, V_SCALE = 0.03, 0.008


class Long:
    """n keys of one head and the G queries of the token at n - 1; B sequences that share the blocks."""

    def __init__(self, seed, n, G, D, B, noise, level):
        """noise, level: scores in powers of two (deviation; of each key, [n])."""
        g = torch.Generator().manual_seed(seed)
        self.n, self.G, self.D, self.B = n, G, D, B
        q = torch.randn((G, D), generator=g)
        q /= q[:, 2:].norm(dim=1, keepdim=True)
        q[:, 0], q[:, 1] = 2.0, 0.125              # the level's coarse and fine part
        self.q = q.bfloat16()
        k = torch.randn((n, D), generator=g) * (noise * LN2)
        coarse = (level * LN2 / 2.0 / K_SCALE).float().clamp(-448, 448).to(torch.float8_e4m3fn).double() * K_SCALE
        k[:, 0], k[:, 1] = coarse.float(), ((level * LN2 - 2.0 * coarse) / 0.125).float()
        v = torch.randn((n, D), generator=g) * 0.5 + 1
        v[0] = -1.0
        nb = n // BLOCK
        self.table = torch.randperm(nb, generator=g).int().numpy()[None]
        code = lambda x, s: (x / s).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
        pool = lambda x: bits(x).view(nb, 1, BLOCK, D)[np.argsort(self.table[0])].view(torch.float8_e4m3fn)  # noqa: E731
        self.pk, self.pv = pool(code(k, K_SCALE)), pool(code(v, V_SCALE))

    def run(self):
        lib = lib_()
        f = lambda x: torch.full((1,), x, device=DEV)  # noqa: E731
        c = lib.KvCache(head_dim=self.D, n_kv_heads=1, batch=self.B, n_blocks=self.pk.shape[0], kv_dtype="e4m3",
                        block_table=torch.from_numpy(self.table.repeat(self.B, 0)).to(DEV), k_scale=f(K_SCALE),
                        v_scale=f(V_SCALE), k=self.pk.to(DEV), v=self.pv.to(DEV))
        c.set_seq_pos(torch.full((self.B,), self.n - 1, dtype=torch.int32, device=DEV))
        q = self.q.to(DEV)[None].repeat(self.B, 1, 1)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        ws = lib.workspace(c.attn_workspace_bytes(self.G), DEV)
        lib.ds4a_paged_attn_decode(c, q, out, ws, lse=lse, scale=1.0)
        assert lib.ds4a_workspace_status(ws) == 0
        return np_(out).astype(np.float64), np_(lse).astype(np.float64)

    def values(self, pool, scale):
        x = kv.e4m3_table()[bits(pool).numpy()] * np.float64(np.float32(scale))
        return x[self.table[0]].transpose(1, 0, 2, 3).reshape(self.n, self.D)

    def check(self):
        """The tolerance, from the arithmetic. A weight is the sum of two 8-bit floats, hi + lo / 16: off by 2^-9 of itself, or
        by 2^-14 absolute where it is small. The reference keeps a tile's largest weight of a row at 2 or more, so that
        this is 2^-15 of it; a tile that falls below is noticed behind it (2^-15 of the tile's before); and it may stay below
        while the row's sum is 2 for each tile up to the next power of two: 2^-14 for all keys of tiles n .. 2 n - 1 is
        then 2^-9 of the sum, and no more than 2^-7 of the last one for all tiles and all that a reference is lowered on
        the way (by 7 powers of two in a share of 1,024 tiles), times the mean value of a tile. Scores: as in kv_step. The
        output is rounded once (2^-8)."""
        out, lse = self.run()
        q, k, v = np_(self.q).astype(np.float64), self.values(self.pk, K_SCALE), self.values(self.pv, V_SCALE)
        s = q @ k.T
        w = np.exp(s - s.max(1, keepdims=True))
        z = w.sum(1, keepdims=True)
        want, a = w @ v / z, np.abs(v)
        top = w.reshape(self.G, -1, TILE).max(2)
        top = top + np.concatenate([np.zeros((self.G, 1)), top[:, :-1]], 1)
        small = top @ a.reshape(-1, TILE, self.D).sum(1) / z * 2.0 ** -15 + 2.0 ** -7 * a.reshape(-1, TILE, self.D).mean(1).max()
        kn, qn = np.sqrt((k * k).sum(1)).max(), np.sqrt((q * q).sum(1)).max()
        ds = (self.D + 4) * 2.0 ** -23 * qn * kn + np.abs(q).max() * 2.0 ** -18 * np.sqrt(self.D) * kn
        rel = 2 * ds + 2.0 ** -21 + self.n * 2.0 ** -23
        tol = (rel + 2.0 ** -9) * (w @ a / z) + small + 2.0 ** -8 * np.abs(want)
        err = np.abs(out - want)
        assert np.isfinite(out).all()
        assert (err <= tol).all(), float((err / tol).max())
        wl = (s.max(1, keepdims=True) + np.log(z))[:, 0]
        assert (np.abs(lse - wl) <= rel + 2.0 ** -20 + 2.0 ** -22 * np.abs(wl)).all()


def sink(n, share, noise):
    """Key 0 holds `share` of the weight of n keys whose scores deviate by `noise` powers of two."""
    level = torch.zeros(n, dtype=torch.float64)
    level[0] = np.log2((n - 1) * share / (1 - share)) + noise * noise * LN2 / 2
    return level


@pytest.mark.parametrize("share", [0.8, 0.9, 0.95])
@pytest.mark.parametrize("noise", [0.0, 0.3, 1.0, 2.0])
@pytest.mark.parametrize("n,B", [(131072, 320), (32768, 320), (131072, 1), (32768, 7)])
def test_a_key_that_holds_most_of_the_weight(n, B, noise, share):
    """Sequences whole or nearly so in one block, and in shares of several."""
    Long(n + B, n, 8, 16, B, noise, sink(n, share, noise)).check()


@pytest.mark.parametrize("G,D,B", [(3, 64, 320), (8, 256, 40), (16, 128, 40), (16, 64, 320), (24, 64, 160), (32, 256, 20),
                                   (40, 64, 160), (64, 256, 20), (40, 48, 3)])
def test_at_every_row_count_and_width(G, D, B):
    n = 32768
    Long(G * D, n, G, D, B, 0.3, sink(n, 0.9, 0.3)).check()


def _levels(kind, n):
    t, g = torch.arange(n) // TILE, torch.Generator().manual_seed(3)
    if kind == "alternating":
        return (t % 2 * 14.0).double()
    if kind == "falling":                       # by 3 powers of two a tile, then flat far below
        return -(t.clamp(max=6) * 3.0).double()
    if kind == "rising":
        return (t.clamp(max=30) * 1.0).double()
    if kind == "random":
        return (torch.rand(n // TILE, generator=g) * 40 - 20).double()[t]
    if kind == "valleys":                       # long runs far apart
        return torch.where(t // 40 % 2 == 0, 0.0, -25.0).double()
    return torch.where(torch.arange(n) % TILE == 5, 11.0, 0.0).double()   # "peaks": one key a tile


@pytest.mark.parametrize("G,B", [(8, 320), (8, 1), (40, 160)])
@pytest.mark.parametrize("noise", [0.1, 4.0])
@pytest.mark.parametrize("kind", ["alternating", "falling", "rising", "random", "valleys", "peaks"])
def test_levels_that_fall_and_rise(kind, noise, G, B):
    n = 32768
    Long(G + B, n, G, 32, B, noise, _levels(kind, n)).check()
