"""Steps with drafts over a paged cache of keys and values, as they are served: block tables, append,
attention, verification, and the next step on what stands. Two layers (bf16, and fp32 rows in 8 bits)
share one block table; every step is compared with oracle/kv.py, then replayed as one captured graph."""
import numpy as np
import pytest
import torch

from helpers import np_
from kv_step import BLOCK, TD, bits
from oracle import kv
from test_gpu_parity import lib_
from test_gpu_rope import recipe

pytestmark = pytest.mark.gpu
DEV, BASE = "cuda", 10000.0
B, N, V, MAXB = 3, 3, 97, 4
I32 = dict(dtype=torch.int32, device=DEV)


class Layer:
    """A layer's cache on the GPU and its mirror on the host (fp64 values, NaN where nothing was written)."""

    def __init__(self, table, nb, H, K, D, dtype, kvd, half):
        lib = lib_()
        self.H, self.K, self.D, self.dtype, self.kvd, self.nb = H, K, D, dtype, kvd, nb
        f8 = kvd == "e4m3"
        g = torch.Generator().manual_seed(D)
        self.k_scale, self.v_scale = (torch.rand(K, generator=g) * 0.01 + 0.01 for _ in range(2))
        self.rope = lib.Rope(n_rot=D // 2, max_pos=MAXB * BLOCK, base=BASE, half=half, scaling="yarn", factor=4.0,
                             orig_len=256.0, device=DEV)
        self.cache = lib.KvCache(head_dim=D, n_kv_heads=K, batch=B, block_table=table, n_blocks=nb, dtype=dtype,
                                 kv_dtype=kvd, rope=self.rope, k_scale=self.k_scale.to(DEV) if f8 else None,
                                 v_scale=self.v_scale.to(DEV) if f8 else None, device=DEV)
        for p in (self.cache.k, self.cache.v):
            bits(p).fill_(0x7F if f8 else float("nan"))
        self.mk, self.mv = (np.full((nb, K, BLOCK, D), np.nan) for _ in range(2))
        rows = B * (N + 1) + 300
        self.x = torch.zeros((rows, (H + 2 * K) * D), dtype=TD[dtype], device=DEV)   # the projections' output
        self.q = torch.zeros((rows, H, D), dtype=TD[dtype], device=DEV)
        self.out = torch.zeros_like(self.q)
        self.lse = torch.zeros((rows, H), device=DEV)
        self.ws = lib.workspace(self.cache.attn_workspace_bytes(H, N + 1), DEV)
        self.pk, self.pv = self.cache.k, self.cache.v

    def run(self, step, max_new):
        lib, n, H, K, D = lib_(), step.max_tokens, self.H, self.K, self.D
        x = self.x[:n]
        self.cache.set_seq_pos(step.seq_pos)
        lib.ds4a_kv_append(self.cache, step.tok_seq, step.tok_pos, x[:, H * D:(H + K) * D].view(n, K, D),
                           x[:, (H + K) * D:].view(n, K, D), q=x[:, :H * D].view(n, H, D), q_out=self.q[:n])
        lib.ds4a_paged_attn_decode(self.cache, self.q[:n], self.out[:n], self.ws, max_new=max_new, cu_len=step.cu_len,
                                   lse=self.lse[:n])

    def held(self, x, scale):
        """Values as the cache holds them."""
        if self.kvd == "e4m3":
            s = scale.numpy()
            return kv.to_e4m3(x.astype(np.float32) * (np.float32(1) / s)[None, :, None]) * s.astype(np.float64)[None, :, None]
        return np_(torch.from_numpy(x).to(TD[self.dtype])).astype(np.float64)

    def compare(self, table, old, cnt, max_new):
        n, H, K, D = int(cnt.sum()), self.H, self.K, self.D
        seq = np.repeat(np.arange(B), cnt)
        cu = np.concatenate([[0], np.cumsum(cnt)])
        pos = old[seq] + np.arange(n) - cu[seq]
        x = self.x[:n]
        cut = lambda a, b: x[:, a * D:b * D].reshape(n, b - a, D)  # noqa: E731
        q = recipe(cut(0, H), pos, self.rope)
        q = torch.from_numpy(q).to(TD[self.dtype])
        assert torch.equal(self.q[:n].cpu(), q)
        k = self.held(recipe(cut(H, H + K), pos, self.rope), self.k_scale)
        v = self.held(np_(cut(H + K, H + 2 * K)).astype(np.float32), self.v_scale)
        kv.append(self.mk, self.mv, table, seq, pos, k, v)

        want = kv.attention(np_(q), self.mk, self.mv, table, old, cu, 1 / np.sqrt(D), 0, max_new)
        qa, kn = np.abs(np_(q)).astype(np.float64), np.sqrt(np.nansum(self.mk ** 2, -1).max())
        o, lse, mag, flat = want
        ds = (D + 4) * 2.0 ** -23 * (np.sqrt((qa * qa).sum(-1)) * kn).max() / np.sqrt(D)
        if self.kvd == "e4m3":
            ds += qa.max() * 2.0 ** -18 * kn
        rel = 2 * ds + 2.0 ** -21 + (2.0 ** -8 if self.kvd == "e4m3" else 2.0 ** -17) + 1024 * 2.0 ** -23
        tol = rel * mag + torch.finfo(TD[self.dtype]).eps / 2 * np.abs(o) + 2.0 ** -14 * flat + 1e-30
        live = ~np.isnan(lse[:, 0])
        bad = (np.abs(np_(self.out[:n]).astype(np.float64) - o)[live] > tol[live]).sum()
        assert bad == 0
        assert np.abs(np_(self.lse[:n]) - lse)[live].max() <= 2 * ds + 1024 * 2.0 ** -23 + 2.0 ** -19


def test_steps_with_drafts():
    lib = lib_()
    rng = np.random.default_rng(3)
    g = torch.Generator().manual_seed(4)
    nb = B * MAXB
    pool = lib.BlockPool(B, MAXB, nb)
    layers = [Layer(pool.table, nb, 8, 2, 64, "bf16", "bf16", True), Layer(pool.table, nb, 6, 2, 80, "f32", "e4m3", False)]
    ctx = np.array([0, 250, 510])            # (tokens that stand; the first steps fill them)
    fill, decode = lib.StepTables(B, 300), lib.StepTables(B, B * (N + 1))
    target = torch.zeros((B * (N + 1), V), device=DEV)
    probs, drafts = torch.zeros((B, N, V), device=DEV), torch.zeros((B, N), **I32)
    ua, us = torch.zeros((B, N), device=DEV), torch.zeros(B, device=DEV)
    tokens, n_out, ctx_out = torch.zeros((B, N + 1), **I32), torch.zeros(B, **I32), torch.zeros(B, **I32)
    ctx_in, new_in = torch.zeros(B, **I32), torch.zeros(B, **I32)

    def fresh():
        for la in layers:
            la.x.copy_(torch.randn(la.x.shape, generator=g))
        t = torch.softmax(torch.randn(target.shape, generator=g) * 2, -1)
        p = torch.softmax(t.view(B, N + 1, V)[:, :N].log() + torch.randn((B, N, V), generator=g) * 0.7, -1)
        target.copy_(t)
        probs.copy_(p)
        drafts.copy_(torch.multinomial(p.reshape(-1, V), 1, generator=g).view(B, N))
        ua.copy_(torch.rand((B, N), generator=g))
        us.copy_(torch.rand(B, generator=g))

    def host_table():
        return pool.table.cpu().numpy()

    # prompts, in chunks of up to 100 tokens a sequence (appended; their outputs are not looked at)
    done = np.zeros(B, np.int64)
    while (done < ctx).any():
        cnt = np.minimum(ctx - done, 100)
        fresh()
        ctx_in.copy_(torch.tensor(done + cnt))
        new_in.copy_(torch.tensor(cnt))
        lib.ds4a_block_tables(pool, ctx_in, new_in, 128, fill)
        for la in layers:
            la.run(fill, N + 1)
            la.compare(host_table(), done, cnt, N + 1)
        done += cnt

    def one_step():
        lib.ds4a_block_tables(pool, ctx_in, new_in, 128, decode)
        for la in layers:
            la.run(decode, N + 1)
        lib.ds4a_verify_drafts(target, drafts, ua, us, tokens, n_out, draft_probs=probs, cu_len=decode.cu_len,
                               seq_pos=decode.seq_pos, ctx_out=ctx_out)

    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    for i in range(8):
        cnt = np.array([1 + N, 1 + rng.integers(0, N + 1), 0 if i == 5 else 1 + N])
        fresh()
        ctx_in.copy_(torch.tensor(ctx + cnt))
        new_in.copy_(torch.tensor(cnt))
        if i < 3:
            one_step()
        else:
            torch.cuda.synchronize()
            if i == 3:
                with torch.cuda.graph(graph, stream=stream):
                    one_step()
            graph.replay()
        torch.cuda.synchronize()
        table = host_table()
        for la in layers:
            la.compare(table, ctx, cnt, N + 1)
            assert lib.ds4a_workspace_status(la.ws) == 0
        cu = np.concatenate([[0], np.cumsum(cnt)])
        for b in range(B):
            want = []
            if cnt[b]:
                want = kv.verify(np_(target)[cu[b]:cu[b + 1]], np_(drafts)[b].astype(int), np_(probs)[b], np_(ua)[b],
                                 float(us[b]), int(cnt[b]))
            assert tokens[b].tolist() == want + [-1] * (N + 1 - len(want))
            assert int(n_out[b]) == len(want) and int(ctx_out[b]) == ctx[b] + len(want)
        ctx = ctx_out.cpu().numpy().astype(np.int64)


def test_a_prefix_that_two_sequences_share():
    """Blocks in both rows of the table: each reads them; appends go to blocks of their own."""
    lib = lib_()
    K, D, H = 2, 64, 4
    table = torch.tensor([[3, 1, -1], [3, 0, -1]], **I32)
    c = lib.KvCache(head_dim=D, n_kv_heads=K, batch=2, block_table=table, n_blocks=4)
    c.k.normal_()
    c.v.normal_()
    c.set_seq_pos(torch.tensor([300, 260], **I32))
    k, v, q = (torch.randn((2, h, D), device=DEV).bfloat16() for h in (K, K, H))
    lib.ds4a_kv_append(c, torch.tensor([0, 1], **I32), torch.tensor([300, 260], **I32), k, v)
    out, lse = torch.empty_like(q), torch.empty((2, H), device=DEV)
    lib.ds4a_paged_attn_decode(c, q, out, lib.workspace(c.attn_workspace_bytes(H)), lse=lse)
    assert torch.equal(c.k[1, :, 44], k[0]) and torch.equal(c.v[0, :, 4], v[1])
    want, wl, mag, _ = kv.attention(np_(q), np_(c.k).astype(np.float64), np_(c.v).astype(np.float64), table.cpu().numpy(),
                                    [300, 260], [0, 1, 2], 1 / 8)
    # tolerance as in kv_step (scores of |q| |k| <= 100, 301 keys, weights in two bf16 parts); bf16 has 8 significant
    # bits, so its values are 2^-7 of their power of two apart and a rounding is off by up to 2^-8 of the value
    tol = (2 * 68 * 2.0 ** -23 * 100 / 8 + 2.0 ** -16) * mag + 2.0 ** -8 * np.abs(want)
    bad = (np.abs(np_(out).astype(np.float64) - want) > tol).sum()
    assert bad == 0
    assert np.abs(np_(lse) - wl).max() <= 2 * 68 * 2.0 ** -23 * 100 / 8 + 301 * 2.0 ** -23 + 2.0 ** -19
