"""ds4a_verify_drafts at every number of blocks a sequence, up to the largest vocabulary, and at thresholds next to a
running sum: whole numbers, equal to the definition in integers."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from helpers import np_
from kv_step import TD
from oracle import kv
from test_gpu_parity import lib_
from test_gpu_verify import check, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


def whole(p, shift):
    """Probabilities in units of 2^-shift (a product with a power of two is exact; ties to even)."""
    return (p.double().nan_to_num(0.0).clamp(0, 1) * 2.0 ** shift).round().long()


def definition(target, drafts, draft_probs, u_accept, u_sample):
    """kv.verify for one sequence, its sums by torch in int64 (below 2^62)."""
    V, m = target.shape[1], len(drafts)
    shift = min(45, 62 - max(0, (V - 1).bit_length()))
    a = 0
    while a < m:
        x = int(drafts[a])
        q = 1.0 if draft_probs is None else float(draft_probs[a, x])
        if not Fraction(float(u_accept[a])) * Fraction(q) < Fraction(float(target[a, x])):
            break
        a += 1
    w = P = whole(target[a], shift)
    if a < m:
        if draft_probs is None:
            w = P.clone()
            w[int(drafts[a])] = 0
        else:
            w = (P - whole(draft_probs[a], shift)).clamp(min=0)
        if int(w.sum()) == 0:
            w = P
    run = w.cumsum(0)
    thr = int(Fraction(float(u_sample)) * int(run[-1]))      # (a whole number is above it where it is above its floor)
    tok = int(torch.searchsorted(run, torch.tensor([thr], device=run.device), right=True)[0])
    return [int(x) for x in drafts[:a]] + [tok]


def go(target, drafts, draft_probs, u_accept, u_sample):
    lib, (B, N) = lib_(), drafts.shape
    i32 = dict(dtype=torch.int32, device=DEV)
    tokens, n_out = torch.full((B, N + 1), 99, **i32), torch.full((B,), 99, **i32)
    lib.ds4a_verify_drafts(target, drafts, u_accept, u_sample, tokens, n_out, draft_probs=draft_probs)
    tokens, n_out, some = tokens.cpu(), n_out.cpu(), target.view(B, N + 1, -1)
    for b in range(B):
        want = definition(some[b], drafts[b], None if draft_probs is None else draft_probs[b], u_accept[b], u_sample[b])
        assert tokens[b].tolist() == want + [-1] * (N + 1 - len(want)) and int(n_out[b]) == len(want), b


def test_the_integer_definition_is_the_oracles():
    for sampled in (True, False):
        x = make(3, 6, 2, 301, "f32", sampled)
        for b in range(6):
            t, q = x["target"][3 * b:3 * b + 3], None if x["draft_probs"] is None else x["draft_probs"][b]
            want = kv.verify(np_(t), x["drafts"][b].numpy(), None if q is None else np_(q), x["u_accept"][b].numpy(),
                             float(x["u_sample"][b]), 3)
            assert definition(t, x["drafts"][b], q, x["u_accept"][b], x["u_sample"][b]) == want


@pytest.mark.parametrize("B", [77, 153, 305, 700])
@pytest.mark.parametrize("dtype,sampled", [("f32", True), ("bf16", True), ("f32", False)])
def test_eight_to_one_blocks_a_sequence(B, dtype, sampled):
    """(On 152 SMs: eight blocks a sequence up to 76 of them, four to 152, two to 304.)"""
    check(make(B, B, 2, 261, dtype, sampled), B, 2)
    rng = np.random.default_rng(B)
    check(make(B + 1, B, 3, 64, dtype, sampled, rng.integers(0, 6, B)), B, 3)


def big(seed, B, V, dtype, N=1, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = torch.randn((B * (N + 1), V), generator=g, device=DEV) * 2
    wide = torch.zeros((B * (N + 1), V + pad), dtype=TD[dtype], device=DEV)
    wide[:, :V] = torch.softmax(logits, -1)
    near = torch.softmax(logits.view(B, N + 1, V)[:, :N] + 0.5 * torch.randn((B, N, V), generator=g, device=DEV), -1)
    drafts = near.argmax(-1).int()
    u = torch.rand((B, N + 1), generator=g, device=DEV)
    u[::3, N] = 1 - 2.0 ** -24                   # the last token with weight: the last chunk, a part of one
    u[1::3, N] = torch.rand((len(u[1::3]),), generator=g, device=DEV) * 0.02 + 0.98
    return wide[:, :V], drafts, near.to(TD[dtype]), u[:, :N].contiguous(), u[:, N].contiguous()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V,pad", [(5, 131072, 0), (5, 131073, 0), (4, 262145, 3), (4, 1 << 20, 0), (3, (1 << 20) - 1, 0),
                                     (310, 100277, 0), (160, 50000, 4)])
def test_large_vocabularies(B, V, pad, dtype):
    """Sums in smaller steps than 2^-45; a warp's many chunks; one and two blocks a sequence."""
    target, drafts, probs, ua, us = big(V + B, B, V, dtype, pad=pad)
    go(target, drafts, probs, ua, us)
    go(target, drafts, None, ua, us)


def test_one_block_for_the_largest_vocabulary():
    """306 sequences without drafts of their own: 2,048 chunks in one block."""
    B, V = 306, 1 << 20
    g = torch.Generator(device=DEV).manual_seed(1)
    target = torch.softmax(torch.randn((B, V), generator=g, device=DEV), -1)
    us = torch.rand(B, generator=g, device=DEV)
    us[::5] = 1 - 2.0 ** -24
    i32 = dict(dtype=torch.int32, device=DEV)
    tokens, n_out = torch.empty((B, 2), **i32), torch.empty(B, **i32)
    lib_().ds4a_verify_drafts(target, torch.zeros((B, 1), **i32), torch.zeros((B, 1), device=DEV), us, tokens, n_out,
                              cu_len=torch.arange(B + 1, **i32))
    for b in range(B):
        assert tokens[b].tolist() == definition(target[b:b + 1], [], None, [], us[b]) + [-1] and int(n_out[b]) == 1


def test_thresholds_next_to_a_running_sum():
    """u times the sum is below a running sum by less than fp64 holds: that token is the first above it."""
    V, shift, rng = 64, 45, np.random.default_rng(5)
    rows, us, want = [], [], []
    while len(rows) < 24:
        T = int(rng.integers(1 << 44, 1 << 45)) | 1
        M = -pow(T, -1, 1 << 24) % (1 << 24)                 # M T = -1 modulo 2^24: u T ends 2^-24 below a whole number
        a = (M * T + 1) >> 24
        if not a or a >= T or M < 1 << 20:
            continue
        pieces = lambda x: [x >> s << s & (1 << s + 22) - 1 for s in (0, 22, 44)]  # noqa: E731  (22 bits each)
        w = np.zeros(V)
        w[[3, 11, 20]] = pieces(a)
        w[[21, 40, 63]] = pieces(T - a)
        first = max(i for i in (3, 11, 20) if w[i])
        p = torch.tensor(w * 2.0 ** -shift)
        assert int(w.sum()) == T and (p.float().double() == p).all()
        rows.append(p.float())
        us.append(M / (1 << 24))
        want.append(first)
    n = len(rows)
    i32 = dict(dtype=torch.int32, device=DEV)
    target, u = torch.stack(rows).to(DEV), torch.tensor(us, dtype=torch.float32, device=DEV)
    for i in range(n):
        assert kv.verify(np_(target[i:i + 1]), [], None, [], float(u[i]), 1) == [want[i]]
    tokens, n_out = torch.empty((n, 2), **i32), torch.empty(n, **i32)
    lib_().ds4a_verify_drafts(target, torch.zeros((n, 1), **i32), torch.zeros((n, 1), device=DEV), u, tokens, n_out,
                              cu_len=torch.arange(n + 1, **i32))
    assert tokens[:, 0].tolist() == want
