"""ds4a_norm_rope against oracle/serving.py.

Tolerance, from the arithmetic: with u = 2^-24, the sum of n <= 1024 squares is off by at
most n u relative (any order), its root by half of that, and the division, two products and
(rotated) two products and a sum add at most 8 u: |error| <= (n / 2 + 8) u (|a| + |b|), a and
b the dims of a rotated pair (b = 0 elsewhere), plus half a step of the stored type."""
import numpy as np
import pytest
import torch

from helpers import np_
from oracle import serving
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV = "cuda"
TD = {"bf16": torch.bfloat16, "f32": torch.float32}
BASE, MAXP = 10000.0, 512


def make_cache(D, rot, dtype, batch=3, cap_raw=128):
    return lib_().LayerCache(ratio=0, head_dim=D, n_rot=rot, batch=batch, comp_cap=0, dtype=dtype,
                             base=BASE, rope_max_pos=MAXP, cap_raw=cap_raw, device=DEV)


def near(got, x, gamma, pos, rot, dtype, rotate):
    D = x.shape[-1]
    want = serving.norm_rope(np_(x), None if gamma is None else np_(gamma), pos, BASE, rot, rotate)
    plain = np.abs(serving.norm_rope(np_(x), None if gamma is None else np_(gamma), pos, BASE, rot,
                                     False))
    if rotate and rot:
        t = plain[..., D - rot:]
        plain[..., D - rot:] = np.repeat(t[..., 0::2] + t[..., 1::2], 2, -1)
    tol = (D / 2 + 8) * 2.0 ** -24 * plain + torch.finfo(TD[dtype]).eps / 2 * np.abs(want) + 1e-38
    err = np.abs(np_(got).astype(np.float64) - want)
    assert (err <= tol).all(), float((err / tol).max())


CASES = [  # n, H, D, rot, dtype, fused, rot_q
    (1, 1, 512, 64, "bf16", False, True), (8, 64, 512, 64, "bf16", True, True),
    (77, 64, 512, 64, "bf16", False, False), (5, 3, 128, 64, "f32", True, True),
    (333, 5, 128, 128, "f32", False, True), (9, 128, 512, 2, "bf16", False, True),
    (4, 7, 1024, 32, "f32", False, True), (4, 7, 1024, 64, "bf16", True, True),
    (6, 2, 20, 6, "bf16", False, True), (6, 3, 84, 4, "bf16", True, True),
    (3, 2, 4, 2, "f32", False, True), (10, 24, 192, 64, "bf16", True, False),
]


@pytest.mark.parametrize("n,H,D,rot,dtype,fused,rot_q", CASES)
def test_norm_rope(n, H, D, rot, dtype, fused, rot_q):
    lib = lib_()
    g = torch.Generator().manual_seed(n * H + D)
    both = (torch.randn((n, (H + 1) * D), generator=g) *
            torch.pow(2.0, torch.randint(-8, 8, (n, 1), generator=g).float())).to(DEV, TD[dtype])
    q, kv = both[:, :H * D].view(n, H, D), both[:, H * D:]
    if not fused:
        q, kv = q.contiguous(), kv.contiguous()
    gq, gk = ((1 + 0.1 * torch.randn(D, generator=g)).to(DEV, TD[dtype]) for _ in range(2))
    pos = torch.randint(0, MAXP, (n,), generator=g, dtype=torch.int32)
    c = make_cache(D, rot, dtype)
    ring0 = c.raw_kv.normal_().clone()
    slots = torch.randperm(3 * 128, generator=g)[:n].int()
    q_out = torch.empty((n, H, D), dtype=TD[dtype], device=DEV)
    lib.ds4a_norm_rope(c, pos.to(DEV), q=q, gamma_q=gq, q_out=q_out, kv=kv, gamma_kv=gk,
                       slots=slots.to(DEV), rot_q=rot_q)
    near(q_out, q, gq, pos.numpy(), rot, dtype, rot_q)
    rows = c.raw_kv.view(-1, D)
    near(rows[slots.long().to(DEV)], kv, gk, pos.numpy(), rot, dtype, True)
    rest = torch.ones(3 * 128, dtype=torch.bool)
    rest[slots.long()] = False
    assert torch.equal(rows[rest.to(DEV)], ring0.view(-1, D)[rest.to(DEV)])
    # the rows token by token, without a gain, alone: the same up to the gain
    out = torch.empty((n, D), dtype=TD[dtype], device=DEV)
    lib.ds4a_norm_rope(c, pos.to(DEV), kv=kv, kv_out=out)
    near(out, kv, None, pos.numpy(), rot, dtype, True)


def test_skipped_tokens_and_dropped_slots():
    lib = lib_()
    n, H, D = 6, 3, 512
    c = make_cache(D, 64, "bf16", batch=1)
    ring0 = c.raw_kv.normal_().clone()
    q = torch.randn((n, H, D), device=DEV).bfloat16()
    kv = torch.randn((n, D), device=DEV).bfloat16()
    pos = torch.tensor([0, -1, MAXP, MAXP - 1, 5, -2**31], dtype=torch.int32)
    slots = torch.tensor([3, 4, 5, -1, 128, 6], dtype=torch.int32)
    out = torch.full_like(q, 9)
    lib.ds4a_norm_rope(c, pos.to(DEV), q=q, q_out=out, kv=kv, slots=slots.to(DEV))
    live = [0, 3, 4]
    near(out[live], q[live], None, pos.numpy()[live], 64, "bf16", False)
    assert (out[[1, 2, 5]] == 9).all()
    near(c.raw_kv[0, 3:4], kv[:1], None, pos.numpy()[:1], 64, "bf16", True)
    keep = [i for i in range(128) if i != 3]
    assert torch.equal(c.raw_kv[0, keep], ring0[0, keep])


def test_in_place_zero_rows_and_non_finite_ones():
    lib = lib_()
    c = make_cache(512, 64, "bf16")
    q = torch.randn((4, 2, 512), device=DEV).bfloat16()
    q[1, 0] = 0
    q[2, 1, 7] = float("nan")
    q[3, 0, 500] = float("inf")
    kv = torch.randn((4, 512), device=DEV).bfloat16()
    q0, kv0 = q.clone(), kv.clone()
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    lib.ds4a_norm_rope(c, pos, q=q, q_out=q, kv=kv, kv_out=kv, rot_q=True)
    near(q[:2], q0[:2], None, np.arange(2), 64, "bf16", True)
    near(kv, kv0, None, np.arange(4), 64, "bf16", True)
    assert (q[1, 0] == 0).all()
    assert q[2, 1].isnan().all() and not q[2, 0].isnan().any() and not q[3, 1].isnan().any()


def test_many_tokens_other_stream_and_replayed_graph():
    lib = lib_()
    n, H, D = 4096, 8, 512
    c = make_cache(D, 64, "bf16")
    q = torch.randn((n, H, D), device=DEV).bfloat16()
    pos = torch.randint(0, MAXP, (n,), dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lib.ds4a_norm_rope(c, pos, q=q, q_out=out, rot_q=True, stream=s)
    s.synchronize()
    near(out[:64], q[:64], None, pos[:64].cpu().numpy(), 64, "bf16", True)
    near(out[-64:], q[-64:], None, pos[-64:].cpu().numpy(), 64, "bf16", True)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.ds4a_norm_rope(c, pos, q=q, q_out=out, rot_q=True)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    q.mul_(2)          # new inputs, same result up to the epsilon
    pos.fill_(1)
    g.replay()
    torch.cuda.synchronize()
    near(out[:64], q[:64], None, np.ones(64), 64, "bf16", True)


def test_offsets_pass_32_bits():
    """The last of so many tokens that their elements are numbered beyond 2^32."""
    lib = lib_()
    H, D = 64, 512
    n = (1 << 32) // (H * D) + 5
    c = make_cache(D, 64, "bf16")
    q = torch.zeros((n, H, D), dtype=torch.bfloat16, device=DEV)
    q[-7:] = torch.randn((7, H, D), device=DEV).bfloat16()
    pos = torch.arange(n, dtype=torch.int32, device=DEV) % MAXP
    out = torch.empty_like(q)
    lib.ds4a_norm_rope(c, pos, q=q, q_out=out, rot_q=True)
    near(out[-7:], q[-7:], None, pos[-7:].cpu().numpy(), 64, "bf16", True)
    assert not out[:-7].any()
