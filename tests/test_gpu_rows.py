"""Compressed rows to and from 4 bits against oracle/serving.py: bit for bit (the
decisions are exact in fp32), at every alignment, type and odd size, with the values at
which a rounding or a scale turns."""
import numpy as np
import pytest
import torch

from helpers import np_
from oracle import serving
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV = "cuda"
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def make_cache(D, rot, dtype, cap, paged=None, batch=1):
    lib = lib_()
    return lib.LayerCache(ratio=128, head_dim=D, n_rot=rot, batch=batch, comp_cap=cap, dtype=dtype,
                          base=160000.0, rope_max_pos=16, qat=lib.FP4_ROWS, device=DEV)


def hard_rows(n, D, dtype, seed):
    """Normal rows of several magnitudes, and rows on the codes' decision points."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, D), generator=g)
    x *= torch.pow(2.0, torch.randint(-30, 30, (n, 1), generator=g).float())
    mid = torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6.25])
    x[::3] = mid[torch.randint(0, 16, (x[::3].shape[0], D), generator=g)] * 0.25
    x[::3] *= torch.sign(torch.randn(x[::3].shape, generator=g))
    return x.to(TD[dtype])


@pytest.mark.parametrize("D,rot,dtype", [(512, 64, "bf16"), (512, 64, "f32"), (128, 64, "f32"),
                                         (336, 64, "bf16"), (1024, 16, "f32"), (1024, 128, "bf16"),
                                         (84, 4, "bf16"), (20, 4, "f32"), (48, 16, "bf16")])
@pytest.mark.parametrize("n", [1, 33])
def test_pack_and_read_back(D, rot, dtype, n):
    lib = lib_()
    cap = n + 5
    c = make_cache(D, rot, dtype, cap)
    c.attn_comp_kv.fill_(0xA5)
    x = hard_rows(n, D, dtype, 3 * n + D).to(DEV)
    slots = torch.randperm(cap, generator=torch.Generator().manual_seed(n))[:n].int().to(DEV)
    lib.ds4a_pack_rows(c, x, slots)
    got = torch.full_like(x, -7)
    lib.ds4a_unpack_rows(c, got, slots)
    torch.cuda.synchronize()
    want = serving.quantise_row(np_(x), rot, dtype)
    assert np.array_equal(np_(got).astype(np.float64), want)
    raw = c.attn_comp_kv[0].cpu().numpy()
    for i in (0, n - 1):      # the bytes, dim by dim
        assert np.array_equal(serving.read_row(raw[int(slots[i])], D, rot, dtype), want[i])
    other = np.setdiff1d(np.arange(cap), slots.cpu().numpy())
    assert (raw[other] == 0xA5).all()


def test_extreme_values():
    """Zeros, subnormals, the largest values, infinities and NaN; a bad block is NaN and
    its neighbours are not."""
    lib = lib_()
    D, rot = 512, 64
    x = torch.ones((8, D))
    x[0] = 0
    x[1] *= 2.0 ** -140
    x[2, :16] = torch.finfo(torch.float32).max
    x[3, 3] = float("inf")
    x[4, 20] = float("nan")
    x[5, 447] = float("-inf")
    x[6, 500] = float("nan")           # rotated tail: kept as it is
    x[7] *= 2.0 ** 126
    c = make_cache(D, rot, "f32", 8)
    x = x.to(DEV)
    got = torch.empty_like(x)
    lib.ds4a_pack_rows(c, x)
    lib.ds4a_unpack_rows(c, got)
    want = serving.quantise_row(np_(x), rot, "f32")
    assert np.array_equal(np_(got).astype(np.float64), want, equal_nan=True)
    assert np.isnan(want).sum() == 3 * 16 + 1


def test_slots_outside_the_pool_and_views():
    lib = lib_()
    c = make_cache(512, 64, "bf16", 8)
    x = hard_rows(6, 512, "bf16", 1).to(DEV)
    slots = torch.tensor([2, -1, 8, 2**31 - 1, 0, -2**31], dtype=torch.int32, device=DEV)
    c.attn_comp_kv.fill_(0x11)
    lib.ds4a_pack_rows(c, x, slots)
    got = torch.full_like(x, 3)
    lib.ds4a_unpack_rows(c, got, slots)
    want = serving.quantise_row(np_(x), 64, "bf16")
    for i, live in enumerate((True, False, False, False, True, False)):
        assert np.array_equal(np_(got[i]), want[i] if live else np.full(512, 3.0))
    assert (c.attn_comp_kv[0, [1, 3, 4, 5, 6, 7]] == 0x11).all()
    # rows that start off 16 bytes take the element-wise form, with the same result
    odd = torch.empty(6 * 512 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(6, 512)
    odd.copy_(x)
    a = c.attn_comp_kv.clone()
    lib.ds4a_pack_rows(c, odd, slots)
    assert torch.equal(a, c.attn_comp_kv)
    back = torch.full((6 * 512 + 1,), 3.0, dtype=torch.bfloat16, device=DEV)[1:].view(6, 512)
    lib.ds4a_unpack_rows(c, back, slots)
    assert torch.equal(back, got)


def test_large_pool_offsets_pass_32_bits():
    lib = lib_()
    cap = (1 << 32) // 384 + 4096
    c = make_cache(512, 64, "bf16", cap)
    slots = torch.tensor([cap - 1, 0, (1 << 32) // 384 + 1], dtype=torch.int32, device=DEV)
    x = hard_rows(3, 512, "bf16", 5).to(DEV)
    lib.ds4a_pack_rows(c, x, slots)
    got = torch.empty_like(x)
    lib.ds4a_unpack_rows(c, got, slots)
    assert np.array_equal(np_(got), serving.quantise_row(np_(x), 64, "bf16"))
