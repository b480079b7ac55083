"""A NaN in a seen value shows in the output however small its weight (ds4a_paged_attn_decode): in a part of
a divided sequence that the others' weights dwarf, and in a tile that only some tokens see whole."""
import numpy as np
import pytest
import torch

from helpers import np_
from kv_step import Step
from test_gpu_paged_attn import run
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
FORMS = [("bf16", "bf16", 128), ("bf16", "bf16", 256), ("bf16", "e4m3", 128), ("f32", "f32", 64), ("f32", "f32", 160),
         ("bf16", "bf16", 20)]


def quiet(step, b, keys, nan_at, dim):
    """Scores of these keys of sequence b some 250 below the others'; a NaN in the value of one."""
    f8 = step.kv_dtype == "e4m3"
    step.q[:, :, 0] = 8.0
    for p in keys:
        blk, r = step.table[b, p // 256], p % 256
        step.pk[blk, :, r, 0] = torch.tensor(-250.0 / 8 / (float(step.k_scale.max()) if f8 else 1.0)).clamp(-448, 448).to(step.pk.dtype)
        if f8:
            step.pk[blk, :, r, 0] = torch.tensor(-448.0).to(step.pk.dtype)
    blk, r = step.table[b, nan_at // 256], nan_at % 256
    step.pv[blk, 1, r, dim] = float("nan")


def look(step, c, cu, row, dim):
    out, lse = run(step, c, cu, scale=4.0 if step.kv_dtype == "e4m3" else 1.0)
    want = np.zeros((step.n, step.H, step.D), bool)
    want[row, step.H // 2:, dim] = True
    assert (np.isnan(np_(out)) == want).all()
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype,kvd,D", FORMS)
def test_in_a_part_of_a_divided_sequence(dtype, kvd, D):
    step = Step(lib_(), D, [6000], [1], 8, 2, D, dtype, kvd, std=0.2)
    quiet(step, 0, range(2048), 300, 5)
    look(step, *step.on_gpu(), slice(None), 5)


@pytest.mark.parametrize("dtype,kvd,D", FORMS)
@pytest.mark.parametrize("old", [40, 700])
def test_in_a_tile_that_some_tokens_see_whole(dtype, kvd, D, old):
    step = Step(lib_(), D + old, [old], [3], 8, 2, D, dtype, kvd, std=0.2)
    quiet(step, 0, [old - 3], old - 3, 7)
    look(step, *step.on_gpu(), slice(None), 7)


@pytest.mark.parametrize("dtype,kvd,D", FORMS)
def test_not_where_it_is_not_seen(dtype, kvd, D):
    """The NaN of a later token's own row, and of one outside the window."""
    step = Step(lib_(), D + 1, [700], [3], 8, 2, D, dtype, kvd, window=600, std=0.2)
    quiet(step, 0, [701, 103], 701, 7)
    blk, r = step.table[0, 0], 103
    step.pv[blk, 1, r, 9] = float("nan")          # seen by the tokens at 700, 701 and 702 from 101, 102 and 103 on
    c, cu = step.on_gpu()
    out, _ = run(step, c, cu, scale=4.0 if kvd == "e4m3" else 1.0)
    want = np.zeros((3, 8, D), bool)
    want[1:, 4:, 7] = True
    want[:, 4:, 9] = True
    assert (np.isnan(np_(out)) == want).all()
