"""One key, or one that all the others vanish beside: its weight is a power of two on every path, and the output its
value, rounded once."""
import pytest
import torch

from kv_step import Step, values_of
from test_gpu_paged_attn import run
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,kvd,D", [("bf16", "bf16", 128), ("bf16", "e4m3", 128), ("bf16", "e4m3", 64), ("f32", "f32", 80)])
@pytest.mark.parametrize("G", [1, 8, 24, 40])
def test_the_output_is_its_value(dtype, kvd, D, G):
    step = Step(lib_(), G + D, [0] * 40, [1] * 40, 2 * G, 2, D, dtype, kvd)
    c, cu = step.on_gpu()
    out, lse = run(step, c, cu)
    v = values_of(step.pv, step.v_scale, kvd)[step.table[:, 0], :, 0]          # [sequence][K][D]
    want = torch.from_numpy(v).repeat_interleave(G, 1)
    got = out.cpu().double()
    if kvd == "e4m3":    # code * scale / (the weights' sum): two roundings of fp32 before the last one
        assert ((got - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -22)).all()
        exact = want.bfloat16().double()
        assert ((got - exact).abs() <= exact.abs() * 2.0 ** -7).all() and (got == exact).double().mean() > 0.999
    else:
        assert torch.equal(got, want.to(out.dtype).double())
