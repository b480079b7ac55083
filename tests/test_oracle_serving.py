"""Pins of oracle/serving.py: the 4-bit row layout (every code dim has a place of its
own, none overlapping another or a scale), hand-made E2M1 roundings, the norm's
closed forms, and block tables by hand."""
import numpy as np
import pytest

from oracle import serving


@pytest.mark.parametrize("D,n_rot,es", [(512, 64, 2), (128, 64, 4), (336, 64, 4), (1024, 32, 2),
                                        (1024, 16, 4), (16, 0, 2), (80, 64, 2)])
def test_row_layout_places_are_disjoint(D, n_rot, es):
    nb, ns, R, tail, nbytes = serving.row_layout(D, n_rot, es)
    assert nbytes % 32 == 0 and nbytes >= tail + n_rot * es and tail == 32 * R
    bits, scales = set(), {}
    for d in range(D - n_rot):
        at, t, sc = serving.dim_place(D, n_rot, d, es)
        mine = {(at * 8 + b) for b in (serving.SIGN[t], *(serving.MAG[t] + i for i in range(3)))}
        assert at + 1 < tail and not mine & bits
        bits |= mine
        assert scales.setdefault(sc, d // 16) == d // 16   # one scale byte per 16 dims
    assert len(scales) == (D - n_rot) // 16
    assert not {8 * s + b for s in scales for b in range(8)} & bits


def test_flash_row_is_384_bytes():
    assert serving.row_layout(512, 64, 2)[4] == 384


def test_quantise_row_by_hand():
    x = np.zeros(24)
    x[:16] = [6, -6, 0.25, 0.26, 0.75, -1.25, 1.75, 2.5, 3.5, 5.0, 5.01, -0.2, 3, 2, 1, 0.5]
    want = [6, -6, 0, 0.5, 1, -1, 2, 2, 4, 4, 6, 0, 3, 2, 1, 0.5]
    x[16:] = 1.2345
    got = serving.quantise_row(x, 8, "f32")
    assert np.array_equal(np.abs(got[:16]), np.abs(want)) and (got[1], got[5]) == (-6, -1)
    assert np.array_equal(got[16:], np.full(8, np.float32(1.2345), np.float64))
    # the scale is the smallest power of two that holds the largest magnitude
    assert np.array_equal(serving.quantise_row(x * 8, 8, "f32")[:16], 8 * got[:16])
    x[0] = 6.001
    assert serving.quantise_row(x, 8, "f32")[0] == 6 and serving.quantise_row(x, 8, "f32")[3] == 0
    x[0] = np.inf
    assert np.isnan(serving.quantise_row(x, 8, "f32")[:16]).all()


def test_norm_closed_forms():
    x = np.full((2, 3, 8), -2.0)
    y = serving.norm_rope(x, None, [0, 5], 10000.0, 4, False)
    assert np.allclose(y, -2.0 / np.sqrt(4.0 + 1e-6))
    g = np.arange(8) + 1.0
    assert np.allclose(serving.norm_rope(x, g, [0, 5], 1e4, 4, False), y * g)
    r = serving.norm_rope(x, None, [0, 5], 10000.0, 4, True)
    assert np.allclose(r[0], y[0]) and np.allclose(r[1, :, :4], y[1, :, :4])   # angle 0; head dims
    assert np.allclose((r ** 2).sum(-1), (y ** 2).sum(-1))                     # norms stay
    assert np.allclose(serving.norm_rope(np.zeros((1, 8)), None, [1], 1e4, 4, True), 0)


def test_block_tables_by_hand():
    pool = {"table": np.full((3, 3), -1), "held": np.array([1, 0, 2]),
            "free_list": np.array([7, 4, -1, -1, -1, 5, 6, 3]), "state": np.array([5, 5, 0, 0])}
    pool["table"][0, 0], pool["table"][2, :2] = 0, (1, 2)
    out = serving.block_tables(pool, [257, 0, 256], [2, 0, 1], 128, 5)
    assert pool["table"].tolist() == [[0, 5, -1], [-1, -1, -1], [1, -1, -1]]
    assert pool["held"].tolist() == [2, 0, 1] and pool["state"].tolist() == [6, 5, 0, 0]
    assert pool["free_list"][2] == 2                       # given back, behind the free ones
    assert out["tok_pos"].tolist() == [255, 256, 255, -1, -1]
    assert out["tok_seq"].tolist() == [0, 0, 2, -1, -1]
    assert out["raw_slot"].tolist() == [127, 0, 2 * 128 + 127, -1, -1]
    assert out["comp_slot4"].tolist() == [63, -1, 64 + 63, -1, -1]
    assert out["comp_slot128"].tolist() == [1, -1, 3, -1, -1]
    assert out["seq_pos"].tolist() == [255, 0, 255] and out["cu_len"].tolist() == [0, 2, 2, 3]
    # more blocks than there are: the last rows go short, and ask again
    out = serving.block_tables(pool, [768, 768, 768], [200, 0, 1], 128, 201)
    assert pool["held"].tolist() == [3, 3, 2] and pool["state"][1:3].tolist() == [0, 1]
    assert out["raw_slot"][:72].tolist() == [-1] * 72 and out["raw_slot"][72] == (768 - 128) % 128
    assert out["comp_slot4"][200] == -1
