"""Pins of oracle/kv.py: facts that hold whatever the implementation."""
import numpy as np
import pytest

from oracle import kv


def test_rotation_keeps_norms_and_relative_positions():
    rng = np.random.default_rng(1)
    for half in (False, True):
        for rot_at, rot in ((0, 16), (4, 8), (8, 8)):
            x, y = rng.normal(size=(2, 1, 3, 16))
            kw = dict(n_rot=rot, base=10000.0, rot_at=rot_at, half=half)
            a = kv.rotate(x, [7], **kw)
            assert np.allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x, axis=-1))
            b = kv.rotate(y, [19], **kw)
            a2, b2 = kv.rotate(x, [107], **kw), kv.rotate(y, [119], **kw)
            assert np.allclose((a * b).sum(-1), (a2 * b2).sum(-1))
            assert np.allclose(kv.rotate(a, [7], inverse=True, **kw), x)
            keep = np.ones(16, bool)
            keep[rot_at:rot_at + rot] = False
            assert (a[..., keep] == x[..., keep]).all()


def test_pairs_of_both_layouts():
    x = np.zeros((1, 1, 8))
    x[..., 2] = 1.0
    a = kv.rotate(x, [1], 8, 10000.0, half=False)       # pair 1: dims 2 and 3
    th = 10000.0 ** (-2 / 8)
    assert np.allclose(a[0, 0], [0, 0, np.cos(th), np.sin(th), 0, 0, 0, 0])
    b = kv.rotate(x, [1], 8, 10000.0, half=True)        # pair 2: dims 2 and 6
    th = 10000.0 ** (-4 / 8)
    assert np.allclose(b[0, 0], [0, 0, np.cos(th), 0, 0, 0, np.sin(th), 0])


def test_scaled_angles():
    th, _ = kv.theta(64, 10000.0)
    lin, _ = kv.theta(64, 10000.0, kind="linear", factor=4.0)
    assert np.allclose(lin * 4, th)
    ntk, _ = kv.theta(64, 10000.0, kind="ntk", factor=4.0)
    assert ntk[0] == th[0] and np.isclose(ntk[-1] * 4, th[-1])   # the slowest pair is stretched whole
    y, mag = kv.theta(64, 10000.0, kind="yarn", factor=4.0, orig_len=4096.0)
    assert np.isclose(mag, 0.1 * np.log(4.0) + 1)
    turns = 4096 * th / (2 * np.pi)
    assert np.allclose(y[turns > 40], th[turns > 40]) and np.allclose(y[turns < 0.7] * 4, th[turns < 0.7])
    assert (y <= th * (1 + 1e-12)).all() and (y * 4 >= th * (1 - 1e-12)).all()
    same, one = kv.theta(64, 10000.0, kind="yarn", factor=1.0, orig_len=4096.0)
    assert np.allclose(same, th) and one == 1.0


def test_e4m3_values():
    t = kv.e4m3_table()
    assert t[0x7E] == 448 and np.isnan(t[0x7F]) and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[0xC0] == -2.0
    assert (np.diff(t[:127]) > 0).all()
    fin = t[~np.isnan(t)]
    assert np.array_equal(kv.to_e4m3(fin), fin)
    mid = (t[:126] + t[1:127]) / 2                       # ties: the even code
    even = np.where(np.arange(126) % 2 == 0, t[:126], t[1:127])
    assert np.array_equal(kv.to_e4m3(mid), even)
    assert list(kv.to_e4m3([1e9, -500.0, np.inf])) == [448, -448, 448] and np.isnan(kv.to_e4m3(np.nan))


def test_attention_of_equal_scores_is_the_mean_and_windows_cut():
    rng = np.random.default_rng(2)
    K, D, nb = 2, 4, 5
    pk, pv = np.zeros((nb, K, 256, D)), rng.normal(size=(nb, K, 256, D))
    table = np.array([[3, 1, -1], [4, 0, 2]])
    q = rng.normal(size=(3, 4, D))
    out, lse, _, _ = kv.attention(q, pk, pv, table, [299, 9], [0, 2, 3], 0.5)
    seen = np.concatenate([pv[3], pv[1][:, :44]], 1)
    assert np.allclose(out[0, 0], seen[0].mean(0)) and np.allclose(out[0, 3], seen[1].mean(0))
    assert np.allclose(lse, [[np.log(300)] * 4, [np.log(301)] * 4, [np.log(10)] * 4])
    out, lse, _, _ = kv.attention(q, pk, pv, table, [299, 9], [0, 2, 3], 0.5, window=1)
    assert np.allclose(out[1, 1], pv[1, 0, 44]) and np.allclose(lse, 0)
    out, lse, _, _ = kv.attention(q[:1], pk, pv, table, [600, 0], [0, 1, 1], 0.5, window=50)   # a block that is not there
    assert (out == 0).all() and np.isneginf(lse).all()


def test_verified_tokens_are_distributed_as_the_target():
    """Summed over the draft's distribution and an even grid of random numbers."""
    V, n = 5, 400
    p = np.array([[0.4, 0.1, 0.2, 0.0, 0.3], [0.2] * 5])
    q = np.array([[0.1, 0.3, 0.2, 0.2, 0.2]])
    got = np.zeros(V)
    u = (np.arange(n) + 0.5) / n
    for x in range(V):
        stands = np.array([len(kv.verify(p, [x], q, [v], 0.5, 2)) == 2 for v in u])
        got[x] += q[0, x] * stands.mean()
        if stands.all():
            continue
        new = [kv.verify(p, [x], q, [1 - 1e-9], v, 2)[0] for v in u]
        got += q[0, x] * (1 - stands.mean()) * np.bincount(new, minlength=V) / n
    assert np.allclose(got, p[0], atol=2 / n)


@pytest.mark.parametrize("greedy", [False, True])
def test_verify_by_hand(greedy):
    p = np.array([[0.5, 0.5, 0, 0], [0, 0, 0.25, 0.75], [0.1, 0.2, 0.3, 0.4]])
    q = None if greedy else np.array([[1.0, 0, 0, 0], [0, 0, 0, 1.0]])
    assert kv.verify(p, [0, 3], q, [0.4, 0.7], 0.35, 3) == [0, 3, 2]     # both stand, then p
    assert kv.verify(p, [0, 3], q, [0.4, 0.8], 0.9, 3) == [0, 2]         # the second falls
    assert kv.verify(p, [0, 3], q, [0.5, 0.0], 0.1, 3) == [1]            # u q = p falls
    assert kv.verify(p, [0, 3], q, [0.4, 0.7], 0.6, 1) == [1]            # no drafts
    assert kv.verify(p, [9, 3], q if greedy else np.zeros((2, 4)), [0.0, 0.0], 0.6, 3) == [1]
