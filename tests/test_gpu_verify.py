"""ds4a_verify_drafts against oracle/kv.py: whole numbers, equal."""
import numpy as np
import pytest
import torch

from helpers import np_
from kv_step import TD
from oracle import kv
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(seed, B, N, V, dtype, sampled, cnt=None, pad=0):
    g = torch.Generator().manual_seed(seed)
    cnt = np.full(B, N + 1) if cnt is None else np.array(cnt)
    cu = np.concatenate([[0], np.cumsum(cnt)])
    logits = torch.randn((int(cu[-1]), V), generator=g) * 2
    target = torch.zeros((int(cu[-1]), V + pad), dtype=TD[dtype])
    target[:, :V] = torch.softmax(logits, -1).to(TD[dtype])
    at = torch.from_numpy(np.minimum(cu[:-1, None] + np.arange(N), np.maximum(cu[1:, None] - 1, 0)).clip(0, len(logits) - 1))
    near = torch.softmax(logits[at] + 0.5 * torch.randn((B, N, V), generator=g), -1)
    drafts = torch.multinomial(near.view(-1, V), 1, generator=g).view(B, N).int()
    if not sampled:
        drafts = torch.where(torch.rand((B, N), generator=g) < 0.5, logits[at].argmax(-1).int(), drafts)
    return dict(target=target[:, :V], drafts=drafts, draft_probs=near.to(TD[dtype]) if sampled else None,
                u_accept=torch.rand((B, N), generator=g), u_sample=torch.rand(B, generator=g), cnt=cnt, cu=cu)


def call(x, B, N, cu=True, **kw):
    lib = lib_()
    i32 = dict(dtype=torch.int32, device=DEV)
    tokens, n_out, ctx = torch.full((B, N + 1), 99, **i32), torch.full((B,), 99, **i32), torch.full((B,), 99, **i32)
    pos = torch.arange(B, **i32) * 7 + 3
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    base = x["target"]._base if x["target"]._base is not None else x["target"]
    target = base.to(DEV)[:, :x["target"].shape[1]]
    lib.ds4a_verify_drafts(target, d(x["drafts"]), d(x["u_accept"]), d(x["u_sample"]), tokens, n_out,
                           draft_probs=d(x["draft_probs"]), cu_len=torch.tensor(x["cu"], **i32) if cu else None,
                           seq_pos=pos, ctx_out=ctx, **kw)
    return tokens.cpu().numpy(), n_out.cpu().numpy(), ctx.cpu().numpy()


def check(x, B, N, **kw):
    tokens, n_out, ctx = call(x, B, N, **kw)
    for b in range(B):
        want = []
        if x["cnt"][b]:
            rows = slice(int(x["cu"][b]), int(x["cu"][b + 1]))
            want = kv.verify(np_(x["target"])[rows], x["drafts"][b].numpy(),
                             None if x["draft_probs"] is None else np_(x["draft_probs"])[b], x["u_accept"][b].numpy(),
                             float(x["u_sample"][b]), int(x["cnt"][b]))
        assert tokens[b].tolist() == want + [-1] * (N + 1 - len(want)), b
        assert n_out[b] == len(want) and ctx[b] == 7 * b + 3 + len(want)


CASES = [(1, 1, 1, "f32", False), (3, 4, 7, "f32", True), (8, 3, 1000, "f32", False), (5, 7, 5003, "f32", True),
         (4, 2, 4096, "bf16", True), (2, 5, 3001, "bf16", False), (30, 2, 129, "f32", True), (2, 40, 300, "f32", True),
         (2, 3, 50021, "f32", True)]


@pytest.mark.parametrize("B,N,V,dtype,sampled", CASES)
def test_verify(B, N, V, dtype, sampled):
    check(make(B * N + V, B, N, V, dtype, sampled), B, N)


@pytest.mark.parametrize("sampled", [True, False])
def test_ragged_free_and_strided(sampled):
    """Sequences with no drafts, with none of their tokens, with more than N; rows of a wider array."""
    cnt = [1, 0, 4, 6, 2, 0]
    x = make(5, 6, 3, 260, "f32", sampled, cnt, pad=3)
    check(x, 6, 3)
    x["cnt"] = np.full(6, 4)
    x = make(6, 6, 3, 260, "bf16", sampled, pad=5)
    check(x, 6, 3, cu=False)


def test_all_stand_and_none():
    for u in (0.0, 1 - 2.0 ** -24):
        x = make(7, 4, 5, 600, "f32", True)
        x["u_accept"][:] = u
        if u == 0:
            x["draft_probs"][:] = x["target"].reshape(4, 6, 600)[:, :5]   # (p = q: all stand)
        check(x, 4, 5)


@pytest.mark.parametrize("u", [0.0, 0.25, 0.5, 1 - 2.0 ** -24])
def test_borders_of_the_sum(u):
    """Running sums that equal the threshold: the next token with weight is taken."""
    V = 1024
    x = make(8, 2, 1, V, "f32", False, [1, 1])
    x["target"][:] = 0
    x["target"][0, ::4] = 1.0 / 256
    x["target"][1, 700:] = 1.0 / 324
    x["u_sample"][:] = u
    check(x, 2, 1)


def test_odd_probabilities():
    """NaN, infinities, negatives, zeros everywhere, drafted tokens that are none."""
    x = make(9, 6, 2, 301, "f32", True)
    t, q = x["target"].view(6, 3, 301), x["draft_probs"]
    t[0, 0, 5], t[0, 0, 9], t[0, 0, 11] = float("nan"), -1.0, 0.9
    q[0, 0, 7] = float("nan")
    x["drafts"][0, 0] = 5
    t[1, 0] = 0.0                            # no weight at all
    q[2, 0] = t[2, 0] + 1e-3                 # p - q nowhere positive: p
    x["u_accept"][2, 0] = 1 - 2.0 ** -24
    x["drafts"][3, 0], x["drafts"][4, 0] = -1, 301
    t[5] = 0.0
    t[5, :, 300] = 3.0                       # above 1
    q[5] = 0.0
    tokens, n_out, _ = call(x, 6, 2)
    for b in range(6):
        with np.errstate(invalid="ignore"):
            want = kv.verify(np_(t)[b], x["drafts"][b].numpy(), np_(q)[b], x["u_accept"][b].numpy(), float(x["u_sample"][b]), 3)
        assert tokens[b].tolist() == want + [-1] * (3 - len(want)), b
    assert tokens[1, 0] == 300


def test_a_graph_replayed_with_other_numbers():
    lib = lib_()
    x, y = make(10, 4, 3, 5000, "f32", True), make(11, 4, 3, 5000, "f32", True)
    i32 = dict(dtype=torch.int32, device=DEV)
    st = {k: x[k].to(DEV).contiguous() for k in ("target", "drafts", "draft_probs", "u_accept", "u_sample")}
    tokens, n_out = torch.empty((4, 4), **i32), torch.empty(4, **i32)
    go = lambda: lib.ds4a_verify_drafts(st["target"], st["drafts"], st["u_accept"], st["u_sample"], tokens, n_out,  # noqa: E731
                                        draft_probs=st["draft_probs"])
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        go()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            go()
    for z in (x, y, x):
        for k in st:
            st[k].copy_(z[k])
        g.replay()
        torch.cuda.synchronize()
        want = call(z, 4, 3)
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(n_out.cpu().numpy(), want[1])
