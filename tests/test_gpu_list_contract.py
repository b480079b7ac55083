"""Decode over bf16 rows and any top-k list that the header allows: entries below 0 are
skipped wherever they stand, the first entry that is not visible ends the list whatever its
value, and rows may stand in any place. The fp64 answer and the bounds are those of
test_gpu_fp4_attention.py, of which the rows' values (exact in bf16) are taken; the partial
outputs of a cluster, bf16 here, are in its 3 u A."""
import numpy as np
import pytest
import torch

from test_gpu_fp4_attention import BASE, DEV, Case, few, late
from test_gpu_parity import lib_

pytestmark = pytest.mark.gpu


def plain_rows(c, paged):
    """The same case on a cache that holds its rows in bf16."""
    lib = lib_()
    cap = c.rows.shape[1]
    kw = dict(block_table=c.c.block_table, n_blocks=c.c.n_blocks) if paged else {}
    p = lib.LayerCache(ratio=4, head_dim=512, n_rot=64, batch=c.B, comp_cap=cap, dtype="bf16", base=BASE,
                       rope_max_pos=c.pos + c.T, index_dim=32, index_rot=32, device=DEV,
                       qat=lib.Q_ROTATED if c.rot_q else 0, **kw)
    rows = torch.tensor(c.rows, device=DEV).bfloat16().view(-1, 512)
    p.attn_comp_kv.view(-1, 512)[c.c.slots(cap).reshape(-1).long()] = rows
    p.raw_kv.copy_(c.ring)
    p.n_tokens = c.pos + c.T
    if c.c.c.seq_pos:
        p.set_seq_pos(c.c.seq_pos)
    c.c = p
    call = lib.CALL_ATTN_DECODE if c.T == 1 else lib.CALL_ATTN_PREFILL
    c.ws = lib.workspace(p.workspace_bytes(call, c.T, 64, c.k))
    return c


def ends_at(value):
    """The list ends halfway at an entry that is not visible; rows follow it."""
    def f(rng, row, vis):
        m = int((row >= 0).sum())
        end = {"first": vis, "near": vis + 3, "huge": 2 ** 31 - 1}[value]
        if m > 2:
            row[m // 2] = end
        elif m < len(row):
            row[m] = end
    return f


def ends_at_once(rng, row, vis):
    row[0] = 2 ** 31 - 1


def last_places(rng, row, vis):
    """Every row in the last places, behind as many places as are visible."""
    m = int((row >= 0).sum())
    row[:] = np.concatenate([row[m:], row[:m]])


def nothing(rng, row, vis):
    row[:] = -1


LISTS = [ends_at("first"), ends_at("near"), ends_at("huge"), ends_at_once, last_places, few, late, nothing]
NAMES = ["first", "near", "huge", "at_once", "last_places", "few", "late", "nothing"]


@pytest.mark.parametrize("cluster", [1, 2, 3, 0])
@pytest.mark.parametrize("lists", LISTS, ids=NAMES)
def test_decode_lists(lists, cluster):
    lib = lib_()
    paged = cluster == 2
    c = plain_rows(Case(4, 3, 1, 3000, 64, top_k=512, lists=lists, ragged=[3000, 1700, 900] if lists is late
                        else [3000, 13, 900], paged=paged, rot_q=cluster == 3), paged)
    lib.ds4a_set_decode_cluster(cluster)
    try:
        c.run()
        c.check()
    finally:
        lib.ds4a_set_decode_cluster(0)


@pytest.mark.parametrize("top_k", [1, 77, 513, 2048])
@pytest.mark.parametrize("lists", [ends_at("huge"), last_places], ids=["huge", "last_places"])
def test_list_lengths(lists, top_k):
    c = plain_rows(Case(4, 2, 1, 7000, 64, top_k=top_k, lists=lists, ragged=[7000, 260]), False)
    c.run()
    c.check()


def test_rows_behind_the_end_do_not_matter():
    """NaN rows listed behind the entry that ends the list."""
    c = plain_rows(Case(4, 2, 1, 4000, 64, top_k=300, lists=ends_at("huge")), False)
    c.run()
    c.check()
    want = c.out.clone()
    for b in range(2):
        row = c.topk_np[b, 0]
        end = int(np.argmax(row == 2 ** 31 - 1))
        assert 0 < end < 299 and (row[end + 1:] >= 0).all()
        c.c.attn_comp_kv[b, torch.tensor(row[end + 1:], device=DEV).long()] = float("nan")
    c.out.fill_(3)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)


def test_the_same_list_on_every_path():
    """Rows in 4 bits, rows in bf16, and a chunk of two tokens."""
    c = Case(4, 2, 1, 3000, 64, top_k=200, lists=ends_at("near"), rot_q=True)
    c.run()
    c.check()
    plain_rows(c, False)
    c.run()
    c.check()
    c = plain_rows(Case(4, 2, 2, 3000, 64, top_k=200, lists=ends_at("huge"), rot_q=True), False)
    c.run()
    c.check()
