"""Hand-overs between the units of a drafted-tree launch, and rows that see nothing for a while.

The GQA kernel's CTAs take units in turn.  With 128 rows or fewer its two streams share a
unit's key tiles, and a unit of one tile leaves the second stream without a step: it goes on
to the next unit while the first one is still at work.  Tolerances as in test_gpu_tree."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import helpers as H
import tree_common as T
from test_gpu_tree import _lib, check    # noqa: F401  (the fixture builds the library)

pytestmark = pytest.mark.gpu


# Requests of 3,050 tokens dealt 1,000 at a time: three shards of 1,000 keys (eight tiles) and one
# of 50 (a single step).  With more units than two waves of SMs there are no KV splits, and the order
# back and forth gives a CTA short and long units by turns.
ONE_STEP = [
    ("tiny_gqa", 3, dict(batch=60)),                                                     # 12 rows a KV head
    ("tiny_gqa", 80, dict(batch=60, num_q_heads=8, num_kv_heads=2)),                     # 320 rows: three blocks of 128
    ("qwen_gqa", 1, dict(batch=24)),
    ("qwen_gqa", 8, dict(batch=24)),                                                     # 128 rows, all of them there
]


@pytest.mark.parametrize("name,L,kw", ONE_STEP)
@pytest.mark.parametrize("length", [3050, 3120, 3000 + 128])
def test_units_of_one_step_between_long_ones(name, L, kw, length):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, mask, _ = T.tree_case(name, L, dcp_size=4, interleave=1000, lengths=("fixed", length), **kw)
    w = inst.w
    dev = torch.device("cuda:0")
    args = [t.to(dev) for t in (inst.q, inst.kv_cache, inst.block_tables, inst.seq_lens)]
    m = torch.as_tensor(mask).to(dev)
    first = None
    for _ in range(10):
        po, lse = dcp.dcp_tree_attn(w.kind, *args, m, w.dcp_size, w.interleave, w.scale, w.head_dim_v)
        if first is None:
            first = po, lse
        assert torch.equal(po, first[0]) and torch.equal(lse, first[1])
    got = {"status": dcp.dcp_get_last_device_status(), "partial_out": first[0].cpu().numpy(), "lse": first[1].cpu().numpy()}
    out, out_lse = dcp.dcp_merge(*first, w.dcp_size)
    got.update(out=out.float().cpu().numpy(), out_lse=out_lse.cpu().numpy())
    # the oracle walks requests one by one: three of them stand for the rest
    few = [0, w.batch // 2, w.batch - 1]
    part = H.wl.Instance(w.with_(batch=len(few)), inst.seq_lens[few], inst.q[few], inst.kv_cache,
                      inst.block_tables[:, few], inst.local_num_blocks[:, few])
    for key in ("partial_out", "lse", "out", "out_lse"):
        got[key] = np.ascontiguousarray(got[key][:, few])
    check(part, np.ascontiguousarray(mask[few]), got=got)


# ---------------------------------------------------------------------------
# MLA: rows of several nodes in one warp, tiles that only some of them see anything of
# ---------------------------------------------------------------------------

def mla_nodes(L, heads, sees, **kw):
    inst, _, _ = T.tree_case("mla_32", L, batch=1, num_q_heads=heads, **kw)
    return inst, T.pack(sees)


@pytest.mark.parametrize("heads", [16, 24, 40, 48, 56, 64, 128])
def test_a_row_waits_tiles_for_its_first_key(heads):
    """256 nodes without context, four tiles: node 200 sees a key of the second tile, its neighbours
    in the warp none before the fourth."""
    L = 256
    sees = np.eye(L, dtype=bool)[None]
    sees[0, 200, 70] = True
    check(*mla_nodes(L, heads, sees, lengths=("fixed", L), dcp_size=1))


@pytest.mark.parametrize("heads", [16, 24, 40, 48, 56])
@pytest.mark.parametrize("dcp_size,interleave", [(1, 128), (2, 1)])
def test_rows_that_see_nothing_are_zero_among_rows_that_do(heads, dcp_size, interleave):
    """Two tiles of node keys a shard; odd nodes see nothing at all."""
    L = 128 * dcp_size
    sees = np.eye(L, dtype=bool)[None]
    sees[0, 1::2] = False
    inst, mask = mla_nodes(L, heads, sees, lengths=("fixed", L), dcp_size=dcp_size, interleave=interleave)
    got = check(inst, mask)
    assert (got["partial_out"][:, :, 1::2] == 0).all() and (got["lse"][:, :, 1::2] == -np.inf).all()


@pytest.mark.parametrize("L,length", [(256, 560), (200, 520), (256, 576)])
def test_sparse_masks_over_splits_that_start_among_the_nodes(L, length):
    """Two KV splits of 320 keys: the second starts with a node."""
    from context_decode_attention_paged_gb300 import binding as dcp
    sees = np.random.default_rng(5).random((1, L, L)) < 0.01
    inst, mask = mla_nodes(L, 16, sees, lengths=("fixed", length), dcp_size=1)
    desc = dcp.desc_from_tensors("mla", inst.q, inst.kv_cache, inst.block_tables, 512)
    rows = L * 16
    assert dcp.dcp_tree_attn_workspace_size(desc, 1) == rows * 2 * 512 * 4 + rows * 2 * 4
    check(inst, mask)
