"""Requests without nodes in a drafted-tree call (the padding of a captured batch): nothing of them is
read but their lengths, their rows are 0 and -inf, and no error is reported."""

from __future__ import annotations

import numpy as np
import pytest

import tree_common as T
from gpu_common import assert_close, assert_lse_close
from test_gpu_tree import _lib    # noqa: F401  (the fixture builds the library)

pytestmark = pytest.mark.gpu

CASES = [
    ("tiny_gqa", 5, dict(lengths=("fixed", 200))),
    ("tiny_gqa", 5, dict(lengths=("fixed", 200), head_dim_qk=96, head_dim_v=96)),        # CUDA-core kernel
    ("qwen_gqa", 20, dict(lengths=("fixed", 300), dcp_size=2)),
    ("mla_32", 5, dict(lengths=("fixed", 300), dcp_size=2)),
    ("mla_32", 5, dict(lengths=("fixed", 300), dcp_size=2, num_q_heads=16)),
    ("mla_32", 2, dict(lengths=("fixed", 100), dcp_size=2, num_q_heads=4)),              # CUDA-core kernel
]


@pytest.mark.parametrize("name,L,kw", CASES)
@pytest.mark.parametrize("block", [-1, 1 << 30])
@pytest.mark.parametrize("length", [200, 0])
def test_the_table_of_a_request_without_nodes_is_not_read(name, L, kw, block, length):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, mask, ql = T.tree_case(name, L, batch=3, q_lens=[L, 0, 1], **kw)
    ref = T.oracle_tree(inst, mask, ql)
    inst.block_tables[:, 1] = block
    inst.seq_lens[1] = min(length, int(inst.seq_lens[1]))
    got = T.run_tree(inst, mask, ql)
    assert got["status"] == dcp.DCP_OK
    assert (got["partial_out"][:, 1] == 0).all() and (got["lse"][:, 1] == -np.inf).all()
    for b in (0, 2):
        assert_close(got["partial_out"][:, b], ref["partial_out"][:, b], "partial_out")
        assert_lse_close(got["lse"][:, b], ref["lse"][:, b], "lse")


@pytest.mark.parametrize("name,L,kw", CASES)
def test_a_bad_block_empties_the_request_in_its_shard_alone(name, L, kw):
    """The last block of request 1 in shard 0: all its rows there, whichever unit holds the block."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, mask, _ = T.tree_case(name, L, batch=3, **kw)
    ref = T.oracle_tree(inst, mask)
    last = int(inst.local_num_blocks[0, 1]) - 1
    inst.block_tables[0, 1, last] = 1 << 30
    got = T.run_tree(inst, mask)
    assert got["status"] == dcp.DCP_ERR_BOUNDS
    assert (got["partial_out"][0, 1] == 0).all() and (got["lse"][0, 1] == -np.inf).all()
    ref["partial_out"][0, 1], ref["lse"][0, 1] = 0.0, -np.inf
    assert_close(got["partial_out"], ref["partial_out"], "partial_out")
    assert_lse_close(got["lse"], ref["lse"], "lse")


@pytest.mark.parametrize("name,L,kw", CASES + [("mla_32", 11, dict(lengths=("fixed", 400), dcp_size=1, num_q_heads=20))])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 3e38])
def test_query_rows_behind_a_request_may_hold_anything(name, L, kw, value):
    """They share MMA tiles and messages with the rows that are there."""
    from context_decode_attention_paged_gb300 import binding as dcp
    n = [L, max(1, L // 2), 1]
    inst, mask, ql = T.tree_case(name, L, batch=3, q_lens=n, **kw)
    ref = T.oracle_tree(inst, mask, ql)
    for b in range(3):
        inst.q[b, n[b]:] = value
    got = T.run_tree(inst, mask, ql)
    assert got["status"] == dcp.DCP_OK
    for key in ("partial_out", "out"):
        assert_close(got[key], ref[key], key)
    for key in ("lse", "out_lse"):
        assert_lse_close(got[key], ref[key], key)
