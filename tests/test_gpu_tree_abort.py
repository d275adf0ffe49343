"""Failure detection inside the drafted-tree kernels, without a GPU fault.

As for the causal kernels: a test-only hook shortens every bounded wait to a few
milliseconds and makes the TMA producer skip one key tile.  The waits on it run
out; the kernel records DCP_ERR_TIMEOUT, leaves zeros and -inf (a CTA that takes
units in turn: for its later units too), drains its copies and MMAs and frees its
tensor memory.  An ordinary launch right after matches the oracle."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import tree_common as T
from gpu_common import assert_close, assert_lse_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooks():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from context_decode_attention_paged_gb300 import build
    build.build()
    from context_decode_attention_paged_gb300 import binding as dcp
    lib = dcp.raw_lib()
    lib.dcp_testing_set_hooks.restype = None
    lib.dcp_testing_set_hooks.argtypes = [ctypes.c_ulonglong, ctypes.c_int32]
    yield lib.dcp_testing_set_hooks
    lib.dcp_testing_set_hooks(0, -1)


CASES = [
    # 128 rows: the streams take the tiles in turn (the second one's first tile never comes)
    ("qwen_gqa", 4, dict(batch=1, num_q_heads=16, num_kv_heads=1, lengths=("fixed", 700), dcp_size=1)),
    # 256 rows: both wait for the tile
    ("qwen_gqa", 16, dict(batch=1, num_q_heads=16, num_kv_heads=1, lengths=("fixed", 700), dcp_size=1)),
    ("tiny_gqa", 3, dict(batch=2, lengths=("fixed", 700), dcp_size=1)),
    # more units than SMs: a CTA's first unit runs out, its others are empty
    ("tiny_gqa", 2, dict(batch=100, lengths=("uniform", 300, 400), dcp_size=1)),
    ("mla_32", 3, dict(batch=1, lengths=("fixed", 300), dcp_size=1)),
    ("mla_32", 9, dict(batch=1, num_q_heads=32, lengths=("fixed", 300), dcp_size=1)),
]


@pytest.mark.parametrize("name,L,kw", CASES)
def test_wait_runs_out_and_the_units_unwind(hooks, name, L, kw):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, mask, _ = T.tree_case(name, L, **kw)
    hooks(5_000_000, 1)                     # 5 ms waits; key tile 1 is never loaded
    try:
        got = T.run_tree(inst, mask)
    finally:
        hooks(0, -1)
    assert got["status"] == dcp.DCP_ERR_TIMEOUT, dcp.status_string(got["status"])
    assert (got["lse"] == -np.inf).all()
    assert (got["partial_out"] == 0).all()
    assert (got["out"] == 0).all()
    got, ref = T.run_tree(inst, mask), T.oracle_tree(inst, mask)
    assert got["status"] == dcp.DCP_OK
    assert_close(got["out"], ref["out"], "out")
    assert_lse_close(got["out_lse"], ref["out_lse"], "out_lse")
