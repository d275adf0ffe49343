"""Drafted trees over keys and values that are not finite: what reaches a row that sees them.

A score of -inf is a weight of 0, whichever part of the key it comes from and whoever computes it;
+inf and NaN make the row NaN.  Tolerances as in test_gpu_tree."""

from __future__ import annotations

import math

import numpy as np
import pytest
import tree_common as T
from gpu_common import assert_close, assert_lse_close
from test_gpu_tree import _lib    # noqa: F401  (the fixture builds the library)

pytestmark = pytest.mark.gpu

L = 48
# (workload, its changes, dims of the key that may hold infinities; MLA: of the rope part, which is no
# value, 512-543 multiplied on one CTA of the pair and 544-575 on the other)
KEYS = [
    ("tiny_gqa", dict(lengths=("fixed", 300), dcp_size=1), (0, 63)),
    ("tiny_gqa", dict(lengths=("fixed", 300), dcp_size=2, interleave=1, head_dim_qk=96, head_dim_v=96), (5,)),
    ("qwen_gqa", dict(batch=1, lengths=("fixed", 500), dcp_size=2, interleave=1), (127,)),
    ("mla_32", dict(batch=1, lengths=("fixed", 300), dcp_size=1), (512, 575)),
    ("mla_32", dict(batch=1, lengths=("fixed", 300), dcp_size=2, interleave=3, num_q_heads=16), (543, 544)),
    ("mla_32", dict(batch=1, lengths=("fixed", 300), dcp_size=1, num_q_heads=4), (512,)),       # CUDA-core kernel
]


def plant(inst, tokens, dims, value):
    """value at the dims of the keys of request 0's tokens; every query entry there becomes positive."""
    for d in dims:
        inst.q[..., d] = inst.q[..., d].abs().clamp(min=0.125)
    for t in tokens:
        blk, slot = T.cell(inst, 0, t)
        for d in dims:
            if inst.w.kind == "gqa":
                inst.kv_cache[0, blk, slot, :, d] = value
            else:
                inst.kv_cache[blk, slot, d] = value


# (factor 32, on the MLA queries: partial scores of 10 and more, sent with their residual)
@pytest.mark.parametrize("name,kw,dims,factor", [(*c, 1) for c in KEYS] + [(*c, 32) for c in KEYS if c[0] == "mla_32"])
def test_a_score_of_minus_infinity_is_a_weight_of_zero(name, kw, dims, factor):
    """Keys of the context and of nodes, of both halves of a 64-key tile; in one dim, and in all."""
    for some in [(d,) for d in dims] + [dims]:
        inst, mask, _ = T.tree_case(name, L, mask="random", **kw)
        w = inst.w
        inst.q *= factor
        S = int(inst.seq_lens[0])
        plant(inst, (0, 5, 37, S - L - 1, S - L + 1, S - L + 2, S - L + 33, S - 1), some, -math.inf)
        got, ref = T.run_tree(inst, mask), T.oracle_tree(inst, mask)
        # a probability is rounded to bf16 once, by at most 2^-8 of it, and they add up to 1: 2^-8 max |v| on an
        # output at the most (scores of 1.5 spread the weights over hundreds of keys, scores of 50 do not)
        values = inst.kv_cache[..., :w.head_dim_v] if name == "mla_32" else inst.kv_cache[1]
        tol = 2e-3 if factor == 1 else 2.0 ** -8 * float(values.abs().max())
        assert got["status"] == 0
        for key in ("partial_out", "out"):
            assert_close(got[key], ref[key], key, abs_tol=tol)
        for key in ("lse", "out_lse"):
            assert_lse_close(got[key], ref[key], key)


@pytest.mark.parametrize("name,kw,dims", KEYS)
def test_a_row_of_weights_of_zero_alone_is_empty(name, kw, dims):
    """No context, every key a node's with a score of -inf for the rows that see it."""
    kw = dict(kw, lengths=("fixed", L))
    inst, _, _ = T.tree_case(name, L, **kw)
    sees = np.eye(L, dtype=bool)[None]
    sees[0, :, 3] = True
    plant(inst, (7, 8, 40), dims[:1], -math.inf)
    sees[0, (7, 8, 40), 3] = False
    got = T.run_tree(inst, T.pack(sees))
    rows = [i for i in range(L) if i not in (7, 8, 40)]
    ref = T.oracle_rows(inst, T.pack(sees), rows)
    assert (got["out"][:, :, [7, 8, 40]] == 0).all() and (got["out_lse"][:, :, [7, 8, 40]] == -np.inf).all()
    assert_close(got["out"][:, :, rows], ref["out"][:, :, rows], "the other rows")
    assert_lse_close(got["out_lse"][:, :, rows], ref["out_lse"][:, :, rows], "lse of the other rows")


@pytest.mark.parametrize("name,kw,dims", [c for c in KEYS if len(c[2]) == 2])
def test_infinities_of_both_signs_in_one_key_make_its_rows_nan(name, kw, dims):
    _, mask, _ = T.tree_case(name, L, mask="random", **kw)
    sees = T.tro.unpack(mask, L)[0]
    for a, b in (dims, dims[::-1]):
        inst, _, _ = T.tree_case(name, L, mask="random", **kw)
        node = int(inst.seq_lens[0]) - L + 5
        for d in dims:
            inst.q[..., d] = inst.q[..., d].abs().clamp(min=0.125)
        ref = T.oracle_rows(inst, mask, np.nonzero(~sees[:, 5])[0])
        plant(inst, (node,), (a,), math.inf)
        plant(inst, (node,), (b,), -math.inf)
        got = T.run_tree(inst, mask)
        assert np.isnan(got["out"][:, :, sees[:, 5]]).all()
        assert_close(got["out"][:, :, ~sees[:, 5]], ref["out"][:, :, ~sees[:, 5]], "rows that do not see it")


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("name,kw", [(c[0], dict(c[1], dcp_size=1)) for c in KEYS if c[0] != "mla_32"])
def test_a_seen_value_that_is_not_finite_counts_however_small_its_weight(name, kw, value, first):
    """Node 2's score lies 300 below the others (or 300 above the context's, and node 40's 300 above
    it): its weight is 0 in fp32, its value is infinite in one dim."""
    inst, mask, _ = T.tree_case(name, L, mask="full", **kw)
    w = inst.w
    inst.q[..., 0] = 8.0
    base = int(inst.seq_lens[0]) - L
    keys = [(2, -300)] if not first else [(2, 300), (40, 600)]
    for node, score in keys:
        blk, slot = T.cell(inst, 0, base + node)
        inst.kv_cache[0, blk, slot, :, 0] = score / (8.0 * w.scale)
    sees = T.tro.unpack(mask, L)
    sees[:, ::2, 2] = False
    ref = T.oracle_tree(inst, T.pack(sees))
    blk, slot = T.cell(inst, 0, base + 2)
    inst.kv_cache[1, blk, slot, :, 7] = value
    got = T.run_tree(inst, T.pack(sees))
    hit = np.zeros(ref["out"].shape, dtype=bool)
    hit[:, :, 1::2, :, 7] = True
    want = np.full(1, value)
    assert np.array_equal(got["out"][hit], np.broadcast_to(want, got["out"][hit].shape), equal_nan=True)
    got["out"][hit] = ref["out"][hit] = 0
    assert_close(got["out"], ref["out"], "every other entry")
    assert_lse_close(got["out_lse"], ref["out_lse"], "out_lse")
