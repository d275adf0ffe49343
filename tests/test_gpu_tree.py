"""GPU parity of the drafted-tree attention: every kernel it runs on, against the oracle.

Tolerances are those of the library's attention (fp32 sums over bf16 inputs, probabilities
rounded for the value product): 2e-3 + 1e-2 |ref| on outputs, 1e-3 on LSE."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import helpers as H
import tree_common as T
from gpu_common import assert_close, assert_lse_close
from oracle import dcp_oracle as orc
from oracle import tree_oracle as tro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from context_decode_attention_paged_gb300 import build
    build.build()


def check(inst, mask, q_lens=None, got=None):
    from context_decode_attention_paged_gb300 import binding as dcp
    got = got or T.run_tree(inst, mask, q_lens)
    assert got["status"] == dcp.DCP_OK, dcp.status_string(got["status"])
    ref = T.oracle_tree(inst, mask, q_lens)
    for key in ("partial_out", "out"):
        assert_close(got[key], ref[key], key)
    for key in ("lse", "out_lse"):
        assert_lse_close(got[key], ref[key], key)
    return got


# (workload, nodes, its changes, tree options)
CASES = [
    ("tiny_gqa", 8, {}, {}),
    ("tiny_gqa", 1, {}, {}),                                                       # a single token
    ("tiny_gqa", 1, dict(lengths=("fixed", 1)), {}),                               # which is the whole request
    ("tiny_gqa", 5, dict(lengths=("fixed", 5), batch=2), dict(mask="random")),     # no context at all
    ("tiny_gqa", 33, dict(batch=3, lengths=("uniform", 33, 700), dcp_size=4, interleave=3), {}),
    ("tiny_gqa", 40, dict(batch=2, lengths=("uniform", 200, 300), dcp_size=8, interleave=1, num_q_heads=16), {}),
    ("tiny_gqa", 64, dict(batch=2, lengths=("uniform", 64, 1100), dcp_size=2, interleave=64), dict(shared=True)),
    ("tiny_gqa", 7, dict(batch=2, lengths=("uniform", 20, 400)), dict(mask="empty")),
    ("tiny_gqa", 7, dict(batch=2, lengths=("uniform", 20, 400)), dict(mask="full")),
    ("tiny_gqa", 256, dict(batch=1, lengths=("fixed", 900), dcp_size=4), dict(mask="random")),
    ("tiny_gqa", 9, dict(batch=4, lengths=("uniform", 30, 500), dcp_size=2, interleave=1), dict(q_lens=[9, 0, 1, 8])),
    ("tiny_gqa", 20, dict(batch=2, num_q_heads=10, num_kv_heads=5, lengths=("uniform", 100, 700), dcp_size=1), {}),
    ("tiny_gqa", 6, dict(batch=2, num_q_heads=24, num_kv_heads=1, lengths=("uniform", 100, 1500)), {}),
    ("tiny_gqa", 11, dict(head_dim_qk=96, head_dim_v=96, lengths=("fixed", 500)), {}),        # CUDA-core kernel
    ("tiny_gqa", 11, dict(block_size=48, lengths=("fixed", 700), interleave=48), dict(mask="random")),
    ("qwen_gqa", 3, dict(batch=2, lengths=("uniform", 300, 2000)), {}),
    ("qwen_gqa", 4, dict(batch=2, lengths=("uniform", 300, 2000)), {}),
    ("qwen_gqa", 8, dict(batch=2, lengths=("uniform", 100, 1500), dcp_size=2), {}),           # 128 rows a KV head
    ("qwen_gqa", 9, dict(batch=2, lengths=("uniform", 100, 1500), dcp_size=2), {}),
    ("qwen_gqa", 16, dict(batch=2, lengths=("uniform", 300, 1500), dcp_size=2, interleave=1), dict(mask="random")),
    ("qwen_gqa", 17, dict(batch=1, lengths=("fixed", 1153), dcp_size=2, interleave=1), {}),
    ("qwen_gqa", 64, dict(batch=2, lengths=("uniform", 100, 1500), dcp_size=2), dict(q_lens=[64, 13])),
    ("qwen_gqa", 40, dict(batch=1, lengths=("fixed", 40), dcp_size=2), {}),
    ("qwen_gqa", 24, dict(batch=1, lengths=("fixed", 20000), dcp_size=2), {}),                # KV splits
    ("qwen_gqa", 2, dict(batch=1, lengths=("fixed", 20000), dcp_size=1), {}),
    ("qwen_gqa", 12, dict(batch=2, block_size=8, lengths=("uniform", 300, 1300), dcp_size=2), {}),
    ("qwen_gqa", 12, dict(batch=2, block_size=16, lengths=("uniform", 300, 1300), dcp_size=4, interleave=3), {}),
    ("qwen_gqa", 12, dict(batch=2, block_size=64, lengths=("uniform", 300, 1300), dcp_size=2, interleave=64), {}),
    ("qwen_gqa", 12, dict(batch=2, block_size=256, lengths=("uniform", 300, 2300), dcp_size=2, interleave=256), {}),
    ("mla_32", 1, dict(batch=2, lengths=("uniform", 100, 900)), {}),
    ("mla_32", 4, dict(batch=2, lengths=("uniform", 100, 900), dcp_size=2, interleave=1), {}),
    ("mla_32", 9, dict(batch=3, lengths=("uniform", 30, 700), dcp_size=2, interleave=3), dict(q_lens=[9, 0, 4])),
    ("mla_32", 6, dict(batch=1, lengths=("fixed", 6), dcp_size=1), dict(mask="random")),
    ("mla_32", 5, dict(batch=1, lengths=("fixed", 300), dcp_size=1), dict(mask="empty")),
    ("mla_32", 70, dict(batch=1, num_q_heads=16, lengths=("fixed", 600), dcp_size=2), {}),
    ("mla_32", 11, dict(batch=2, num_q_heads=32, lengths=("uniform", 30, 600), dcp_size=2), {}),
    ("mla_32", 3, dict(batch=2, num_q_heads=48, lengths=("uniform", 30, 600), dcp_size=2), {}),
    ("mla_32", 20, dict(batch=2, num_q_heads=16, lengths=("uniform", 30, 600), dcp_size=2, interleave=1),
     dict(mask="random", q_lens=[20, 9])),                                          # eight nodes a unit, partly there
    ("mla_32", 9, dict(batch=2, num_q_heads=64, lengths=("uniform", 9, 600), dcp_size=4, interleave=3),
     dict(mask="random")),                                                          # two nodes a unit
    ("mla_32", 7, dict(batch=3, num_q_heads=20, lengths=("uniform", 30, 600), dcp_size=2), {}),   # not a multiple of 8
    ("mla_32", 40, dict(batch=1, num_q_heads=16, lengths=("fixed", 20000), dcp_size=1), {}),      # KV splits
    ("mla_32", 5, dict(batch=2, num_q_heads=4, lengths=("uniform", 30, 300), dcp_size=2), {}),     # CUDA-core kernel
    ("mla_32", 7, dict(batch=2, block_size=16, lengths=("uniform", 100, 700), dcp_size=2, interleave=16), {}),
    ("mla_32", 7, dict(batch=2, block_size=64, lengths=("uniform", 100, 700), dcp_size=2, interleave=1), {}),
    ("mla_mtp", 8, dict(lengths=("fixed", 30000)), {}),                                        # KV splits
]


@pytest.mark.parametrize("name,L,kw,opt", CASES)
def test_tree_matches_the_oracle(name, L, kw, opt):
    check(*T.tree_case(name, L, **kw, **opt))


@pytest.mark.parametrize("name,L,kw", [
    ("tiny_gqa", 5, dict(batch=2, lengths=("uniform", 60, 300))),
    ("qwen_gqa", 12, dict(batch=1, lengths=("fixed", 700), dcp_size=2)),
    ("mla_32", 4, dict(batch=1, lengths=("fixed", 400), dcp_size=2)),
])
def test_a_chain_is_the_causal_query(name, L, kw):
    """A tree without branches is dcp_decode_attn's causal query of the same length."""
    from gpu_common import run_gpu
    inst, _, _ = T.tree_case(name, L, **kw)
    got = T.run_tree(inst, T.pack(np.tril(np.ones((1, L, L), dtype=bool))))
    want = run_gpu(inst)
    assert_close(got["out"], want["out"], "out")
    assert_lse_close(got["out_lse"], want["out_lse"], "out_lse")


SPECIAL = [
    ("tiny_gqa", 9, dict(batch=1, lengths=("fixed", 300), dcp_size=2, interleave=1)),
    ("tiny_gqa", 9, dict(batch=1, head_dim_qk=96, head_dim_v=96, lengths=("fixed", 300))),
    ("qwen_gqa", 6, dict(batch=1, lengths=("fixed", 500), dcp_size=2, interleave=1)),
    ("qwen_gqa", 20, dict(batch=1, lengths=("fixed", 500), dcp_size=1)),
    ("mla_32", 6, dict(batch=1, lengths=("fixed", 300), dcp_size=2, interleave=1)),
    ("mla_32", 12, dict(batch=1, num_q_heads=32, lengths=("fixed", 300), dcp_size=1)),
    ("mla_32", 12, dict(batch=1, num_q_heads=16, lengths=("fixed", 300), dcp_size=2, interleave=1)),
]


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name,L,kw", SPECIAL)
def test_hidden_nodes_may_hold_anything(name, L, kw, value):
    """Node 2 holds NaN or infinities in its key and value: the rows that do not see it are what
    they are without it, the rows that see it are not finite; stale slots hold them too."""
    inst, _, _ = T.tree_case(name, L, **kw)
    sees = np.tril(np.ones((1, L, L), dtype=bool))
    sees[:, :, 2] = False
    sees[:, 2, 2] = sees[:, L - 1, 2] = True
    H.poison_unused_slots(inst)
    mask = T.pack(sees)
    ref = T.oracle_tree(inst, mask)
    blk, slot = T.cell(inst, 0, int(inst.seq_lens[0]) - L + 2)
    if inst.w.kind == "gqa":
        inst.kv_cache[:, blk, slot] = value
    else:
        inst.kv_cache[blk, slot] = value
    got = T.run_tree(inst, mask)
    rows = [i for i in range(L) if i not in (2, L - 1)]
    assert_close(got["out"][:, :, rows], ref["out"][:, :, rows], "rows that do not see it")
    assert_lse_close(got["out_lse"][:, :, rows], ref["out_lse"][:, :, rows], "lse of rows that do not see it")
    assert not np.isfinite(got["out"][:, :, [2, L - 1]]).any()


@pytest.mark.parametrize("name,L,kw", [c for c in SPECIAL if c[0] != "mla_32"])
def test_a_seen_value_that_is_not_finite_reaches_its_dims_alone(name, L, kw):
    """An infinite value entry of a seen node makes that output entry infinite, and no other."""
    inst, _, _ = T.tree_case(name, L, **kw)
    sees = np.tril(np.ones((1, L, L), dtype=bool))
    sees[:, 3:, 2] = False
    mask = T.pack(sees)
    ref = T.oracle_tree(inst, mask)
    blk, slot = T.cell(inst, 0, int(inst.seq_lens[0]) - L + 2)
    inst.kv_cache[1, blk, slot, :, 5] = math.inf
    got = T.run_tree(inst, mask)
    hit = np.zeros(ref["out"].shape, dtype=bool)
    hit[:, :, 2, :, 5] = True
    assert (got["out"][hit] == math.inf).all()
    want = ref["out"].copy()
    want[hit] = 0
    got["out"][hit] = 0
    assert_close(got["out"], want, "every other entry")


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dim", [0, 5, -1])
@pytest.mark.parametrize("name,L,kw", SPECIAL)
def test_a_seen_key_that_is_not_finite_makes_its_rows_nan(name, L, kw, dim, value):
    """One entry of node 2's key (MLA: of its rope part, which is no value): the rows that see it
    are NaN (an infinite score against itself), the others are what they are without it."""
    inst, _, _ = T.tree_case(name, L, **kw)
    sees = np.tril(np.ones((1, L, L), dtype=bool))
    sees[:, 3:, 2] = False
    mask = T.pack(sees)
    ref = T.oracle_tree(inst, mask)
    blk, slot = T.cell(inst, 0, int(inst.seq_lens[0]) - L + 2)
    if inst.w.kind == "gqa":
        inst.q[:, 2, :, dim] = inst.q[:, 2, :, dim].abs() + 0.1          # +inf scores
        inst.kv_cache[0, blk, slot, :, dim] = value
    else:
        d = 575 if dim == -1 else 512 + 32 * (dim > 0) + dim
        inst.q[:, 2, :, d] = inst.q[:, 2, :, d].abs() + 0.1
        inst.kv_cache[blk, slot, d] = value
    rows = [i for i in range(L) if i != 2]
    got = T.run_tree(inst, mask)
    assert np.isnan(got["out"][:, :, 2]).all()
    assert_close(got["out"][:, :, rows], ref["out"][:, :, rows], "rows that do not see it")


def test_stress_inputs_hold_the_bar():
    """Softmaxes dominated by a few nearly cancelling keys, and growing scores."""
    for name, L, kw in (("qwen_gqa", 4, dict(batch=2, lengths=("uniform", 700, 1500), dcp_size=2)),
                        ("qwen_gqa", 20, dict(batch=1, lengths=("fixed", 1500), dcp_size=2)),
                        ("mla_32", 3, dict(batch=2, lengths=("uniform", 700, 1500), dcp_size=2))):
        inst, mask, _ = T.tree_case(name, L, **kw)
        if name == "mla_32" or L * 16 <= 128:
            check(H.plant_dominant_keys(inst), mask)
        inst, mask, _ = T.tree_case(name, L, **kw)
        dims = slice(None) if name == "qwen_gqa" else slice(512, None)
        check(H.scale_keys_by_position(inst, lambda x: 0.2 + 6 * x, key_dims=dims), mask)


@pytest.mark.parametrize("name,L,kw", [
    ("tiny_gqa", 5, dict(batch=2, lengths=("fixed", 64))),
    ("tiny_gqa", 5, dict(batch=2, head_dim_qk=96, head_dim_v=96, lengths=("fixed", 64))),
    ("qwen_gqa", 20, dict(batch=2, lengths=("fixed", 300), dcp_size=2)),
    ("mla_32", 5, dict(batch=2, lengths=("fixed", 300), dcp_size=2)),
])
@pytest.mark.parametrize("bad", ["short", "count", "negative", "table", "block"])
def test_bad_requests_are_skipped_and_reported(name, L, kw, bad):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, mask, _ = T.tree_case(name, L, **kw)
    ref = T.oracle_tree(inst, mask)
    ql = torch.tensor([L, L], dtype=torch.int32)
    if bad == "short":
        inst.seq_lens[0] = L - 1
    elif bad == "count":
        ql[0] = L + 1
    elif bad == "negative":
        ql[0] = -2
    elif bad == "table":
        inst.seq_lens[0] = 10 ** 6
    else:
        pool = inst.kv_cache.shape[1] if inst.w.kind == "gqa" else inst.kv_cache.shape[0]
        inst.block_tables[:, 0] = pool
    got = T.run_tree(inst, mask, ql)
    assert got["status"] == dcp.DCP_ERR_BOUNDS
    if bad != "table":                    # a short table reads what it has; the rest are zero
        assert (got["out"][:, 0] == 0).all() and (got["out_lse"][:, 0] == -np.inf).all()
    assert_close(got["out"][:, 1], ref["out"][:, 1], "the other request")


def test_rows_behind_a_request_are_zero_and_empty():
    inst, mask, ql = T.tree_case("qwen_gqa", 8, batch=3, lengths=("uniform", 60, 300), dcp_size=2, q_lens=[0, 8, 3])
    got = T.run_tree(inst, mask, ql)
    assert (got["partial_out"][:, 0] == 0).all() and (got["lse"][:, 0] == -np.inf).all()
    assert (got["out"][:, 2, 3:] == 0).all() and (got["out_lse"][:, 2, 3:] == -np.inf).all()


def test_two_streams_and_a_graph_replay_agree():
    """The same call on two streams at once (a workspace each), and captured and replayed after its
    inputs changed in place."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, mask, _ = T.tree_case("qwen_gqa", 6, batch=1, lengths=("fixed", 9000), dcp_size=2)
    w = inst.w
    ref = T.run_tree(inst, mask)
    dev = torch.device("cuda:0")
    q, kv, bt, sl = (t.to(dev) for t in (inst.q, inst.kv_cache, inst.block_tables, inst.seq_lens))
    m = torch.as_tensor(mask).to(dev)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [dcp.dcp_tree_attn(w.kind, q, kv, bt, sl, m, w.dcp_size, w.interleave, w.scale, w.head_dim_v, stream=s)
           for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for po, lse in got:
        assert np.array_equal(po.cpu().numpy(), ref["partial_out"]) and np.array_equal(lse.cpu().numpy(), ref["lse"])
    desc = dcp.desc_from_tensors(w.kind, q, kv, bt, w.head_dim_v)
    ws = torch.empty((max(1, dcp.dcp_tree_attn_workspace_size(desc, w.dcp_size)),), dtype=torch.uint8, device=dev)
    po, lse = torch.empty_like(got[0][0]), torch.empty_like(got[0][1])
    graph = torch.cuda.CUDAGraph()
    keep = q.clone()
    q.zero_()
    with torch.cuda.graph(graph):
        dcp.dcp_tree_attn(w.kind, q, kv, bt, sl, m, w.dcp_size, w.interleave, w.scale, w.head_dim_v, partial_out=po,
                          lse=lse, workspace=ws)
    q.copy_(keep)
    for _ in range(2):
        po.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(po.cpu().numpy(), ref["partial_out"]) and np.array_equal(lse.cpu().numpy(), ref["lse"])


@pytest.mark.parametrize("name,kw,rope", [
    ("qwen_gqa", dict(batch=2, lengths=("uniform", 200, 600), dcp_size=2, interleave=1), dict(rot_dim=128, base=1e6)),
    ("mla_32", dict(batch=2, num_q_heads=16, lengths=("uniform", 200, 600), dcp_size=2),
     dict(rot_dim=64, rot_offset=512, layout="interleaved")),
])
def test_a_verify_step_end_to_end(name, kw, rope):
    """Append a tree, attend, merge, commit one path, and decode one more token: the last step
    equals a plain decode over a cache that was written without any tree."""
    from context_decode_attention_paged_gb300 import binding as dcp
    L = 7
    w = H.small(name, q_len=L, **kw)
    inst = H.build_instance(w)
    parents = [-1, 0, 0, 1, 2, 4, 3]
    path = [0, 2, 4, 5]
    mask, depth = dcp.tree_mask(parents)
    dev = torch.device("cuda:0")
    kv, bt, sl = inst.kv_cache.to(dev), inst.block_tables.to(dev), inst.seq_lens.to(dev)
    table = dcp.dcp_rope_table(**rope)
    k, v, q = T.append_inputs(w, L, 9)
    _, qr = dcp.dcp_kv_cache_append(w.kind, T.to_gpu(k), T.to_gpu(v), kv, bt, sl, w.dcp_size, w.interleave, table,
                                    q=T.to_gpu(q), pos_offsets=depth.view(1, L).to(dev))
    po, lse = dcp.dcp_tree_attn(w.kind, qr, kv, bt, sl, mask.view(1, L, 1).to(dev), w.dcp_size, w.interleave, w.scale,
                                w.head_dim_v)
    out, out_lse = dcp.dcp_merge(po, lse, w.dcp_size)
    step = H.wl.Instance(w, inst.seq_lens, qr.cpu(), kv.cpu(), inst.block_tables, None)
    ref = T.oracle_tree(step, mask.view(1, L, 1).numpy())
    assert_close(out.float().cpu().numpy(), ref["out"], "verify")
    assert_lse_close(out_lse.cpu().numpy(), ref["out_lse"], "verify lse")
    take = torch.full((w.batch,), len(path), dtype=torch.int32, device=dev)
    acc = torch.tensor([path] * w.batch, dtype=torch.int32, device=dev)
    lens = dcp.dcp_kv_cache_commit(w.kind, kv, bt, sl, L, acc, take, w.dcp_size, w.interleave)
    # the same tokens appended without a tree: the path's rows in order
    kv2 = inst.kv_cache.to(dev)
    pick = lambda t: None if t is None else t[:, path].contiguous().to(dev)   # noqa: E731
    dcp.dcp_kv_cache_append(w.kind, pick(k), pick(v), kv2, bt, lens, w.dcp_size, w.interleave, table)
    q1 = torch.randn((w.batch, 1, w.num_q_heads, w.head_dim_qk), generator=torch.Generator().manual_seed(2)).to(
        torch.bfloat16).to(dev)
    a = dcp.dcp_decode_attn(w.kind, q1, kv, bt, lens, w.dcp_size, w.interleave, w.scale, 1, w.head_dim_v)
    b = dcp.dcp_decode_attn(w.kind, q1, kv2, bt, lens, w.dcp_size, w.interleave, w.scale, 1, w.head_dim_v)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK
