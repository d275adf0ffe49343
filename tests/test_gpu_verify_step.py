"""Calls around the verify step that the element-wise tests do not make: large batches, units split
against a last wave, block ids that are bad early or late in a table, and a whole step captured in
a graph."""

import numpy as np
import pytest
import torch

import helpers as H
import tree_common as T
from gpu_common import assert_close, assert_lse_close, run_gpu
from test_gpu_tree import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,L,kw,q_lens", [
    ("mla_32", 3, dict(batch=130, num_q_heads=16, lengths=("uniform", 3, 90), dcp_size=2), "ragged"),
    ("mla_32", 2, dict(batch=129, num_q_heads=64, lengths=("uniform", 2, 70), dcp_size=1), None),
    ("qwen_gqa", 3, dict(batch=130, lengths=("uniform", 3, 90), dcp_size=2), "ragged"),
    ("tiny_gqa", 40, dict(batch=200, lengths=("uniform", 40, 90), dcp_size=2), "ragged"),
])
def test_more_requests_than_a_kernel_ranks_itself(name, L, kw, q_lens):
    """Beyond 128 requests the MLA kernel's order comes from a pre-pass and the GQA kernel takes the
    units as they are."""
    if q_lens:
        q_lens = np.random.default_rng(8).integers(0, L + 1, kw["batch"]).tolist()
    check(*T.tree_case(name, L, q_lens=q_lens, **kw))


def test_units_that_fill_a_little_more_than_two_waves_are_split():
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, mask, _ = T.tree_case("mla_32", 160, batch=1, lengths=("fixed", 8000), dcp_size=1)
    w = inst.w
    desc = dcp.DcpAttnDesc(dcp.KINDS[w.kind], w.batch, 160, w.num_q_heads, 1, w.head_dim_qk, w.head_dim_v, w.block_size,
                           inst.kv_cache.shape[0], inst.block_tables.shape[2])
    assert dcp.dcp_tree_attn_launches(desc, 1) == 2                     # the attention and the join
    rows = [0, 1, 77, 158, 159]
    got = T.run_tree(inst, mask)
    assert got["status"] == dcp.DCP_OK
    ref = T.oracle_rows(inst, mask, rows)
    for key in ("out", "out_lse"):
        close = assert_close if key == "out" else assert_lse_close
        close(got[key][:, :, rows], ref[key][:, :, rows], key)


@pytest.mark.parametrize("at", [0, 1, 9, -1])
@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("name,kw", [
    ("mla_32", dict(block_size=128)), ("mla_32", dict(block_size=64)), ("mla_32", dict(block_size=16, interleave=16)),
    ("qwen_gqa", dict(block_size=64)), ("tiny_gqa", dict()),
])
def test_a_bad_block_anywhere_skips_its_request(name, kw, tree, at):
    """Loads of the first tiles may be out when the scan of the table finds the bad entry."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, mask, _ = T.tree_case(name, 4, batch=2, lengths=("fixed", 1700), dcp_size=1, **kw)
    run = (lambda: T.run_tree(inst, mask)) if tree else (lambda: run_gpu(inst))
    ref = run()
    assert ref["status"] == dcp.DCP_OK
    used = (1700 - (0 if tree else 3) + inst.w.block_size - 1) // inst.w.block_size
    inst.block_tables[0, 0, used - 1 if at < 0 else at] = inst.kv_cache.shape[1 if inst.w.kind == "gqa" else 0]
    got = run()
    assert got["status"] == dcp.DCP_ERR_BOUNDS
    assert (got["out"][:, 0] == 0).all() and (got["out_lse"][:, 0] == -np.inf).all()
    assert np.array_equal(got["out"][:, 1], ref["out"][:, 1]) and np.array_equal(got["lse"][:, 1], ref["lse"][:, 1])


@pytest.mark.parametrize("name,kw,rope", [
    ("qwen_gqa", dict(batch=3, dcp_size=2, interleave=1), dict(rot_dim=128, base=1e6)),
    ("mla_32", dict(batch=3, num_q_heads=32, dcp_size=2), dict(rot_dim=64, rot_offset=512, layout="interleaved")),
])
def test_a_captured_verify_step_replays(name, kw, rope):
    """Append, attend, merge and commit in one graph, lengths advanced in place: three replays equal
    three eager steps bit for bit, on a stream of their own."""
    from context_decode_attention_paged_gb300 import binding as dcp
    L = 6
    inst = H.build_instance(H.small(name, q_len=L, lengths=("fixed", 900), **kw))
    w, dev = inst.w, torch.device("cuda:0")
    mask, depth = dcp.tree_mask([-1, 0, 0, 1, 2, 4])
    mask, depth = mask.view(1, L, 1).to(dev), depth.view(1, L).to(dev)
    table = dcp.dcp_rope_table(**rope)
    bt = inst.block_tables.to(dev)
    acc = torch.tensor([[0, 2, 4], [0, 1, 0], [0, 2, 4]], dtype=torch.int32, device=dev)
    take = torch.tensor([3, 2, 1], dtype=torch.int32, device=dev)
    k, v, q = (T.to_gpu(t) for t in T.append_inputs(w, L, 9))
    base = torch.tensor([800, 511, 100], dtype=torch.int32, device=dev)

    class State:
        def __init__(self):
            self.kv, self.lens, self.q_out = inst.kv_cache.to(dev), base + L, torch.empty_like(q).contiguous()
            desc = dcp.desc_from_tensors(w.kind, self.q_out, self.kv, bt, w.head_dim_v)
            self.ws = torch.empty((max(1, dcp.dcp_tree_attn_workspace_size(desc, w.dcp_size)),), dtype=torch.uint8,
                                  device=dev)
            self.po = torch.empty((w.dcp_size, w.batch, L, w.num_q_heads, w.head_dim_v), device=dev)
            self.lse = torch.empty(self.po.shape[:-1], device=dev)
            self.out = None

        def step(self):
            dcp.dcp_kv_cache_append(w.kind, k, v, self.kv, bt, self.lens, w.dcp_size, w.interleave, table, q=q,
                                    q_out=self.q_out, pos_offsets=depth)
            dcp.dcp_tree_attn(w.kind, self.q_out, self.kv, bt, self.lens, mask, w.dcp_size, w.interleave, w.scale,
                              w.head_dim_v, partial_out=self.po, lse=self.lse, workspace=self.ws)
            self.out = dcp.dcp_merge(self.po, self.lse, w.dcp_size)
            dcp.dcp_kv_cache_commit(w.kind, self.kv, bt, self.lens, L, acc, take, w.dcp_size, w.interleave,
                                    new_seq_lens=self.lens)
            self.lens += L

    eager, want = State(), []
    for _ in range(3):
        eager.step()
        want.append((eager.out[0].clone(), eager.out[1].clone()))
    torch.cuda.synchronize()
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK
    s, side = State(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.step()
    for out, out_lse in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.out[0], out) and torch.equal(s.out[1], out_lse)
    assert torch.equal(s.kv, eager.kv) and torch.equal(s.lens, eager.lens)
    assert s.lens.tolist() == [800 + 3 * 3 + L, 511 + 2 * 3 + L, 100 + 3 + L]


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("name", ["mla_32", "qwen_gqa"])
def test_a_table_wider_than_any_length(name, tree):
    """2^20 entries of 4,096 tokens: the splits' first tokens stay 32-bit."""
    inst, mask, _ = T.tree_case(name, 4, batch=1, lengths=("fixed", 9000), dcp_size=1, block_size=4096)
    inst.block_tables = torch.nn.functional.pad(inst.block_tables, (0, (1 << 20) - inst.block_tables.shape[2]))
    if tree:
        check(inst, mask)
    else:
        from gpu_common import check_against_oracle
        check_against_oracle(inst)


@pytest.mark.parametrize("name,L,kw,opt", [
    ("qwen_gqa", 20, dict(batch=3, lengths=("uniform", 100, 900), dcp_size=2), dict(q_lens=[20, 5, 0])),
    ("qwen_gqa", 40, dict(batch=2, lengths=("uniform", 100, 900), dcp_size=2, interleave=1),
     dict(q_lens=[40, 9], mask="random")),
    ("qwen_gqa", 33, dict(batch=2, num_q_heads=40, lengths=("uniform", 100, 1500), dcp_size=1), dict(q_lens=[33, 13])),
    ("qwen_gqa", 33, dict(batch=1, num_q_heads=40, lengths=("fixed", 33), dcp_size=2), {}),
    ("qwen_gqa", 19, dict(batch=2, num_q_heads=64, num_kv_heads=2, lengths=("uniform", 100, 1500)), {}),
    ("tiny_gqa", 150, dict(batch=2, lengths=("uniform", 150, 600), dcp_size=2), dict(q_lens=[150, 31])),
])
def test_odd_numbers_of_row_blocks(name, L, kw, opt):
    """Three and five blocks of 128 rows, the last one partly there, nodes that lie across two
    blocks, and requests that end before a block."""
    check(*T.tree_case(name, L, **kw, **opt))
