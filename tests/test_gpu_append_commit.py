"""GPU parity of the rotary append and of committing an accepted path.

Tolerance of a rotated value y = m (x0 c - x1 s): one rounding to bf16 (half a
step, 2^-8 |y|) plus the fp32 arithmetic before it - c and s are within
2^-22 (phase to 2^-32 of a turn, its conversion to fp32 2^-24 of half a turn
times pi, the function's own 2^-23), and the two products and the sum add
3 * 2^-24 - so 2^-20 m (|x0| + |x1|) covers it.  Everything else is exact."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import helpers as H
import tree_common as T
from oracle import dcp_oracle as orc
from oracle import tree_oracle as tro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from context_decode_attention_paged_gb300 import build
    build.build()


def _assert_rotated(got, want, x, mscale, what):
    err = np.abs(got - want)
    tol = np.abs(want) * 2.0 ** -8 + mscale * 2.0 ** -20 * 2 * np.abs(x).max()
    assert (err <= tol).all(), f"{what}: {err.max()} at {np.unravel_index(np.argmax(err - tol), err.shape)}"


ROPES = {
    "half": dict(rot_dim=64),
    "half_part": dict(rot_dim=32, rot_offset=16),
    "half_odd_offset": dict(rot_dim=20, rot_offset=6),          # value by value
    "half_short": dict(rot_dim=8),                              # half a vector of pairs: value by value
    "half_three": dict(rot_dim=48),                             # three vectors: one block a token
    "inter_three": dict(rot_dim=24, rot_offset=16, layout="interleaved"),
    "inter": dict(rot_dim=64, layout="interleaved"),
    "inter_part": dict(rot_dim=24, rot_offset=8, layout="interleaved"),
    "inter_odd": dict(rot_dim=2, rot_offset=5, layout="interleaved"),
    "linear": dict(rot_dim=64, scaling="linear", factor=8.0),
    "ntk": dict(rot_dim=64, scaling="ntk", factor=4.0),
    "yarn": dict(rot_dim=64, scaling="yarn", factor=40.0, original_max_position=4096, base=1e6),
    "mscale": dict(rot_dim=64, mscale=0.25),
}
MLA_ROPES = {
    "mla_inter": dict(rot_dim=64, rot_offset=512, layout="interleaved", scaling="yarn", factor=40.0,
                      original_max_position=4096),
    "mla_half": dict(rot_dim=64, rot_offset=512),
}

CASES = [("tiny_gqa", dict(batch=3, lengths=("uniform", 9, 700), dcp_size=4, interleave=3), 7, r) for r in ROPES] + [
    ("tiny_gqa", dict(batch=1, lengths=("fixed", 1), dcp_size=2, interleave=1), 1, "half"),
    ("tiny_gqa", dict(batch=2, lengths=("fixed", 5), dcp_size=2, interleave=1), 5, "half"),       # nothing before them
    ("tiny_gqa", dict(batch=2, num_q_heads=10, num_kv_heads=5, head_dim_qk=72, head_dim_v=72, block_size=24,
                      lengths=("uniform", 40, 300)), 3, "half"),
    ("qwen_gqa", dict(batch=4, lengths=("uniform", 300, 5000)), 33, "half"),
    ("mla_32", dict(batch=3, num_q_heads=16, lengths=("uniform", 129, 3000), interleave=1), 5, "mla_inter"),
    ("mla_32", dict(batch=2, num_q_heads=128, lengths=("fixed", 257), dcp_size=2), 1, "mla_half"),
    ("mla_mtp", dict(num_q_heads=4, lengths=("fixed", 40000)), 4, "mla_inter"),
]


def _append(inst, n, rope_kw, fused=True, q_lens=None, offsets=None, with_q=True, in_place=False, seed=5):
    from context_decode_attention_paged_gb300 import binding as dcp
    w = inst.w
    k, v, q = T.append_inputs(w, n, seed, fused)
    rope = dcp.dcp_rope_table(**rope_kw)
    kv = inst.kv_cache.cuda()
    gq = T.to_gpu(q) if with_q else None
    q_out = None if not with_q else gq if in_place else torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    dcp.dcp_kv_cache_append(w.kind, T.to_gpu(k), T.to_gpu(v), kv, inst.block_tables.cuda(), inst.seq_lens.cuda(),
                            w.dcp_size, w.interleave, rope, q=gq, q_out=q_out, q_lens=None if ql is None else ql.cuda(),
                            pos_offsets=None if off is None else off.cuda())
    torch.cuda.synchronize()
    freqs = tro.rope_freqs(rope_kw["rot_dim"], rope_kw.get("base", 10000.0), rope_kw.get("scaling", "none"),
                           rope_kw.get("factor", 1.0), rope_kw.get("original_max_position", 0))
    m = rope_kw.get("mscale", 0.1 * math.log(rope_kw["factor"]) + 1.0 if rope_kw.get("scaling") == "yarn" else 1.0)
    first = np.full(q.shape, 7.0) if not in_place else orc.to_f64(q)
    want, want_q = tro.ref_append(w.kind, orc.to_f64(inst.kv_cache), orc.to_f64(k), None if v is None else orc.to_f64(v),
                                  orc.to_f64(q) if with_q else None, inst.block_tables.numpy(), inst.seq_lens.numpy(),
                                  w.dcp_size, w.interleave, w.block_size, freqs, rope_kw.get("layout", "half"),
                                  rope_kw.get("rot_offset", 0), m, q_lens, offsets, first)
    _assert_rotated(orc.to_f64(kv), want, orc.to_f64(k), m, "cache")
    # outside the rotated dims of the new keys nothing differs in a bit
    lo = rope_kw.get("rot_offset", 0)
    same = np.ones(want.shape, dtype=bool)
    rows = np.abs(orc.to_f64(inst.kv_cache) - want) > 0
    touched = rows.any(axis=-1, keepdims=True)
    if w.kind == "gqa":
        touched[1] = False
    same[..., lo:lo + rope_kw["rot_dim"]] &= ~np.broadcast_to(touched, want.shape)[..., lo:lo + rope_kw["rot_dim"]]
    assert np.array_equal(orc.to_f64(kv)[same], want[same])
    if with_q:
        _assert_rotated(orc.to_f64(q_out), want_q, orc.to_f64(q), m, "queries")
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK
    return kv, q_out


@pytest.mark.parametrize("name,kw,n,rope", CASES)
def test_append_matches_the_oracle(name, kw, n, rope):
    _append(H.build_instance(H.small(name, **kw)), n, {**ROPES, **MLA_ROPES}[rope])


@pytest.mark.parametrize("fused,in_place,with_q", [(False, False, True), (False, True, True), (True, False, False)])
def test_append_rows_of_their_own_in_place_and_without_queries(fused, in_place, with_q):
    inst = H.build_instance(H.small("qwen_gqa", batch=2, lengths=("uniform", 100, 900), dcp_size=2, interleave=16))
    _append(inst, 3, dict(rot_dim=128), fused=fused, in_place=in_place, with_q=with_q)


@pytest.mark.parametrize("name,kw,rope", [
    ("tiny_gqa", dict(batch=4, lengths=("uniform", 20, 300), dcp_size=2, interleave=1), dict(rot_dim=32)),
    ("mla_32", dict(batch=4, num_q_heads=16, lengths=("uniform", 20, 300)), MLA_ROPES["mla_inter"]),
])
@pytest.mark.parametrize("shared", [True, False])
def test_append_trees_of_different_sizes(name, kw, rope, shared):
    """Offsets are depths (several nodes share a position), a request holds fewer nodes than rows
    or none, and the rows behind them stay as they were."""
    inst = H.build_instance(H.small(name, **kw))
    rng = np.random.default_rng(4)
    offsets = rng.integers(0, 5, size=(1 if shared else 4, 6)).tolist()
    _append(inst, 6, rope, q_lens=[6, 0, 1, 5], offsets=offsets)


def test_append_many_tokens_of_ragged_requests():
    """More tasks than the SMs hold at once: the blocks number them over the tokens that are there
    (empty requests among them, a bad one reported and skipped)."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small("tiny_gqa", batch=9, num_q_heads=64, num_kv_heads=8, lengths=("fixed", 700),
                                    dcp_size=2))
    lens = [500, 0, 1, 700, 33, 0, 256, 700, 0]
    _append(inst, 700, dict(rot_dim=64), q_lens=lens)
    w = inst.w
    k, v, q = T.append_inputs(w, 700, 5)
    ql = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ql[3] = 701
    kv = inst.kv_cache.cuda()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    dcp.dcp_kv_cache_append(w.kind, T.to_gpu(k), T.to_gpu(v), kv, inst.block_tables.cuda(), inst.seq_lens.cuda(),
                            w.dcp_size, w.interleave, dcp.dcp_rope_table(64), q=T.to_gpu(q), q_out=out, q_lens=ql)
    assert dcp.dcp_get_last_device_status() == dcp.DCP_ERR_BOUNDS
    assert (out[3] == 7).all() and (out[0, 500:] == 7).all() and not (out[0, :500] == 7).all(dim=-1).any()
    assert not (out[7] == 7).all(dim=-1).any() and not (out[2, 0] == 7).all(dim=-1).any()


def test_append_far_and_negative_positions_keep_their_angle():
    """A position offset reaches any int32 position: the phase is exact modulo a turn."""
    inst = H.build_instance(H.small("tiny_gqa", batch=2, lengths=("fixed", 40)))
    _append(inst, 3, dict(rot_dim=64), offsets=[[2_000_000_000, 123_456_789, -37], [-2_000_000_000, 1_000_003, 0]])


def test_append_copies_special_values():
    """Infinities and NaN pass the unrotated part bit for bit and stay in their own pair."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small("tiny_gqa", batch=1, lengths=("fixed", 33)))
    w = inst.w
    k, v, _ = T.append_inputs(w, 1, 5, fused=False)
    k[0, 0, 0, 3], k[0, 0, 1, 50], v[0, 0, 0, 0] = math.inf, math.nan, -math.inf
    kv = inst.kv_cache.cuda()
    dcp.dcp_kv_cache_append(w.kind, k.cuda(), v.cuda(), kv, inst.block_tables.cuda(), inst.seq_lens.cuda(), w.dcp_size,
                            w.interleave, dcp.dcp_rope_table(32))
    blk, slot = T.cell(inst, 0, 32)
    row = kv[0, blk, slot].float().cpu().numpy()
    assert np.isnan(row[1, 50]) and np.isfinite(np.delete(row[1], 50)).all()
    assert not np.isfinite(row[0, 3]) and not np.isfinite(row[0, 19])
    assert np.isfinite(np.delete(row[0], [3, 19])).all()
    assert kv[1, blk, slot, 0, 0].item() == -math.inf


@pytest.mark.parametrize("bad", ["short", "count", "negative", "table", "block"])
def test_append_reports_and_skips_bad_requests(bad):
    """One bad request of two sets DCP_ERR_BOUNDS; its cache rows stay, the other's are written."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small("tiny_gqa", batch=2, lengths=("fixed", 40)))
    w = inst.w
    k, v, q = T.append_inputs(w, 3, 5)
    sl, bt = inst.seq_lens.clone(), inst.block_tables.clone()
    ql = torch.tensor([3, 3], dtype=torch.int32)
    if bad == "short":
        sl[0] = 2
    elif bad == "count":
        ql[0] = 4
    elif bad == "negative":
        ql[0] = -1
    elif bad == "table":
        sl[0] = 10 ** 6
    else:
        bt[:, 0] = inst.kv_cache.shape[1]
    kv = inst.kv_cache.cuda()
    dcp.dcp_kv_cache_append(w.kind, T.to_gpu(k), T.to_gpu(v), kv, bt.cuda(), sl.cuda(), w.dcp_size, w.interleave,
                            dcp.dcp_rope_table(64), q=T.to_gpu(q), q_lens=ql.cuda())
    assert dcp.dcp_get_last_device_status() == dcp.DCP_ERR_BOUNDS
    changed = (kv.cpu() != inst.kv_cache).any(dim=-1).any(dim=-1)[0]
    want = {T.cell(inst, 1, t) for t in (37, 38, 39)}
    assert {tuple(x) for x in torch.nonzero(changed).tolist()} == want


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------

COMMITS = [
    ("tiny_gqa", dict(batch=4, lengths=("uniform", 20, 300), dcp_size=4, interleave=3), 9,
     [[0, 1, 2, 0], [0, 3, 5, 8], [4, 0, 0, 0], [2, 3, 4, 5]], [3, 4, 1, 0], None),
    ("tiny_gqa", dict(batch=2, lengths=("fixed", 9), dcp_size=2, interleave=1), 9,
     [[0, 1, 2, 3, 4, 5, 6, 7, 8], [1, 2, 3, 4, 5, 6, 7, 8, 0]], [9, 8], None),            # all nodes; every row moves
    ("tiny_gqa", dict(batch=3, num_kv_heads=1, num_q_heads=8, lengths=("uniform", 30, 90)), 6,
     [[1, 2], [0, 0], [0, 3]], [2, 0, 2], [3, 0, 4]),                                        # counts of their own
    ("qwen_gqa", dict(batch=2, lengths=("uniform", 300, 900)), 33, [[1, 9, 20, 32], [0, 2, 4, 6]], [4, 4], None),
    ("mla_32", dict(batch=2, num_q_heads=4, lengths=("uniform", 129, 700), interleave=1), 64,
     [list(range(0, 64, 4)), list(range(1, 33, 2))], [16, 11], None),
    ("mla_32", dict(batch=1, num_q_heads=4, lengths=("fixed", 300), dcp_size=2), 200, [list(range(0, 200))], [200], None),
    ("mla_32", dict(batch=1, num_q_heads=4, lengths=("fixed", 700), dcp_size=2), 300, [list(range(44, 300))], [256], None),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name,kw,L,path,take,q_lens", COMMITS)
def test_commit_is_bit_exact(name, kw, L, path, take, q_lens, in_place):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small(name, **kw))
    w = inst.w
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    kv, sl = inst.kv_cache.cuda(), inst.seq_lens.cuda()
    lens = dcp.dcp_kv_cache_commit(w.kind, kv, inst.block_tables.cuda(), sl, L, i32(path), i32(take), w.dcp_size,
                                   w.interleave, q_lens=i32(q_lens), new_seq_lens=sl if in_place else None)
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK
    want, want_lens = tro.ref_commit(w.kind, orc.to_f64(inst.kv_cache), inst.block_tables.numpy(), inst.seq_lens.numpy(), L,
                                     path, take, w.dcp_size, w.interleave, w.block_size, q_lens)
    assert np.array_equal(orc.to_f64(kv), want)
    assert lens.tolist() == want_lens.tolist()


@pytest.mark.parametrize("path,take,q_len0", [
    ([0, 2, 2], 3, 5), ([0, 3, 1], 3, 5), ([-1, 1, 2], 3, 5), ([0, 1, 5], 3, 5), ([0, 1, 2], 4, 5), ([0, 1, 2], -1, 5),
    ([0, 1, 2], 3, 2), ([0, 1, 2], 3, 99), ([0, 1, 2], 3, -3)])
def test_commit_skips_bad_paths(path, take, q_len0):
    """A path that does not increase, leaves the tree or is longer than its row: the request's rows
    and length stay, the other request commits."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small("tiny_gqa", batch=2, lengths=("fixed", 40)))
    w = inst.w
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    kv = inst.kv_cache.cuda()
    lens = dcp.dcp_kv_cache_commit(w.kind, kv, inst.block_tables.cuda(), inst.seq_lens.cuda(), 6, i32([path, [0, 4, 0]]),
                                   i32([take, 2]), w.dcp_size, w.interleave, q_lens=i32([q_len0, 6]))
    assert dcp.dcp_get_last_device_status() == dcp.DCP_ERR_BOUNDS
    assert lens.tolist() == [40, 36]
    changed = (kv.cpu() != inst.kv_cache).any(dim=-1).any(dim=-1)[0]
    assert {tuple(x) for x in torch.nonzero(changed).tolist()} == {T.cell(inst, 1, 35)}


def test_commit_reports_bad_blocks():
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small("tiny_gqa", batch=1, lengths=("fixed", 40), dcp_size=1))
    w = inst.w
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    for bad in (-1, inst.kv_cache.shape[1], None):
        bt, sl = inst.block_tables.clone(), inst.seq_lens.clone()
        if bad is None:
            sl[0] = 10 ** 6                                  # past the block table
        else:
            bt[:] = bad
        kv = inst.kv_cache.cuda()
        lens = dcp.dcp_kv_cache_commit(w.kind, kv, bt.cuda(), sl.cuda(), 8, i32([[0, 4]]), i32([2]), w.dcp_size,
                                       w.interleave)
        assert dcp.dcp_get_last_device_status() == dcp.DCP_ERR_BOUNDS
        assert lens.tolist() == sl.tolist() and torch.equal(kv.cpu(), inst.kv_cache)


@pytest.mark.parametrize("dim,rope", [(400008, dict(rot_dim=64, rot_offset=8)), (262136, dict(rot_dim=128)),
                                      (524280, dict(rot_dim=64, rot_offset=64, layout="interleaved"))])
def test_heads_of_hundreds_of_thousands_of_dims(dim, rope):
    """Every vector that does not turn is copied, up to rows of 1 MB."""
    from context_decode_attention_paged_gb300 import binding as dcp
    g = torch.Generator().manual_seed(2)
    k, q = torch.randn((1, 1, dim), generator=g).to(torch.bfloat16), torch.randn((1, 1, 8, dim), generator=g).to(torch.bfloat16)
    cache = torch.zeros((2, 1, dim), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[[0, 1]]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([2], dtype=torch.int32, device="cuda")
    _, q_out = dcp.dcp_kv_cache_append("mla", k.cuda(), None, cache, table, lens, 1, 1, dcp.dcp_rope_table(**rope), q=q.cuda())
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK
    f = tro.rope_freqs(rope["rot_dim"], 1e4)
    args = f, rope.get("layout", "half"), rope.get("rot_offset", 0), 1.0
    for got, x in ((cache[1, 0], k[0, 0]), (q_out[0, 0], q[0, 0])):
        _assert_rotated(orc.to_f64(got.cpu()), tro.rotate(orc.to_f64(x), 1, *args), orc.to_f64(x), 1.0, "row")
    lo, hi = rope.get("rot_offset", 0), rope.get("rot_offset", 0) + rope["rot_dim"]
    assert torch.equal(cache[1, 0, hi:].cpu(), k[0, 0, hi:]) and torch.equal(q_out[..., hi:].cpu(), q[..., hi:])
    assert torch.equal(q_out[..., :lo].cpu(), q[..., :lo]) and (cache[0] == 0).all()
