"""Edges of the 8-bit cache's operators: hidden and special values, scales far apart, bad requests, far offsets, streams and
graphs, bounded waits, and a run of the operators as a serving loop uses them."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import helpers as H
import kv8_common as K
import test_gpu_kv8_append as A
from oracle import dcp_oracle as orc
from oracle import kv8_oracle as k8o
from oracle import tree_oracle as tro

pytestmark = pytest.mark.gpu

TC = dict(batch=3, lengths=("uniform", 200, 900))
SHAPES = [("tiny_gqa", 3, TC), ("qwen_gqa", 1, TC), ("qwen_gqa", 5, TC), ("qwen_gqa", 2, dict(TC, block_size=48)),
          ("mla_32", 2, dict(TC, num_q_heads=8))]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from context_decode_attention_paged_gb300 import build
    build.build()


def _cell(inst, b, t):
    w = inst.w
    return tro.cell_of(inst.block_tables.numpy(), b, t, w.interleave, w.dcp_size, w.block_size)


def _row(inst, codes, b, t, pool):
    blk, slot = _cell(inst, b, t)
    return codes[pool, blk, slot] if inst.w.kind == "gqa" else codes[blk, slot]


@pytest.mark.parametrize("name,Lq,kw", SHAPES)
def test_slots_that_no_token_occupies_may_hold_nan(name, Lq, kw):
    inst, codes, scales, _ = K.kv8_case(name, Lq, **kw)
    want = K.oracle_attn(inst, codes, scales)
    live = np.zeros(codes.shape, dtype=bool)
    for b, S in enumerate(inst.seq_lens.tolist()):
        for t in range(S):
            for pool in (0, 1) if inst.w.kind == "gqa" else (0,):
                _row(inst, live, b, t, pool)[...] = True
    poisoned = np.where(live, codes, 127).astype(np.uint8)
    K.check_attn(K.run_attn(inst, poisoned, scales), want, codes, scales)


@pytest.mark.parametrize("name,Lq,kw", [s for s in SHAPES if s[1] > 1])
def test_nan_values_and_keys_of_hidden_tokens_stay_hidden_and_seen_ones_show(name, Lq, kw):
    """The last token's value (GQA: and key) holds NaN: every earlier query of the request is as before, the last one's
    value entry (with a NaN key: its whole row) is NaN."""
    for pool, key in ((1, False), (0, True)) if name != "mla_32" else ((0, True),):
        inst, codes, scales, _ = K.kv8_case(name, Lq, **kw)
        b = 1
        S = int(inst.seq_lens[b])
        row = _row(inst, codes, b, S - 1, pool)
        row[..., 5] = 127 | 128 * (pool == 1)
        want = K.oracle_attn(inst, codes, scales)
        got = K.run_attn(inst, codes, scales)
        last = np.isnan(want["out"][:, b, Lq - 1])
        assert last.any() and not np.isnan(want["out"][:, b, :Lq - 1]).any()
        if key:
            # a score of NaN makes the row NaN in the shard that holds the key
            assert np.isnan(got["out"][:, b, Lq - 1]).all()
            for x in (got, want):
                for k in ("out", "out_lse", "partial_out", "lse"):
                    x[k][:, b, Lq - 1] = 0.0
        if not key:
            K.check_attn(got, want, codes, scales)
        else:
            K.check_attn(got, want, codes, scales)


@pytest.mark.parametrize("name,Lq,kw", SHAPES)
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_a_query_that_is_not_finite_makes_its_row_nan_alone(name, Lq, kw, value):
    inst, codes, scales, _ = K.kv8_case(name, Lq, **kw)
    want = K.oracle_attn(inst, codes, scales)
    inst.q[1, 0, 3, 7] = value
    got = K.run_attn(inst, codes, scales)
    N, per = inst.w.dcp_size, inst.w.num_q_heads // inst.w.dcp_size
    assert np.isnan(got["out"][3 // per, 1, 0, 3 % per]).all()
    got["out"][3 // per, 1, 0, 3 % per] = want["out"][3 // per, 1, 0, 3 % per]
    got["out_lse"][3 // per, 1, 0, 3 % per] = want["out_lse"][3 // per, 1, 0, 3 % per]
    for k in ("partial_out", "lse"):
        got[k][:, 1, 0, 3] = want[k][:, 1, 0, 3]
    K.check_attn(got, want, codes, scales)


@pytest.mark.parametrize("name,Lq,kw", SHAPES[:3])
def test_scales_far_apart(name, Lq, kw):
    """Value scales from 2^-20 to 2^20 a block: an output is off by 2^-11 + 2^-12 of sum p |v|, its own size, not of the
    largest value (kv8_common.check_attn's bound with the weights that it comes from)."""
    inst, codes, scales, _ = K.kv8_case(name, Lq, **kw)
    rng = np.random.default_rng(9)
    scales[1] = rng.integers(107, 148, scales[1].shape).astype(np.uint8)
    got, want = K.run_attn(inst, codes, scales), K.oracle_attn(inst, codes, scales)
    values = k8o.dequantise(codes, scales)
    values[1] = np.abs(values[1])
    w = inst.w
    size = tro.ref_tree(w.kind, orc.to_f64(inst.q), values, inst.block_tables.numpy(), inst.seq_lens.numpy(), K.chain(Lq),
                        w.dcp_size, w.interleave, w.block_size, w.scale, w.head_dim_v)["partial_out"]
    err = np.abs(got["partial_out"] - want["partial_out"])
    assert (err <= (2.0 ** -11 + 2.0 ** -12) * size + 1e-30).all(), float((err / (size + 1e-30)).max())
    assert np.abs(got["out_lse"] - want["out_lse"]).max() <= 2e-4


@pytest.mark.parametrize("name,Lq,kw", [("qwen_gqa", 1, dict(batch=2, lengths=("fixed", 3000), dcp_size=1)),
                                        ("tiny_gqa", 3, dict(batch=2, lengths=("fixed", 2500), dcp_size=1))])
def test_scores_that_grow_along_the_sequence(name, Lq, kw):
    """Key scales that rise with the block: the running reference moves again and again, across tiles and cut units."""
    inst, codes, scales, _ = K.kv8_case(name, Lq, std=6.0, **kw)
    for b in range(inst.w.batch):
        nb = -(-int(inst.seq_lens[b]) // inst.w.block_size)
        for j in range(nb):
            scales[0, int(inst.block_tables[0, b, j])] = 119 + (10 * j) // nb
    want = K.oracle_attn(inst, codes, scales)
    assert want["lse"].max() > 40
    K.check_attn(K.run_attn(inst, codes, scales), want, codes, scales)


@pytest.mark.parametrize("name,Lq,kw", SHAPES[:4])
@pytest.mark.parametrize("size", [-2.0 ** 110, 2.0 ** 110])
def test_scores_of_any_finite_size(name, Lq, kw, size):
    """All keys are ones, so a row's scores are one number, about 2^114.  LSE: the product is exact, then 4 roundings and
    that of the logarithm.  The weights are equal within a part of the work; parts are joined by their fp32 LSEs, whose step
    is 2^90 here, so the logarithm of a part's count is lost and parts of any counts weigh the same: what holds of an output
    is that it lies among the values seen, but for the roundings of the sums and quotients (a few times 2^-24 of the largest)."""
    inst, codes, scales, _ = K.kv8_case(name, Lq, **kw)
    codes[0] = k8o.encode(np.ones(codes[0].shape))
    scales[...] = 127
    inst.q.fill_(size)
    got, want = K.run_attn(inst, codes, scales), K.oracle_attn(inst, codes, scales)
    seen = want["lse"] != -np.inf
    assert np.isfinite(want["lse"][seen]).all() and np.array_equal(got["lse"] != -np.inf, seen)
    vmax = np.abs(k8o.dequantise(codes, scales)[1]).max()
    values, w = k8o.dequantise(codes, scales), inst.w
    for b, S in enumerate(inst.seq_lens.tolist()):
        rows = np.stack([_row(inst, values, b, t, 1) for t in range(S)])                  # [S][Hkv][D]
        shard = np.arange(S) // w.interleave % w.dcp_size
        for r in range(w.dcp_size):
            for i in range(Lq):
                held = np.repeat(rows[(shard == r) & (np.arange(S) <= S - Lq + i)], w.num_q_heads // w.num_kv_heads, axis=1)
                out = got["partial_out"][r, b, i]
                if len(held):
                    assert (out >= held.min(0) - 2.0 ** -20 * vmax).all() and (out <= held.max(0) + 2.0 ** -20 * vmax).all()
                else:
                    assert not out.any()
    assert (np.abs(got["lse"][seen] - want["lse"][seen]) <= 2.0 ** -21 * np.abs(want["lse"][seen])).all()


def test_a_sink_beside_a_hundred_thousand_small_weights():
    """One key 12 above the rest (e^-12 is 2^-17.3) over 100,000 others that together outweigh it."""
    inst, codes, scales, _ = K.kv8_case("qwen_gqa", 1, batch=1, num_q_heads=16, num_kv_heads=1, lengths=("fixed", 100000),
                                        dcp_size=1, block_size=256)
    q = orc.to_f64(inst.q)[0, 0]
    codes[0] = k8o.encode(np.random.default_rng(1).standard_normal(codes[0].shape) * 0.02)       # (scores near 0)
    blk, slot = _cell(inst, 0, 50)
    scales[0] = 127
    direction = np.linalg.lstsq(q, np.full(16, 12.0 / inst.w.scale), rcond=None)[0]
    codes[0, blk, slot, 0] = k8o.encode(direction)
    want = K.oracle_attn(inst, codes, scales)
    sink = np.exp(q @ k8o.VALUES[codes[0, blk, slot, 0]] * inst.w.scale - want["out_lse"].reshape(-1))
    assert ((sink > 0.3) & (sink < 0.95)).any()
    K.check_attn(K.run_attn(inst, codes, scales), want, codes, scales)


@pytest.mark.parametrize("name,Lq,kw", SHAPES)
@pytest.mark.parametrize("what", ["short", "count", "negative", "table", "block"])
def test_bad_requests_are_empty_and_reported(name, Lq, kw, what):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, codes, scales, _ = K.kv8_case(name, Lq, **kw)
    ql = torch.full((3,), Lq, dtype=torch.int32)
    want = K.oracle_attn(inst, codes, scales, ql)
    shards = list(range(inst.w.dcp_size))
    if what == "short":
        inst.seq_lens[1] = Lq - 1
    elif what == "count":
        ql[1] = Lq + 1
    elif what == "negative":
        ql[1] = -1
    elif what == "block":
        shards = [0]
        inst.block_tables[0, 1, 0] = inst.kv_cache.shape[1 if inst.w.kind == "gqa" else 0]
    elif what == "table":
        # more tokens than the table has room for: reported (and cut off, as the decode kernels do)
        inst.seq_lens[1] = inst.block_tables.shape[2] * inst.w.block_size * inst.w.dcp_size + 50 * inst.w.interleave
        inst.block_tables[:, 1] = inst.block_tables[:, 1].clamp(min=0)
    got = K.run_attn(inst, codes, scales, ql)
    assert got["status"] == dcp.DCP_ERR_BOUNDS
    if what != "table":
        for r in shards:
            assert (got["partial_out"][r, 1] == 0).all() and (got["lse"][r, 1] == -np.inf).all()
    for b in (0, 2):
        for k in ("partial_out", "lse"):
            x, y = got[k][:, b], want[k][:, b]
            fin = np.isfinite(y)
            assert np.array_equal(fin, np.isfinite(x)) and np.abs(x[fin] - y[fin]).max() < 0.02


def test_requests_without_queries_read_no_table():
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, codes, scales, _ = K.kv8_case("qwen_gqa", 2, **TC)
    ql = torch.tensor([2, 0, 1], dtype=torch.int32)
    want = K.oracle_attn(inst, codes, scales, ql)
    inst.block_tables[:, 1] = 1 << 30
    got = K.run_attn(inst, codes, scales, ql)
    assert got["status"] == dcp.DCP_OK
    K.check_attn(got, want, codes, scales)
    inst.seq_lens[1] = 0
    got = K.run_attn(inst, codes, scales, ql)
    assert got["status"] == dcp.DCP_OK
    K.check_attn(got, want, codes, scales)


@pytest.mark.parametrize("types", [("uint8", "float8_e8m0fnu"), ("float8_e4m3fn", "uint8"), ("float8_e4m3fn", "float8_e8m0fnu")])
def test_types_of_codes_and_scales(types):
    inst, codes, scales, _ = K.kv8_case("tiny_gqa", 1, **TC)
    a, b = K.run_attn(inst, codes, scales), K.run_attn(inst, codes, scales, types=types)
    assert np.array_equal(a["partial_out"], b["partial_out"]) and np.array_equal(a["lse"], b["lse"])


def test_binding_refuses_other_tensors():
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, codes, scales, _ = K.kv8_case("tiny_gqa", 1, **TC)
    with pytest.raises(dcp.DcpError):
        K.run_attn(inst, codes.astype(np.int8).view(np.uint8)[:, :, :, :1], scales)        # heads of q and cache differ
    with pytest.raises(dcp.DcpError):
        K.run_attn(inst, codes, scales[:, :-1])
    with pytest.raises(dcp.DcpError):
        K.run_attn(inst, codes, scales, types=("int8", "uint8"))
    with pytest.raises(dcp.DcpError):
        K.run_attn(inst, codes, scales, workspace=torch.empty((64,), dtype=torch.uint8, device="cuda"))
    with pytest.raises(dcp.DcpError):
        K.run_attn(inst, codes, scales, lse=torch.empty((2, 3, 1, 8), device="cpu"))


def test_blocks_behind_four_gigabytes():
    """Codes whose offsets pass 32 bits: appended, read back and attended at the pool's end."""
    from context_decode_attention_paged_gb300 import binding as dcp
    hkv, D, bs, nb, n = 8, 128, 128, 40000, 200
    cache = torch.zeros((2, nb, bs, hkv, D), dtype=torch.uint8, device="cuda")             # 10.5 GB
    scales = torch.full((2, nb, hkv), 127, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn((1, n, hkv, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((1, 1, 16, D), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[[nb - 1, nb - 7]]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    dcp.dcp_kv8_append("gqa", k, v, cache, scales, table, lens, 1, bs)
    ok, ov = dcp.dcp_kv8_read("gqa", cache, scales, table, lens, n, 1, bs)
    for a, b in ((ok, k), (ov, v)):
        assert ((a.float() - b.float()).abs() <= 2.0 ** -4 * b.float().abs() + 2.0 ** -14).all()
    po, lse = dcp.dcp_kv8_decode_attn("gqa", q, cache, scales, table, lens, 1, bs, D ** -0.5, 1, D)
    x = torch.einsum("hgd,thd->hgt", q[0, 0].double().view(hkv, 2, D), ok[0].double()) * D ** -0.5
    want = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), ov[0].double()).reshape(16, D)
    assert (po[0, 0, 0].double() - want).abs().max() <= 2.0 ** -10 * ov.abs().max()
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK


@pytest.mark.parametrize("name,Lq,kw", SHAPES[:3])
def test_streams_graphs_and_changed_lengths(name, Lq, kw):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, codes, scales, _ = K.kv8_case(name, Lq, **kw)
    w = inst.w
    on = lambda t: torch.as_tensor(t).cuda()   # noqa: E731
    q, c, s, bt, sl = on(inst.q), on(codes), on(scales), on(inst.block_tables), on(inst.seq_lens)
    desc = dcp.desc_from_tensors(w.kind, q, c, bt, w.head_dim_v)
    new = lambda: dict(partial_out=torch.empty((w.dcp_size, w.batch, Lq, w.num_q_heads, w.head_dim_v), device="cuda"),   # noqa: E731
                       lse=torch.empty((w.dcp_size, w.batch, Lq, w.num_q_heads), device="cuda"),
                       workspace=torch.empty((dcp.dcp_kv8_decode_attn_workspace_size(desc, w.dcp_size) or 1,),
                                             dtype=torch.uint8, device="cuda"))
    call = lambda b, **x: dcp.dcp_kv8_decode_attn(w.kind, q, c, s, bt, sl, w.dcp_size, w.interleave, w.scale, Lq,   # noqa: E731
                                                  w.head_dim_v, **b, **x)
    first, other = new(), new()
    call(first)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    call(other, stream=side)                            # two streams at once
    call(first)
    torch.cuda.synchronize()
    assert torch.equal(first["partial_out"], other["partial_out"]) and torch.equal(first["lse"], other["lse"])
    with torch.cuda.stream(side):
        call(other)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call(other)
    for shorter in (0, 37, 150):
        sl.copy_(torch.clamp(inst.seq_lens - shorter, min=Lq))
        other["partial_out"].fill_(9.0)
        graph.replay()
        call(first)
        torch.cuda.synchronize()
        assert torch.equal(first["partial_out"], other["partial_out"]) and torch.equal(first["lse"], other["lse"])


@pytest.mark.parametrize("name,Lq,kw", [("qwen_gqa", 1, dict(batch=1, num_q_heads=16, num_kv_heads=1, lengths=("fixed", 700), dcp_size=1)),
                                        ("qwen_gqa", 4, dict(batch=2, num_q_heads=8, num_kv_heads=1, lengths=("fixed", 700), dcp_size=1)),
                                        ("qwen_gqa", 9, dict(batch=1, num_q_heads=16, num_kv_heads=1, lengths=("fixed", 700), dcp_size=1)),
                                        ("tiny_gqa", 1, dict(batch=100, lengths=("uniform", 300, 400), dcp_size=1))])
def test_wait_runs_out_and_the_cta_unwinds(name, Lq, kw):
    """As for the other kernels: waits of 5 ms, and key tile 1 of every request is never loaded."""
    from context_decode_attention_paged_gb300 import binding as dcp
    hooks = dcp.raw_lib().dcp_testing_set_hooks
    hooks.restype, hooks.argtypes = None, [ctypes.c_ulonglong, ctypes.c_int32]
    inst, codes, scales, _ = K.kv8_case(name, Lq, **kw)
    hooks(5_000_000, 1)
    try:
        got = K.run_attn(inst, codes, scales)
    finally:
        hooks(0, -1)
    assert got["status"] == dcp.DCP_ERR_TIMEOUT
    assert np.isfinite(got["partial_out"]).all()
    got = K.run_attn(inst, codes, scales)
    assert got["status"] == dcp.DCP_OK
    K.check_attn(got, K.oracle_attn(inst, codes, scales), codes, scales)


# ---------------------------------------------------------------------------
# appends
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name,kw,n,rope,kdim", [("tiny_gqa", TC, 3, A.HALF, 64), ("qwen_gqa", TC, 150, dict(rot_dim=128), 128),
                                                  ("mla_32", dict(TC, num_q_heads=4), 40, A.LATENT, 512)])
def test_rows_of_special_and_of_huge_values(name, kw, n, rope, kdim):
    inst = H.build_instance(H.small(name, **kw))
    codes, scales = A._cache8(inst)

    def change(k, v, q):
        k[0, 1, ..., 3] = float("inf")
        k[1, 0, ..., 9] = float("nan")
        k[2, 2] *= 2.0 ** 90                     # squares past fp32's range
        q[2, 1] *= 2.0 ** 100
        if v is not None:
            v[0, 2, ..., 5], v[1, 1, ..., 6] = float("-inf"), float("nan")

    with np.errstate(all="ignore"):
        cache, sc, q_out, k, v, want_q = A._call("kv8", inst, n, rope, kdim, kdim if name != "mla_32" else 0, None, None, codes,
                                                 scales, change=change)
        A._check_codes(inst, codes, scales, cache, sc, k, v, None)
    A._near_bf16(orc.to_f64(q_out), want_q, "queries")


@pytest.mark.parametrize("which", ["norm", "kv8"])
@pytest.mark.parametrize("what", ["short", "count", "negative", "block"])
def test_bad_appends_are_skipped_and_reported(which, what):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small("tiny_gqa", batch=3, lengths=("uniform", 100, 300)))
    w = inst.w
    codes, scales = A._cache8(inst)
    n, lens, ql, table = 4, inst.seq_lens.clone(), torch.full((3,), 4, dtype=torch.int32), inst.block_tables.clone()
    if what == "short":
        lens[1] = 3
    elif what == "count":
        ql[1] = 5
    elif what == "negative":
        ql[1] = -1
    else:
        table[:, 1] = -5
    g = torch.Generator().manual_seed(2)
    k, v, q = (torch.randn((3, n, h, 64), generator=g).to(torch.bfloat16).cuda() for h in (2, 2, 8))
    cache = inst.kv_cache.cuda() if which == "norm" else torch.from_numpy(codes).cuda()
    sc = torch.from_numpy(scales).cuda()
    before, sc_before = cache.clone(), sc.clone()
    q_out = torch.full_like(q, 7.0)
    args = (k, v, cache) + ((sc,) if which == "kv8" else ())
    call = dcp.dcp_kv8_append if which == "kv8" else dcp.dcp_kv_cache_append_norm
    call("gqa", *args, table.cuda(), lens.cuda(), w.dcp_size, w.interleave, dcp.dcp_rope_table(64), q=q, q_out=q_out,
         q_lens=ql.cuda())
    assert dcp.dcp_get_last_device_status() == dcp.DCP_ERR_BOUNDS
    changed = (cache != before).flatten(2).any(-1)[0]                                  # [blocks]
    own = [set(inst.block_tables[:, b].flatten().tolist()) for b in range(3)]
    assert not any(bool(changed[x]) for x in own[1] - own[0] - own[2])
    assert any(bool(changed[x]) for x in own[0]) and any(bool(changed[x]) for x in own[2])
    if what != "block":
        assert (q_out[1] == 7.0).all()
    assert (q_out[0] != 7.0).any()
    assert torch.equal(sc[:, sorted(own[1] - own[0] - own[2])], sc_before[:, sorted(own[1] - own[0] - own[2])])


@pytest.mark.parametrize("which", ["norm", "kv8"])
@pytest.mark.parametrize("n", [1, 20, 150])
def test_appends_without_queries_on_another_stream_and_replayed(which, n):
    """Rows alone, and with queries, on a stream of their own and from a graph: the same bytes."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small("qwen_gqa", batch=2, num_q_heads=8, lengths=("uniform", 200, 400)))
    w = inst.w
    codes, scales = A._cache8(inst)
    g = torch.Generator().manual_seed(2)
    k, v, q = (torch.randn((2, n, h, 128), generator=g).to(torch.bfloat16).cuda() for h in (4, 4, 8))
    start = inst.kv_cache.cuda() if which == "norm" else torch.from_numpy(codes).cuda()
    wt, rt = torch.rand((128,)).cuda(), dcp.dcp_rope_table(128)
    table, lens = inst.block_tables.cuda(), inst.seq_lens.cuda()
    call = dcp.dcp_kv8_append if which == "kv8" else dcp.dcp_kv_cache_append_norm
    results = []
    for mode in ("plain", "rows", "stream", "graph"):
        cache, sc = start.clone(), torch.from_numpy(scales).cuda()
        q_out = torch.zeros_like(q)
        args = ("gqa", k, v, cache) + ((sc,) if which == "kv8" else ()) + (table, lens, w.dcp_size, w.interleave, rt)
        kw = dict(k_weight=wt, **({} if mode == "rows" else dict(q_weight=wt, q=q, q_out=q_out)))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        if mode == "stream":
            call(*args, **kw, stream=side)
        elif mode == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                call(*args, **kw)
            graph.replay()
            graph.replay()                     # (the second time the rows are there already: the same bytes)
        else:
            call(*args, **kw)
        torch.cuda.synchronize()
        results.append((cache, sc, q_out))
    for cache, sc, q_out in results[1:]:
        assert torch.equal(cache.view(torch.uint8), results[0][0].view(torch.uint8)) and torch.equal(sc, results[0][1])
    assert torch.equal(results[0][2], results[2][2]) and torch.equal(results[0][2], results[3][2])
    assert not results[1][2].any()


def test_a_batch_of_more_entries_than_threads():
    inst, codes, scales, _ = K.kv8_case("tiny_gqa", 1, batch=500, num_q_heads=4, num_kv_heads=1, dcp_size=4, interleave=2,
                                        lengths=("uniform", 1, 60))
    K.check_attn(K.run_attn(inst, codes, scales), K.oracle_attn(inst, codes, scales), codes, scales)


def test_far_and_negative_positions_in_both_layouts():
    inst = H.build_instance(H.small("tiny_gqa", batch=2, lengths=("fixed", 40)))
    for rope in (A.HALF, A.INTER):
        cache, _, q_out, k, v, want_q = A._call("norm", inst, 3, rope, 64, 64, None, [[2_000_000_000, -41, 5], [-2_000_000_000, 0, 7]])
        A._near_bf16(orc.to_f64(q_out), want_q, "queries")


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("name,kw,rope", [
    ("qwen_gqa", dict(batch=3, num_q_heads=16, num_kv_heads=2, lengths=("fixed", 400), dcp_size=2, interleave=16), dict(rot_dim=128)),
    ("tiny_gqa", dict(batch=4, lengths=("fixed", 300), dcp_size=2, interleave=1), A.HALF),
    ("mla_32", dict(batch=2, num_q_heads=4, lengths=("fixed", 200), dcp_size=2), A.LATENT),
])
def test_a_prompt_and_decode_steps_over_the_8_bit_cache(name, kw, rope, captured):
    """A prompt chunk, then decode steps (append, attention, merge), against the oracle on what the cache holds by its
    own reading back; the rows read back are the prepared ones to half a code's step."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small(name, **kw))
    w = inst.w
    gqa = w.kind == "gqa"
    steps, prompt = 4, int(inst.seq_lens[0]) - 4
    g = torch.Generator(device="cuda").manual_seed(11)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    row = (w.num_kv_heads, w.head_dim_qk) if gqa else (w.head_dim_qk,)
    shape = tuple(inst.kv_cache.shape)
    cache = torch.full(shape, 127, dtype=torch.uint8, device="cuda")                  # NaN wherever nothing is stored
    scales = torch.zeros((2, shape[1], shape[3]) if gqa else shape[:1], dtype=torch.uint8, device="cuda")
    table = inst.block_tables.cuda()
    lens = torch.full((w.batch,), prompt, dtype=torch.int32, device="cuda")
    rt = dcp.dcp_rope_table(**rope)
    dim = 512 if not gqa else w.head_dim_qk
    kw_, qw_ = torch.rand((dim,), generator=g, device="cuda") + 0.5, torch.rand((dim,), generator=g, device="cuda") + 0.5
    common = dict(k_weight=kw_, q_weight=qw_ if gqa else None)
    all_k, all_v = rand(w.batch, prompt, *row), rand(w.batch, prompt, *row) if gqa else None
    dcp.dcp_kv8_append(w.kind, all_k, all_v, cache, scales, table, lens, w.dcp_size, w.interleave, rt, k_weight=kw_)
    ks = [rand(w.batch, 1, *row) for _ in range(steps)]
    vs = [rand(w.batch, 1, *row) if gqa else None for _ in range(steps)]
    qs = [rand(w.batch, 1, w.num_q_heads, w.head_dim_qk) for _ in range(steps)]
    k, v, q = ks[0].clone(), None if vs[0] is None else vs[0].clone(), qs[0].clone()
    q_out = torch.empty_like(q)
    po = torch.empty((w.dcp_size, w.batch, 1, w.num_q_heads, w.head_dim_v), device="cuda")
    lse = torch.empty((w.dcp_size, w.batch, 1, w.num_q_heads), device="cuda")
    desc = dcp.desc_from_tensors(w.kind, q, cache, table, w.head_dim_v)
    ws = torch.empty((max(1, dcp.dcp_kv8_decode_attn_workspace_size(desc, w.dcp_size)),), dtype=torch.uint8, device="cuda")
    out = torch.empty((w.dcp_size, w.batch, 1, w.num_q_heads // w.dcp_size, w.head_dim_v), dtype=torch.bfloat16, device="cuda")

    def step():
        dcp.dcp_kv8_append(w.kind, k, v, cache, scales, table, lens, w.dcp_size, w.interleave, rt, q=q, q_out=q_out, **common)
        dcp.dcp_kv8_decode_attn(w.kind, q_out, cache, scales, table, lens, w.dcp_size, w.interleave, w.scale, 1, w.head_dim_v,
                                partial_out=po, lse=lse, workspace=ws)
        dcp.dcp_merge(po, lse, w.dcp_size, out=out, want_lse=False)

    graph = None
    for i in range(steps):
        lens += 1
        k.copy_(ks[i])
        q.copy_(qs[i])
        if gqa:
            v.copy_(vs[i])
        if captured and i >= 1:
            if graph is None:
                graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph, stream=side):
                    step()
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        S = prompt + i + 1
        rk, rv = dcp.dcp_kv8_read(w.kind, cache, scales, table, lens, S, w.dcp_size, w.interleave)
        rk, rv = orc.to_f64(rk), None if rv is None else orc.to_f64(rv)
        assert np.isfinite(rk).all()
        x = np.concatenate([orc.to_f64(all_k)] + [orc.to_f64(t) for t in ks[:i + 1]], axis=1)
        freqs = (tro.rope_freqs(64 if rope["rot_dim"] == 64 else 128, 1e4), rope.get("layout", "half"), rope.get("rot_offset", 0), 1.0)
        want = k8o.prepared(x, kw_.double().cpu().numpy(), 1e-6, [S] * w.batch, None, None, freqs)
        assert (np.abs(rk - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -14 * np.abs(want).max()).all()
        qq = orc.to_f64(q_out)
        o = np.zeros((w.batch, w.num_q_heads, w.head_dim_v))
        group = w.num_q_heads // w.num_kv_heads
        for b in range(w.batch):
            for h in range(w.num_q_heads):
                kk = rk[b, :, h // group] if gqa else rk[b]
                vv = rv[b, :, h // group] if gqa else rk[b][:, :w.head_dim_v]
                s = kk @ qq[b, 0, h] * w.scale
                p = np.exp(s - s.max())
                o[b, h] = p @ vv / p.sum()
        per = w.num_q_heads // w.dcp_size
        got = orc.to_f64(out).transpose(1, 0, 3, 2, 4).reshape(w.batch, w.num_q_heads, w.head_dim_v)
        vmax = np.abs(rv if gqa else rk).max()
        assert (np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * vmax).all(), (i, per)
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK
