"""Values at the ends of their ranges in the 8-bit cache's operators: what a formula makes of them whichever kernel, and
wherever a border between CTAs falls."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import helpers as H
import kv8_common as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from context_decode_attention_paged_gb300 import build
    build.build()


LONG = dict(batch=1, dcp_size=1, num_kv_heads=1, num_q_heads=8)


@pytest.mark.parametrize("S", [100, 3000, 60000])
@pytest.mark.parametrize("name,kw", [("tiny_gqa", LONG), ("tiny_gqa", dict(LONG, num_q_heads=32)),
                                     ("tiny_gqa", dict(LONG, block_size=48)), ("mla_32", dict(batch=1, dcp_size=1, num_q_heads=8))])
@pytest.mark.parametrize("at", [0.1, 0.95])
def test_a_nan_value_shows_however_light_its_part_of_the_shard(name, kw, S, at):
    """Keys of one tenth score 256 below the others: their weights are 0 in fp32, a part of the shard that holds them
    alone weighs 0 against the others, and a NaN among their values makes its dim NaN all the same."""
    inst, codes, scales, _ = K.kv8_case(name, 1, None, (0, 0), lengths=("fixed", S), **kw)
    w = inst.w
    gqa = w.kind == "gqa"
    one = int(K.k8o.encode([1.0])[0])
    d_k, v_dim = (w.head_dim_qk if gqa else 64), 5
    inst.q.zero_()
    inst.q[..., -d_k:] = 128.0 / (d_k * w.scale)       # scores of 128 (to bf16) for keys of 1, -128 for keys of -1
    (codes[0] if gqa else codes)[..., -d_k:] = one
    light = range(int(at * S) - S // 20, int(at * S) + S // 20)
    table = inst.block_tables.numpy()[0, 0]
    for t in light:
        cell = (table[t // w.block_size], t % w.block_size)
        (codes[0][cell] if gqa else codes[cell])[..., -d_k:] = one | 128
    t = int(at * S)
    cell = (table[t // w.block_size], t % w.block_size)
    if gqa:
        codes[1][cell][..., v_dim] = 127
    else:
        # (a latent row's values are its keys: the score of a row with NaN is NaN, so the whole output row is)
        codes[cell][..., v_dim] = 127
    want = K.oracle_attn(inst, codes, scales)
    assert np.isnan(want["out"][..., v_dim]).all()
    got = K.run_attn(inst, codes, scales)
    K.check_attn(got, want, codes, scales)


@pytest.mark.parametrize("dim", [512, 592])
def test_long_heads_on_the_cuda_cores(dim):
    inst, codes, scales, _ = K.kv8_case("tiny_gqa", 2, None, batch=2, head_dim_qk=dim, head_dim_v=dim, lengths=("uniform", 20, 200))
    got = K.run_attn(inst, codes, scales)
    assert got["status"] == 0
    K.check_attn(got, K.oracle_attn(inst, codes, scales), codes, scales)


@pytest.mark.parametrize("dim", [600, 768])
def test_heads_too_long_to_attend_are_refused_and_leave_the_next_call_alone(dim):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, codes, scales, _ = K.kv8_case("tiny_gqa", 1, None, batch=2, head_dim_qk=dim, head_dim_v=dim, lengths=("fixed", 30))
    with pytest.raises(dcp.DcpError) as e:
        K.run_attn(inst, codes, scales)
    assert e.value.code == dcp.DCP_ERR_UNSUPPORTED
    inst, codes, scales, _ = K.kv8_case("tiny_gqa", 1, None, batch=2, lengths=("fixed", 30))
    K.check_attn(K.run_attn(inst, codes, scales), K.oracle_attn(inst, codes, scales), codes, scales)


@pytest.mark.parametrize("byte", [0, 1, 2, 60, 86, 87, 127, 167, 168, 200, 236, 237, 238, 240, 245, 246, 247, 253, 254, 255])
@pytest.mark.parametrize("n,kw", [(3, dict()), (40, dict(block_size=64, interleave=64, dcp_size=1))])
def test_appends_into_blocks_of_any_scale(byte, n, kw):
    """Blocks whose scale byte is none that an append writes: it stays where the new rows are within 448 of its factor,
    else the earlier codes are rounded to the new one (of 255 they are NaN).  Powers of two make every step exact but the
    rounding to codes, so codes and scales are the oracle's bit for bit."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small("tiny_gqa", batch=2, lengths=("uniform", 150, 170), **kw))
    w = inst.w
    rng = np.random.default_rng(byte)
    shape = tuple(inst.kv_cache.shape)
    codes = rng.integers(0, 256, shape).astype(np.uint8)
    scales = np.full((2, shape[1], shape[3]), byte, dtype=np.uint8)
    table, lens = inst.block_tables, inst.seq_lens
    for at in (-12, -3, 4, 7, 9, 12, 60, 200):                   # largest magnitude of the rows over the factor, log2
        e = int(np.clip(byte - 127 + at, -130, 127))
        rows = [torch.from_numpy(rng.uniform(-1, 1, (2, n, shape[3], w.head_dim_qk)) * 2.0 ** (e - 1)).to(torch.bfloat16)
                for _ in range(2)]
        c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
        dcp.dcp_kv8_append("gqa", rows[0].cuda(), rows[1].cuda(), c, s, table.cuda(), lens.cuda(), w.dcp_size, w.interleave)
        assert dcp.dcp_get_last_device_status() == dcp.DCP_OK
        with np.errstate(all="ignore"):
            want_c, want_s, _ = K.k8o.ref_kv8_append("gqa", codes, scales, rows[0].double().numpy(), rows[1].double().numpy(),
                                                     table.numpy(), lens.tolist(), w.dcp_size, w.interleave, w.block_size)
        assert np.array_equal(s.cpu().numpy(), want_s), (at, np.unique(s.cpu().numpy()), np.unique(want_s))
        assert np.array_equal(c.cpu().numpy(), want_c), (at, int((c.cpu().numpy() != want_c).sum()))


@pytest.mark.parametrize("name,Lq,kw", [("tiny_gqa", 1, {}), ("qwen_gqa", 3, dict(block_size=32)), ("qwen_gqa", 9, {}),
                                        ("tiny_gqa", 2, dict(block_size=48)), ("mla_32", 1, dict(num_q_heads=8))])
@pytest.mark.parametrize("power", [100, 120, -100, -130])
def test_huge_and_tiny_queries_against_keys_of_zero(name, Lq, kw, power):
    """Scores are 0 whatever the query's and the block's factors are, and the rows the values' means: no product of the
    factors alone may leave fp32's range."""
    inst, codes, scales, _ = K.kv8_case(name, Lq, None, (40, 40) if power > 0 else (-40, -40), batch=2,
                                        lengths=("uniform", 200, 700), **kw)
    gqa = inst.w.kind == "gqa"
    keys, values = (codes[0], codes[1]) if gqa else (codes, None)
    keys[...] = np.where(np.random.default_rng(1).random(keys.shape) < 0.5, 0, 128)
    if gqa:
        scales[1] = 127
    signs = torch.rand(inst.q.shape, generator=torch.Generator().manual_seed(2)) < 0.5
    inst.q.copy_(torch.where(signs, -1.0, 1.0) * 2.0 ** power)
    want = K.oracle_attn(inst, codes, scales)
    assert np.isfinite(want["out"]).all()
    K.check_attn(K.run_attn(inst, codes, scales), want, codes, scales)


@pytest.mark.parametrize("dim,norm_dim", [(64, 64), (128, 96), (256, 256), (576, 512)])
@pytest.mark.parametrize("top", [63, 66, 100])
def test_norms_of_heads_that_span_many_binades(dim, norm_dim, top):
    """One dim whose square is at the end of fp32's range or past it, others far below it that large weights bring back:
    each is within a bf16 rounding of the formula (2^-8, and 2^-18 for fp32 sums) as far as fp32 holds x / root.
    That quotient is one fp32 product, whose smallest step is 2^-149: below 2^-126 it is off by up to half of that,
    2^-150, and the value by 2^-150 times the weight."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small("tiny_gqa", batch=2, lengths=("uniform", 20, 60), head_dim_qk=dim, head_dim_v=dim,
                                    num_q_heads=4, num_kv_heads=2))
    w = inst.w
    g = torch.Generator().manual_seed(dim)
    rows = lambda h: (1 + torch.rand((2, 3, h, dim), generator=g)) * 2.0 ** -60   # noqa: E731
    k, q = rows(2).to(torch.bfloat16), rows(4).to(torch.bfloat16)
    for t in (k, q):
        t[..., 3] = 2.0 ** top
        t[..., 5] *= 2.0 ** -18
    weight = torch.full((norm_dim,), 2.0 ** 60)
    weight[3] = 1.0
    cache, q_out = inst.kv_cache.cuda(), torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    dcp.dcp_kv_cache_append_norm("gqa", k.cuda(), k.cuda(), cache, inst.block_tables.cuda(), inst.seq_lens.cuda(), w.dcp_size,
                                 w.interleave, k_weight=weight.cuda(), q_weight=weight.cuda(), eps=1e-6, q=q.cuda(), q_out=q_out)
    want = K.k8o.norm(q.double().numpy(), weight.double().numpy(), 1e-6)
    want_k = K.k8o.norm(k.double().numpy(), weight.double().numpy(), 1e-6)
    got = q_out.double().cpu().numpy()
    step = np.zeros(dim)
    step[:norm_dim] = 2.0 ** -150 * weight.double().numpy()
    near = lambda g, r: (np.abs(g - r) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(r) + step).all()   # noqa: E731
    assert near(got, want)
    for b in range(2):
        for i in range(3):
            blk, slot = K.tro.cell_of(inst.block_tables.numpy(), b, int(inst.seq_lens[b]) - 3 + i, w.interleave, w.dcp_size,
                                      w.block_size)
            row = cache[0, blk, slot].double().cpu().numpy()
            assert near(row, want_k[b, i])
