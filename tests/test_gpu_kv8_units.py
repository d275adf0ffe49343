"""Work units of the 8-bit attention kernel: many short and empty ones in turn on a CTA, and the same answer every time."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import kv8_common as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from context_decode_attention_paged_gb300 import build
    build.build()


SHORT = [
    # (Lq, ragged q_lens, overrides): 16, 32 and 64 rows; a tile a unit, or none
    (1, False, dict(batch=700, lengths=("uniform", 1, 40), dcp_size=4, interleave=1)),
    (2, True, dict(batch=500, lengths=("uniform", 2, 60), dcp_size=8, interleave=4, num_q_heads=32)),
    (8, True, dict(batch=300, lengths=("uniform", 8, 300), dcp_size=4, interleave=16, num_q_heads=16)),
    (1, True, dict(batch=200, lengths=("uniform", 1, 500), dcp_size=2, interleave=1, head_dim_qk=128, head_dim_v=128)),
]


@pytest.mark.parametrize("Lq,ragged,kw", SHORT)
def test_many_short_and_empty_units_give_the_same_answer_every_time(Lq, ragged, kw):
    from context_decode_attention_paged_gb300 import binding as dcp
    q_lens = np.random.default_rng(4).integers(0, Lq + 1, kw["batch"]).tolist() if ragged else None
    inst, codes, scales, ql = K.kv8_case("tiny_gqa", Lq, q_lens, **kw)
    assert K.kind_of(inst) == dcp.DCP_KERNEL_GQA_TC
    got = K.run_attn(inst, codes, scales, ql)
    assert got["status"] == dcp.DCP_OK
    K.check_attn(got, K.oracle_attn(inst, codes, scales, ql), codes, scales)
    for _ in range(20):
        again = K.run_attn(inst, codes, scales, ql)
        assert again["status"] == dcp.DCP_OK
        for key in ("partial_out", "lse", "out"):
            assert np.array_equal(got[key], again[key]), key


@pytest.mark.parametrize("tile", [0, 1, 2])
@pytest.mark.parametrize("Lq,kw", [(1, dict(batch=150, lengths=("uniform", 1, 900), dcp_size=2, interleave=1)),
                                   (3, dict(batch=120, lengths=("uniform", 3, 900), dcp_size=2, num_q_heads=16)),
                                   (8, dict(batch=60, lengths=("uniform", 8, 700), dcp_size=1, num_q_heads=16)),
                                   (1, dict(batch=90, lengths=("uniform", 1, 900), dcp_size=1, head_dim_qk=128, head_dim_v=128))])
def test_waits_that_run_out_write_the_outputs_alone(Lq, kw, tile):
    """Waits of 5 ms, and one tile of every unit is never loaded: CTAs give up early or late in their units, ragged ones
    among them.  What lies around the outputs and the workspace stays; rows are the oracle's or 0 and -inf."""
    import ctypes

    from context_decode_attention_paged_gb300 import binding as dcp
    hooks = dcp.raw_lib().dcp_testing_set_hooks
    hooks.restype, hooks.argtypes = None, [ctypes.c_ulonglong, ctypes.c_int32]
    inst, codes, scales, _ = K.kv8_case("tiny_gqa", Lq, **kw)
    w = inst.w
    desc = dcp.desc_from_tensors(w.kind, inst.q, inst.kv_cache, inst.block_tables, w.head_dim_v)
    sizes = (w.dcp_size * w.batch * Lq * w.num_q_heads * w.head_dim_v, w.dcp_size * w.batch * Lq * w.num_q_heads,
             (dcp.dcp_kv8_decode_attn_workspace_size(desc, w.dcp_size) + 3) // 4)
    around = 1 << 16
    held = [torch.full((n + 2 * around,), 1234.5, dtype=torch.float32, device="cuda") for n in sizes]
    po, lse, ws = (t[around:around + n] for t, n in zip(held, sizes))
    shape = (w.dcp_size, w.batch, Lq, w.num_q_heads)
    kw = dict(partial_out=po.view(*shape, w.head_dim_v), lse=lse.view(*shape), workspace=ws.view(torch.uint8))
    hooks(5_000_000, tile)
    try:
        got = K.run_attn(inst, codes, scales, **kw)
    finally:
        hooks(0, -1)
    assert got["status"] == dcp.DCP_ERR_TIMEOUT
    for t in held:
        assert bool((t[:around] == 1234.5).all()) and bool((t[-around:] == 1234.5).all())
    want = K.oracle_attn(inst, codes, scales)
    gave_up = (got["lse"] == -np.inf) & (want["lse"] != -np.inf)
    assert gave_up.any() and (got["partial_out"][gave_up] == 0).all() and np.isfinite(got["partial_out"]).all()
    got = K.run_attn(inst, codes, scales, **kw)
    assert got["status"] == dcp.DCP_OK
    K.check_attn(got, want, codes, scales)


@pytest.mark.parametrize("S", [2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 4000])
@pytest.mark.parametrize("Lq", [1, 3])
def test_lengths_up_to_the_end_of_32_bits(S, Lq):
    """One request whose table names three blocks over and over, and at its end one whose slots behind the last token hold
    NaN.  A CTA of 444 sums 37,786 tiles or so one after the other: fp32 sums of n terms of like size are off by up to
    n / 2 2^-24 (a softmax thread's, n one a tile: 1.2e-3), where each addition truncates n / 2 2^-23.  In what portions
    the tensor cores add a tile's 128 products is theirs to choose; one by one, the most, n is 128 a tile: 0.29 of an
    output of up to 2.  (2.8e-2 was seen.)  The LSE is what tells that every key counts once."""
    from context_decode_attention_paged_gb300 import binding as dcp
    D, H, bs = 64, 8, 128
    rng = np.random.default_rng(3)
    codes = np.empty((2, 4, bs, 1, D), dtype=np.uint8)
    codes[0] = K.k8o.encode(rng.standard_normal((4, bs, 1, D)))
    codes[1] = K.k8o.encode(rng.uniform(1, 2, (4, bs, 1, D)))
    scales = np.full((2, 4, 1), 127, dtype=np.uint8)
    entries = -(-S // bs)
    table = (torch.arange(2 ** 24, dtype=torch.int32, device="cuda") % 3).view(1, 1, -1)
    table[0, 0, entries - 1] = 3
    last = S - (entries - 1) * bs                                # tokens of the last block
    codes[:, 3, last:] = 127
    q = torch.randn((1, Lq, H, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    c, s, lens = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), torch.tensor([S], dtype=torch.int32).cuda()
    po, lse = dcp.dcp_kv8_decode_attn("gqa", q.cuda(), c, s, table, lens, 1, 128, 0.125, Lq, D)
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK
    vals = np.nan_to_num(K.k8o.VALUES[codes])[:, :, :, 0]
    x = np.exp(0.125 * np.einsum("ihd,bkd->ihbk", q[0].double().numpy(), vals[0]))
    for i in range(Lq):
        full = np.bincount(np.arange(entries - 1) % 3, minlength=4).astype(np.float64)
        count = np.repeat(full[:, None], bs, axis=1)
        seen = last - (Lq - 1 - i)                               # (negative: in the block before)
        count[3, :max(seen, 0)] += 1
        if seen < 0:
            count[(entries - 2) % 3, bs + seen:] -= 1
        w = x[i] * count
        z = w.sum((1, 2))
        want = np.einsum("hbk,bkd->hd", w, vals[1]) / z[:, None]
        assert np.abs(lse[0, 0, i].double().cpu().numpy() - np.log(z)).max() <= 1.2e-3 + 2e-4
        assert np.abs(po[0, 0, i].double().cpu().numpy() - want).max() <= (1.2e-3 + 0.29 + 2.0 ** -11 + 2.0 ** -12) * 2
