"""Latent rows in 8 bits attended by the bf16 kernel: the rows read back are a bf16 cache of one shard."""

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


@pytest.mark.parametrize("Lq,kw", [(1, dict(batch=2, num_q_heads=128, dcp_size=4, interleave=16, lengths=("uniform", 1, 900))),
                                   (4, dict(batch=3, num_q_heads=64, dcp_size=2, interleave=128, lengths=("uniform", 4, 700))),
                                   (1, dict(batch=8, num_q_heads=16, dcp_size=1, block_size=32, lengths=("uniform", 1, 300)))])
def test_rows_read_back_are_a_bf16_cache_of_one_shard(Lq, kw):
    """Rows come back exactly (4 bits times a power of two), so the outputs are within the two kernels' own accuracy of one
    another: of the bf16 one 2e-3 + 1e-2 |o|, LSE 1e-3, for values about 1; of this one 2^-11 and 2^-12 of the largest
    value, LSE 2e-4, as kv8_common.check_attn has it; each output is rounded to bf16 on top, 2^-8 of it twice."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, codes, scales, _ = K.kv8_case("mla_32", Lq, None, (-6, -5), std=20, **kw)
    w = inst.w
    got = K.run_attn(inst, codes, scales)
    K.check_attn(got, K.oracle_attn(inst, codes, scales), codes, scales)
    q, table, lens = inst.q.cuda(), inst.block_tables.cuda(), inst.seq_lens.cuda()
    n = -(-int(inst.seq_lens.max()) // w.block_size) * w.block_size
    rows, _ = dcp.dcp_kv8_read("mla", torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), table, lens, n,
                               w.dcp_size, w.interleave)
    own = torch.arange(w.batch * n // w.block_size, dtype=torch.int32, device="cuda").view(1, w.batch, -1)
    cache = rows.view(-1, w.block_size, w.head_dim_qk)
    desc = dcp.desc_from_tensors("mla", q, cache, own, w.head_dim_v)
    assert dcp.dcp_decode_attn_kernel_kind(desc, 1) == dcp.DCP_KERNEL_MLA_TC
    o, lse = dcp.dcp_decode_attn("mla", q, cache, own, lens, 1, w.block_size, w.scale, Lq, w.head_dim_v)
    out, out_lse = dcp.dcp_merge(o, lse, 1)
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK
    # [1][B][Lq][Hq][Dv] against the shards' head slices [N][B][Lq][Hq / N][Dv]
    here = np.moveaxis(got["out"], 0, 2).reshape(w.batch, Lq, w.num_q_heads, w.head_dim_v)
    there = out[0].float().cpu().numpy()
    vmax = np.abs(K.k8o.dequantise(codes, scales)).max()
    tol = 2e-3 + 1e-2 * np.abs(here) + (2.0 ** -11 + 2.0 ** -12) * vmax + 2 * 2.0 ** -8 * np.abs(here)
    assert (np.abs(here - there) <= tol).all(), float((np.abs(here - there) - tol).max())
    lse_here = np.moveaxis(got["out_lse"], 0, 2).reshape(w.batch, Lq, w.num_q_heads)
    assert np.abs(lse_here - out_lse[0].cpu().numpy()).max() <= 1e-3 + 2e-4
