"""GPU parity of decode attention over the 8-bit cache (tolerances in kv8_common.check_attn)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import kv8_common as K
from oracle import kv8_oracle as k8o

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from context_decode_attention_paged_gb300 import build
    build.build()


CASES = [
    # (workload, Lq, q_lens, overrides)
    ("tiny_gqa", 1, None, {}),
    ("tiny_gqa", 1, None, dict(batch=3, lengths=("uniform", 1, 40), dcp_size=4, interleave=1)),        # empty shards
    ("tiny_gqa", 3, [3, 1, 0, 2], dict(batch=4, lengths=("uniform", 3, 700), interleave=3)),
    ("tiny_gqa", 5, None, dict(batch=2, lengths=("fixed", 5), interleave=1)),                          # queries alone
    ("tiny_gqa", 1, None, dict(batch=1, lengths=("fixed", 1))),
    ("tiny_gqa", 2, None, dict(batch=2, num_q_heads=32, num_kv_heads=1, block_size=8, lengths=("uniform", 100, 900))),
    ("tiny_gqa", 1, None, dict(batch=2, head_dim_qk=128, head_dim_v=128, block_size=32, lengths=("uniform", 100, 900))),
    ("tiny_gqa", 1, None, dict(batch=2, num_q_heads=3, num_kv_heads=3, dcp_size=1, lengths=("uniform", 100, 900))),
    ("tiny_gqa", 1, None, dict(batch=2, num_q_heads=14, num_kv_heads=2, dcp_size=2, block_size=64,
                               lengths=("uniform", 100, 900))),
    ("tiny_gqa", 1, None, dict(batch=130, lengths=("uniform", 1, 300))),
    ("qwen_gqa", 1, None, dict(batch=3, lengths=("uniform", 300, 3000))),
    ("qwen_gqa", 4, [4, 2, 1], dict(batch=3, lengths=("uniform", 300, 3000), interleave=1)),
    ("qwen_gqa", 1, None, dict(batch=2, block_size=256, lengths=("uniform", 300, 3000), dcp_size=2)),
    ("qwen_gqa", 9, None, dict(batch=2, block_size=16, lengths=("uniform", 300, 2000), dcp_size=2)),   # row tiles
    ("qwen_gqa", 33, [33, 20], dict(batch=2, num_q_heads=8, num_kv_heads=2, lengths=("uniform", 300, 2000), dcp_size=2)),
    ("qwen_gqa", 1, None, dict(batch=1, num_q_heads=16, num_kv_heads=1, lengths=("fixed", 30000), dcp_size=1)),
    ("qwen_gqa", 1, None, dict(batch=1, num_q_heads=64, num_kv_heads=8, lengths=("fixed", 20000), dcp_size=8,
                               interleave=1)),
    ("qwen_gqa", 1, None, dict(batch=2, block_size=48, lengths=("uniform", 300, 900))),                # CUDA cores
    ("tiny_gqa", 2, [1, 2], dict(batch=2, head_dim_qk=72, head_dim_v=72, lengths=("uniform", 30, 400))),
    ("mla_32", 2, [2, 1], dict(batch=2, num_q_heads=16, lengths=("uniform", 100, 600))),
]


@pytest.mark.parametrize("name,Lq,q_lens,kw", CASES)
def test_against_the_oracle(name, Lq, q_lens, kw):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst, codes, scales, ql = K.kv8_case(name, Lq, q_lens, **kw)
    got = K.run_attn(inst, codes, scales, ql)
    assert got["status"] == dcp.DCP_OK
    K.check_attn(got, K.oracle_attn(inst, codes, scales, ql), codes, scales)
