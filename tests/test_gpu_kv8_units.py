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
