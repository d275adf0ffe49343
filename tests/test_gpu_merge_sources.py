"""dcp_merge with sources that do not count: shards without keys, wherever they are and whatever their
partial rows hold.

Weights and sums are fp32 (a few times 2^-24 of the row), the output is rounded to bf16 once (2^-8 of
it): the bounds below are 2^-8 |ref| + 1e-5 max |partial| and, on the LSE, 1e-5."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import dcp_oracle as orc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from context_decode_attention_paged_gb300 import build
    build.build()


LIVE = [(1, [0]), (2, [0]), (2, [1]), (8, [0, 1]), (8, [7]), (8, [1, 4, 6]), (8, list(range(8))), (8, []), (32, [0]),
        (32, [31]), (32, [3, 4, 5, 17, 30]), (5, [4]), (16, [0, 2, 3, 8])]


@pytest.mark.parametrize("dv", [4, 64, 128, 132, 512])
@pytest.mark.parametrize("N,live", LIVE)
@pytest.mark.parametrize("trash", [0.0, float("nan"), float("inf")])
def test_shards_without_keys_do_not_count(N, live, dv, trash):
    from context_decode_attention_paged_gb300 import binding as dcp
    g = torch.Generator().manual_seed(N * 1000 + dv)
    po = torch.randn((N, 3, 2, N * 2, dv), generator=g)
    lse = torch.randn((N, 3, 2, N * 2), generator=g) * 3
    dead = [r for r in range(N) if r not in live]
    ref, ref_lse = orc.ref_merge(*(torch.where(torch.tensor([r in live for r in range(N)]).view(-1, *[1] * (t.dim() - 1)),
                                               t, torch.full_like(t, fill)).double().numpy()
                                   for t, fill in ((po, 0.0), (lse, -float("inf")))))
    po[dead], lse[dead] = trash, -float("inf")
    out, out_lse = dcp.dcp_merge(po.cuda(), lse.cuda(), N)
    out, out_lse = out.double().cpu().numpy(), out_lse.double().cpu().numpy()
    assert (np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-5 * 6).all()
    if live:
        assert (np.abs(out_lse - ref_lse) <= 1e-5).all()
    else:
        assert (out == 0).all() and (out_lse == -np.inf).all()


def test_rows_differ_in_the_shards_that_count():
    """Every subset of five shards in one call, a row each."""
    from context_decode_attention_paged_gb300 import binding as dcp
    N = 5
    g = torch.Generator().manual_seed(1)
    po, lse = torch.randn((N, 32, 1, N, 64), generator=g), torch.randn((N, 32, 1, N), generator=g)
    for b in range(32):
        for r in range(N):
            if not (b >> r) & 1:
                po[r, b], lse[r, b] = 0.0, -float("inf")
    ref, ref_lse = orc.ref_merge(po.double().numpy(), lse.double().numpy())
    for b in range(32):
        for r in range(N):
            if not (b >> r) & 1:
                po[r, b] = float("nan")
    out, out_lse = dcp.dcp_merge(po.cuda(), lse.cuda(), N)
    assert (np.abs(out.double().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-5 * 6).all()
    got = out_lse.double().cpu().numpy()
    some = ref_lse > -np.inf
    assert np.array_equal(got == -np.inf, ~some) and (np.abs(got[some] - ref_lse[some]) <= 1e-5).all()


@pytest.mark.parametrize("N", [1, 2, 5, 8, 31, 32])
@pytest.mark.parametrize("others", [-float("inf"), 0.5])
def test_a_nan_lse_makes_its_rows_nan_and_no_others(N, others):
    """The partials end with the last shard's rows: nothing lies behind them."""
    from context_decode_attention_paged_gb300 import binding as dcp
    g = torch.Generator().manual_seed(N)
    po = torch.randn((N, 2, 1, N * 2, 128), generator=g)
    lse = torch.full((N, 2, 1, N * 2), others)
    lse[N // 2, 1, 0, 1::2] = float("nan")
    lse[:, 0] = torch.randn((N, 1, N * 2), generator=g)
    clean = lse.clone()
    clean[:, 1, 0, 1::2] = -float("inf")
    ref, ref_lse = orc.ref_merge(po.double().numpy(), clean.double().numpy())
    out, out_lse = dcp.dcp_merge(po.cuda(), lse.cuda(), N)
    out, out_lse = out.double().cpu().numpy(), out_lse.double().cpu().numpy()
    hit = np.zeros(out_lse.shape, dtype=bool)
    hit[:, 1, 0, 1::2] = True
    assert np.isnan(out[hit]).all() and np.isnan(out_lse[hit]).all()
    assert (np.abs(out[~hit] - ref[~hit]) <= 2.0 ** -8 * np.abs(ref[~hit]) + 1e-5 * 6).all()
    got, want = out_lse[~hit], ref_lse[~hit]
    some = want > -np.inf
    assert np.array_equal(got == -np.inf, ~some) and (np.abs(got[some] - want[some]) <= 1e-5).all()
