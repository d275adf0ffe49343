"""Limits of the rotary table and of the calls that take it, without a GPU."""

from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

from test_tree_cpu import _append, _desc, _rope, lib    # noqa: F401  (the fixture builds the library)

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dcp.h")


@pytest.mark.parametrize("name", ["DCP_TREE_MAX_NODES", "DCP_COMMIT_MAX_ACCEPT", "DCP_ROPE_MAX_DIM"])
def test_the_binding_has_the_limits_of_the_header(lib, name):    # noqa: F811
    with open(HEADER) as f:
        assert int(re.search(rf"#define {name} (\d+)", f.read()).group(1)) == getattr(lib, name)


def test_rot_dim_ends_at_its_limit(lib):    # noqa: F811
    most = lib.DCP_ROPE_MAX_DIM
    assert lib.dcp_rope_table(most, device="cpu").steps.shape == (most // 2,)
    with pytest.raises(lib.DcpError):
        lib.dcp_rope_table(most + 2, device="cpu")
    d = _desc(lib, head_dim_qk=2 * most, head_dim_v=2 * most)
    assert _append(lib, d, rope=_rope(lib, rot_dim=most + 2)) == lib.DCP_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(scaling=1, factor=1e-310), dict(scaling=2, factor=1e-320, rot_dim=4),
                                dict(scaling=3, factor=1e-310, original_max_position=4096)])
def test_frequencies_past_the_range_of_a_double_are_refused(lib, kw):    # noqa: F811
    """A tiny factor divides a frequency to infinity (or takes the NTK base to 0): no rotation at all
    came of it before."""
    out = (ctypes.c_uint64 * 512)()
    assert lib.raw_lib().dcp_rope_steps(ctypes.byref(_rope(lib, **kw)), None, out) == lib.DCP_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(scaling=1, factor=1e-300), dict(scaling=2, factor=0.5),
                                dict(scaling=3, factor=0.25, original_max_position=4096)])
def test_factors_below_one_are_taken(lib, kw):    # noqa: F811
    out = (ctypes.c_uint64 * 512)()
    assert lib.raw_lib().dcp_rope_steps(ctypes.byref(_rope(lib, **kw)), None, out) == lib.DCP_OK


@pytest.mark.parametrize("steps", [torch.zeros(31, dtype=torch.int64), torch.zeros(32, dtype=torch.int32),
                                   torch.zeros(64, dtype=torch.int64)[::2], torch.zeros(0, dtype=torch.int64)])
def test_the_binding_refuses_a_table_that_is_not_the_rotations(lib, monkeypatch, steps):    # noqa: F811
    """A table made by hand, or for fewer dims: the kernel would read past its end."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)      # (where CPU tensors are)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)                 # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)               # noqa: E731
    rope = lib.RopeTable(lib.dcp_rope_table(64, device="cpu").desc, steps)
    with pytest.raises(lib.DcpError, match="rope table"):
        lib.dcp_kv_cache_append("gqa", bf(1, 1, 2, 64), bf(1, 1, 2, 64), bf(2, 4, 16, 2, 64), i32(2, 1, 2), i32(1), 2, 16,
                                rope)
