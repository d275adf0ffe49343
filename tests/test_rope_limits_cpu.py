"""Limits of the rotary table and of the calls that take it, without a GPU."""

from __future__ import annotations

import ctypes
import os
import re

import pytest

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
