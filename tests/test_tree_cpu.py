"""Speculative-verify operators without a GPU: the ABI's refusals, the frequency table, the tree
helper, and pins of the oracle they are compared with."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import helpers as H
import tree_common as T
from oracle import dcp_oracle as orc
from oracle import tree_oracle as tro


@pytest.fixture(scope="module")
def lib():
    from context_decode_attention_paged_gb300 import build
    build.build()
    from context_decode_attention_paged_gb300 import binding
    return binding


FAKE = ctypes.c_void_p(0x10000)   # 256-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x10008)


def _desc(lib, **kw):
    f = dict(kind="gqa", batch=2, q_len=4, num_q_heads=8, num_kv_heads=2, head_dim_qk=64, head_dim_v=64, block_size=16,
             num_blocks=64, max_local_blocks=32)
    f.update(kw)
    return lib.make_desc(**f)


def _rope(lib, **kw):
    f = dict(rot_dim=64, rot_offset=0, layout=0, scaling=0, original_max_position=0, mscale=1.0, base=1e4, factor=1.0,
             beta_fast=32.0, beta_slow=1.0)
    f.update(kw)
    return lib.DcpRopeDesc(**f)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def _tree(lib, d, q=FAKE, cache=FAKE, mask=FAKE, stride=0, n=2, inter=16, scale=0.1, po=FAKE, ws=FAKE, ws_bytes=0):
    return lib.raw_lib().dcp_tree_attn(ctypes.byref(d), q, cache, FAKE, FAKE, None, mask, stride, n, inter, scale, po,
                                       FAKE, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,extra", [
    (dict(batch=0), {}), (dict(q_len=0), {}), (dict(num_q_heads=7), {}), (dict(head_dim_v=32), {}), (dict(kind=5), {}),
    (dict(kind="mla", num_kv_heads=2), {}), ({}, dict(n=0)), ({}, dict(n=33)), ({}, dict(inter=0)),
    ({}, dict(scale=0.0)), ({}, dict(scale=math.nan)), ({}, dict(q=None)), ({}, dict(q=ODD)), ({}, dict(cache=ODD)),
    ({}, dict(mask=None)), ({}, dict(mask=ctypes.c_void_p(0x10002))), ({}, dict(stride=3)), ({}, dict(stride=-4)),
    (dict(q_len=33), dict(stride=65)), ({}, dict(po=ODD)),
])
def test_tree_attn_refuses(lib, kw, extra):
    assert _tree(lib, _desc(lib, **kw), **extra) == lib.DCP_ERR_INVALID_ARG


def test_tree_attn_refuses_shapes_it_has_no_kernel_for(lib):
    assert _tree(lib, _desc(lib, q_len=257)) == lib.DCP_ERR_UNSUPPORTED
    assert _tree(lib, _desc(lib, head_dim_qk=60, head_dim_v=60)) == lib.DCP_ERR_UNSUPPORTED
    d = _desc(lib, q_len=257)
    assert lib.dcp_tree_attn_workspace_size(d, 2) == 0 and lib.dcp_tree_attn_launches(d, 2) == 0
    assert lib.dcp_tree_attn_kernel_kind(d, 2) == lib.DCP_KERNEL_NONE


def test_tree_attn_refuses_a_small_or_misaligned_workspace(lib):
    d = _desc(lib, batch=1, max_local_blocks=2000, num_blocks=4000)
    need = lib.dcp_tree_attn_workspace_size(d, 2)
    assert need > 0 and lib.dcp_tree_attn_launches(d, 2) == 2
    assert _tree(lib, d, ws=None, ws_bytes=need) == lib.DCP_ERR_INVALID_ARG
    assert _tree(lib, d, ws_bytes=need - 1) == lib.DCP_ERR_INVALID_ARG
    assert _tree(lib, d, ws=ctypes.c_void_p(0x10010), ws_bytes=need) == lib.DCP_ERR_INVALID_ARG


def _append(lib, d, rope=None, steps=FAKE, k=FAKE, v=FAKE, q=None, q_out=None, strides=None, off=None, off_stride=0,
            cache=FAKE, n=2, inter=16):
    rope = rope or _rope(lib)
    s = None if strides is None else ctypes.byref(lib.DcpAppendStrides(*strides))
    return lib.raw_lib().dcp_kv_cache_append(ctypes.byref(d), ctypes.byref(rope), steps, k, v, q, s, q_out, off,
                                             off_stride, None, cache, FAKE, FAKE, n, inter, None)


@pytest.mark.parametrize("kw,extra", [
    ({}, dict(v=None)), (dict(kind="mla", num_kv_heads=1, head_dim_qk=576), {}),
    (dict(kind="mla", num_kv_heads=2), dict(v=None)), (dict(batch=0), {}), (dict(q_len=0), {}), (dict(block_size=0), {}),
    (dict(head_dim_qk=60), {}), ({}, dict(n=0)), ({}, dict(inter=0)), ({}, dict(k=None)), ({}, dict(k=ODD)),
    ({}, dict(v=ODD)), ({}, dict(cache=ODD)), ({}, dict(steps=None)), ({}, dict(steps=ctypes.c_void_p(0x10004))),
    ({}, dict(q=FAKE)), ({}, dict(q_out=FAKE)), ({}, dict(q=ODD, q_out=FAKE)), ({}, dict(q=FAKE, q_out=ODD)),
    (dict(num_q_heads=0), dict(q=FAKE, q_out=FAKE)), ({}, dict(off=FAKE, off_stride=3)),
    ({}, dict(off=FAKE, off_stride=-4)), ({}, dict(strides=(512, 4, 512, 128, 0, 0))),
    ({}, dict(strides=(512, 120, 512, 128, 0, 0))), ({}, dict(strides=(512, 128, 514, 128, 0, 0))),
    ({}, dict(strides=(-512, 128, 512, 128, 0, 0))),
    ({}, dict(q=FAKE, q_out=FAKE, strides=(512, 128, 512, 128, 4096, 1024))),           # in place, rows apart
    (dict(batch=1 << 16, q_len=1 << 16, max_local_blocks=1), {}),
])
def test_append_refuses(lib, kw, extra):
    assert _append(lib, _desc(lib, **kw), **extra) == lib.DCP_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=66), dict(rot_dim=32, rot_offset=40),
                                dict(rot_offset=-8), dict(layout=2), dict(mscale=math.inf)])
def test_append_refuses_rotations(lib, kw):
    assert _append(lib, _desc(lib), rope=_rope(lib, **kw)) == lib.DCP_ERR_INVALID_ARG


def _commit(lib, d, cache=FAKE, acc=FAKE, num=FAKE, most=3, lens=FAKE, n=2, inter=16):
    return lib.raw_lib().dcp_kv_cache_commit(ctypes.byref(d), cache, FAKE, FAKE, None, acc, num, most, lens, n, inter, None)


@pytest.mark.parametrize("kw,extra", [
    ({}, dict(cache=None)), ({}, dict(cache=ODD)), ({}, dict(acc=None)), ({}, dict(num=None)), ({}, dict(lens=None)),
    ({}, dict(most=0)), ({}, dict(n=0)), ({}, dict(inter=0)), (dict(kind=3), {}), (dict(q_len=0), {}),
    (dict(head_dim_qk=60), {}), (dict(kind="mla", num_kv_heads=2), {})])
def test_commit_refuses(lib, kw, extra):
    assert _commit(lib, _desc(lib, **kw), **extra) == lib.DCP_ERR_INVALID_ARG


def test_commit_refuses_paths_longer_than_it_takes(lib):
    assert _commit(lib, _desc(lib), most=257) == lib.DCP_ERR_UNSUPPORTED


def test_the_binding_refuses_tensors_that_are_not_on_the_gpu(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)            # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)          # noqa: E731
    rope = lib.dcp_rope_table(64, device="cpu")
    cache, table, lens = bf(2, 4, 16, 2, 64), i32(2, 1, 2), i32(1)
    for call in (lambda: lib.dcp_kv_cache_append("gqa", bf(1, 1, 2, 64), bf(1, 1, 2, 64), cache, table, lens, 2, 16, rope),
                 lambda: lib.dcp_tree_attn("gqa", bf(1, 1, 8, 64), cache, table, lens, i32(1, 1, 1), 2, 16, 0.1, 64),
                 lambda: lib.dcp_kv_cache_commit("gqa", cache, table, lens, 1, i32(1, 1), i32(1), 2, 16,
                                                 new_seq_lens=i32(1))):
        with pytest.raises(lib.DcpError, match="current device"):
            call()


def test_the_binding_refuses_shapes(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)            # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)          # noqa: E731
    cache, table, lens = bf(2, 4, 16, 2, 64), i32(2, 1, 2), i32(1)
    with pytest.raises(lib.DcpError, match="tree_mask is"):
        lib.dcp_tree_attn("gqa", bf(1, 33, 8, 64), cache, table, lens, i32(1, 33, 1), 2, 16, 0.1, 64)
    with pytest.raises(lib.DcpError, match="head dim"):
        lib.dcp_tree_attn("gqa", bf(1, 1, 8, 32), cache, table, lens, i32(1, 1, 1), 2, 16, 0.1, 64)
    with pytest.raises(lib.DcpError, match="block_tables is"):
        lib.dcp_tree_attn("gqa", bf(1, 1, 8, 64), cache, table, lens, i32(1, 1, 1), 4, 16, 0.1, 64)
    with pytest.raises(lib.DcpError, match="MLA cache is"):
        lib.dcp_kv_cache_commit("mla", cache, table, lens, 1, i32(1, 1), i32(1), 2, 16, new_seq_lens=i32(1))


# ---------------------------------------------------------------------------
# the frequency table
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kw", [
    dict(rot_dim=64), dict(rot_dim=2), dict(rot_dim=128, base=1e6), dict(rot_dim=64, scaling="linear", factor=8.0),
    dict(rot_dim=64, scaling="ntk", factor=4.0), dict(rot_dim=64, scaling="yarn", factor=40.0, original_max_position=4096),
    dict(rot_dim=96, scaling="yarn", factor=0.5, original_max_position=2048, beta_fast=16.0, beta_slow=2.0)])
def test_rope_table_holds_the_frequencies(lib, kw):
    """steps / 2^64 turns per position: the frequency to its 53 bits (the two powers round apart by a
    few times 2^-53 ln(base)), cut at 2^-64 of a turn."""
    table = lib.dcp_rope_table(device="cpu", **kw)
    want = tro.rope_freqs(kw["rot_dim"], kw.get("base", 1e4), kw.get("scaling", "none"), kw.get("factor", 1.0),
                          kw.get("original_max_position", 0), kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0))
    got = np.array([int(s) % (1 << 64) for s in table.steps.tolist()], dtype=np.float64) / 2.0 ** 64
    assert np.allclose(got * 2 * math.pi, want, rtol=1e-14, atol=2 * math.pi * 2.0 ** -64)
    yarn = kw.get("scaling") == "yarn" and kw["factor"] > 1
    assert table.desc.mscale == pytest.approx(0.1 * math.log(40.0) + 1 if yarn else 1.0)


def test_rope_table_of_given_frequencies(lib):
    """Whole turns drop out, negative frequencies turn the other way."""
    freqs = [0.0, 1.0, 2 * math.pi * 5.25, -0.5]
    table = lib.dcp_rope_table(8, inv_freq=freqs, device="cpu")
    got = [int(s) % (1 << 64) / 2.0 ** 64 for s in table.steps.tolist()]
    assert got == pytest.approx([0.0, 1 / (2 * math.pi), 0.25, 1 - 0.5 / (2 * math.pi)], abs=1e-15)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=3), dict(rot_dim=0), dict(base=1.0), dict(base=math.inf), dict(scaling=7), dict(scaling=1, factor=0.0),
    dict(scaling=2, rot_dim=2, factor=2.0), dict(scaling=3, factor=2.0), dict(scaling=3, factor=2.0,
                                                                           original_max_position=9, beta_slow=0.0),
    dict(scaling=3, factor=2.0, original_max_position=9, beta_fast=1.0), dict(layout=9), dict(mscale=math.nan)])
def test_rope_steps_refuses(lib, kw):
    out = (ctypes.c_uint64 * 512)()
    assert lib.raw_lib().dcp_rope_steps(ctypes.byref(_rope(lib, **kw)), None, out) == lib.DCP_ERR_INVALID_ARG


def test_rope_steps_refuses_frequencies_that_are_not_finite(lib):
    with pytest.raises(lib.DcpError):
        lib.dcp_rope_table(4, inv_freq=[1.0, math.inf], device="cpu")
    with pytest.raises(lib.DcpError, match="inv_freq is"):
        lib.dcp_rope_table(4, inv_freq=[1.0], device="cpu")


# ---------------------------------------------------------------------------
# the tree helper
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 70])
def test_tree_mask_is_the_ancestors(lib, L):
    par = T.random_parents(L, L, trees=3)
    mask, depth = lib.tree_mask(torch.from_numpy(par))
    assert mask.shape == (3, L, (L + 31) // 32) and mask.dtype == torch.int32 and depth.shape == (3, L)
    sees = tro.unpack(mask.numpy(), L)
    for t in range(3):
        for i in range(L):
            chain, j = {i}, i
            while par[t, j] >= 0:
                j = par[t, j]
                chain.add(j)
            assert set(np.nonzero(sees[t, i])[0]) == chain and depth[t, i] == len(chain) - 1
    one, _ = lib.tree_mask(par[0])
    assert torch.equal(one, mask[0])


@pytest.mark.parametrize("parents", [[0], [-1, 1], [-1, 2, 0], [-2]])
def test_tree_mask_refuses_children_before_parents(lib, parents):
    with pytest.raises(lib.DcpError):
        lib.tree_mask(parents)


# ---------------------------------------------------------------------------
# pins of the oracle
# ---------------------------------------------------------------------------

def test_rotation_keeps_lengths_and_relative_positions():
    """Rotations preserve a pair's length, and the product of two rotated rows depends on the
    difference of their positions alone."""
    rng = np.random.default_rng(0)
    x, y = rng.standard_normal((2, 3, 32))
    f = tro.rope_freqs(16, 100.0)
    for layout in ("half", "interleaved"):
        r = lambda v, p: tro.rotate(v, p, f, layout, 8)   # noqa: E731
        assert np.allclose((r(x, 77) ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose((r(x, 50) * r(y, 20)).sum(-1), (r(x, 1030) * r(y, 1000)).sum(-1))
        assert np.array_equal(r(x, 9)[..., :8], x[..., :8]) and np.array_equal(r(x, 9)[..., 24:], x[..., 24:])
        assert np.allclose(r(x, 0), x)


@pytest.mark.parametrize("name,kw", [("tiny_gqa", dict(batch=2, lengths=("uniform", 20, 90), dcp_size=2, interleave=3)),
                                     ("mla_32", dict(batch=1, num_q_heads=4, lengths=("fixed", 70), dcp_size=4, interleave=1))])
def test_the_tree_oracle_is_the_causal_oracle_on_a_chain(name, kw):
    inst, _, _ = T.tree_case(name, 6, **kw)
    got = T.oracle_tree(inst, T.pack(np.tril(np.ones((1, 6, 6), dtype=bool))))
    want = H.oracle_decode(inst)
    for key in ("partial_out", "out"):
        assert np.allclose(got[key], want[key], atol=1e-12)
    assert np.allclose(got["out_lse"], want["out_lse"], atol=1e-12)


def test_the_tree_oracle_on_a_path_is_the_decode_of_the_committed_cache():
    """A leaf's row equals the last token's decode after its path was committed: what the three
    operators mean together.  A planted mistake (the path off by one) does not."""
    L, path = 6, [0, 2, 5]
    inst, _, _ = T.tree_case("tiny_gqa", L, batch=1, lengths=("fixed", 50), dcp_size=2, interleave=3)
    w = inst.w
    sees = np.zeros((1, L, L), dtype=bool)
    sees[0, 5, path] = True
    leaf = T.oracle_tree(inst, T.pack(sees))["out"][:, :, 5]
    q, kv, bt, sl = H.oracle_inputs(inst)

    def decode(p):
        cache, lens = tro.ref_commit(w.kind, kv, bt, sl, L, [p], [3], w.dcp_size, w.interleave, w.block_size)
        return orc.ref_dcp_decode(w.kind, q[:, 5:6], cache, bt, lens, w.dcp_size, w.interleave, w.block_size, w.scale, 1,
                                  w.head_dim_v)["out"][:, :, 0]

    assert np.allclose(decode(path), leaf, atol=1e-12)
    assert not np.allclose(decode([0, 1, 5]), leaf, atol=1e-3)


def test_the_append_oracle_without_rotation_is_the_cache_write():
    inst = H.build_instance(H.small("tiny_gqa", batch=2, lengths=("uniform", 20, 90), dcp_size=2, interleave=3))
    w = inst.w
    k, v, _ = T.append_inputs(w, 3, 1)
    _, kv, bt, sl = H.oracle_inputs(inst)
    args = orc.to_f64(k), orc.to_f64(v)
    got, _ = tro.ref_append(w.kind, kv, *args, None, bt, sl, w.dcp_size, w.interleave, w.block_size, np.zeros(32), "half", 0,
                            1.0)
    want = orc.ref_kv_cache_write(w.kind, kv, *args, bt, sl, w.dcp_size, w.interleave, w.block_size, 3)
    assert np.array_equal(got, want)
