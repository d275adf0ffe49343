"""The 8-bit cache and the normalised append without a GPU: refusals of the ABI, kernel kinds and workspaces, and pins of
the oracle they are compared with."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import helpers as H
import kv8_common as K
from oracle import dcp_oracle as orc
from oracle import kv8_oracle as k8o
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


def _norm(lib, dim=64, eps=1e-6, q=0x10000, k=0x10000):
    return lib.DcpNormDesc(dim, eps, q, k)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def _append(lib, which, d, rope="default", steps=FAKE, norm="default", k=FAKE, v=FAKE, q=FAKE, q_out=FAKE, strides=None,
            off=None, off_stride=0, cache=FAKE, scales=FAKE, table=FAKE, lens=FAKE, n=2, inter=16):
    rope = _rope(lib) if rope == "default" else rope
    norm = _norm(lib) if norm == "default" else norm
    head = (ctypes.byref(d), rope, steps, norm, k, v, q, strides, q_out, off, off_stride, None, cache)
    fn = lib.raw_lib().dcp_kv_cache_append_norm if which == "norm" else lib.raw_lib().dcp_kv8_append
    mid = () if which == "norm" else (scales,)
    return fn(*head, *mid, table, lens, n, inter, None)


@pytest.mark.parametrize("which", ["norm", "kv8"])
@pytest.mark.parametrize("kw,extra", [
    (dict(batch=0), {}), (dict(kind=7), {}), (dict(kind="mla", num_kv_heads=2), {}), (dict(head_dim_qk=60), {}),
    ({}, dict(n=0)), ({}, dict(inter=0)), ({}, dict(k=None)), ({}, dict(v=None)), ({}, dict(q=None)), ({}, dict(q_out=None)),
    ({}, dict(k=ODD)), ({}, dict(v=ODD)), ({}, dict(q=ODD)), ({}, dict(cache=None)), ({}, dict(cache=ODD)),
    ({}, dict(table=None)), ({}, dict(lens=None)), ({}, dict(rope=None)), ({}, dict(steps=None)),
    ({}, dict(off=FAKE, off_stride=3)), (dict(kind="mla", num_kv_heads=1), {}),
])
def test_appends_refuse(lib, which, kw, extra):
    assert _append(lib, which, _desc(lib, **kw), **extra) == lib.DCP_ERR_INVALID_ARG


@pytest.mark.parametrize("which", ["norm", "kv8"])
def test_appends_refuse_norms_and_rotations_out_of_range(lib, which):
    bad = lib.DCP_ERR_INVALID_ARG
    for dim in (0, 4, 12, 72, -8):
        assert _append(lib, which, _desc(lib), norm=_norm(lib, dim=dim)) == bad
    for eps in (0.0, -1.0, 1e-21, 1e21, math.inf, math.nan):
        assert _append(lib, which, _desc(lib), norm=_norm(lib, eps=eps)) == bad
    assert _append(lib, which, _desc(lib), norm=_norm(lib, q=0x10002)) == bad
    for rope in (dict(rot_dim=3), dict(rot_dim=66), dict(rot_offset=8), dict(layout=2), dict(mscale=math.inf)):
        assert _append(lib, which, _desc(lib), rope=_rope(lib, **rope)) == bad
    s = lib.DcpAppendStrides(4, 128, 128, 128, 512, 512)
    assert _append(lib, which, _desc(lib), strides=ctypes.byref(s)) == bad
    assert _append(lib, which, _desc(lib, head_dim_qk=776, head_dim_v=776)) == lib.DCP_ERR_UNSUPPORTED
    if which == "kv8":
        assert _append(lib, which, _desc(lib), scales=None) == bad


def _read(lib, d, cache=FAKE, scales=FAKE, table=FAKE, lens=FAKE, n=5, k=FAKE, v=FAKE, size=2, inter=16):
    return lib.raw_lib().dcp_kv8_read(ctypes.byref(d), cache, scales, table, lens, None, n, k, v, size, inter, None)


@pytest.mark.parametrize("kw,extra", [
    (dict(batch=0), {}), (dict(head_dim_qk=60), {}), ({}, dict(n=0)), ({}, dict(n=-3)), ({}, dict(size=0)),
    ({}, dict(inter=0)), ({}, dict(cache=None)), ({}, dict(cache=ODD)), ({}, dict(scales=None)), ({}, dict(table=None)),
    ({}, dict(lens=None)), ({}, dict(k=None, v=None)), ({}, dict(k=ODD)), ({}, dict(v=ODD)),
    (dict(kind="mla", num_kv_heads=1), {}), (dict(kind="mla", num_kv_heads=1), dict(k=None)),
    (dict(batch=1 << 20), dict(n=1 << 12)),
])
def test_read_refuses(lib, kw, extra):
    assert _read(lib, _desc(lib, **kw), **extra) == lib.DCP_ERR_INVALID_ARG


def _attn(lib, d, q=FAKE, cache=FAKE, scales=FAKE, table=FAKE, lens=FAKE, n=2, inter=16, scale=0.1, causal=4, po=FAKE,
          lse=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return lib.raw_lib().dcp_kv8_decode_attn(ctypes.byref(d), q, cache, scales, table, lens, None, n, inter, scale, causal,
                                             po, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,extra", [
    (dict(batch=0), {}), (dict(q_len=0), {}), (dict(num_q_heads=7), {}), (dict(head_dim_v=32), {}), (dict(kind=5), {}),
    (dict(kind="mla", num_kv_heads=2), {}), ({}, dict(n=0)), ({}, dict(n=33)), ({}, dict(inter=0)), ({}, dict(causal=3)),
    ({}, dict(scale=0.0)), ({}, dict(scale=math.nan)), ({}, dict(q=None)), ({}, dict(q=ODD)), ({}, dict(cache=ODD)),
    ({}, dict(scales=None)), ({}, dict(table=None)), ({}, dict(lens=None)), ({}, dict(po=ODD)), ({}, dict(lse=None)),
    ({}, dict(ws=None)), ({}, dict(ws=ctypes.c_void_p(0x10010))), ({}, dict(ws_bytes=100)),
])
def test_attn_refuses(lib, kw, extra):
    assert _attn(lib, _desc(lib, **kw), **extra) == lib.DCP_ERR_INVALID_ARG


def test_attn_kinds_workspaces_and_launches(lib):
    kind = lambda **kw: lib.dcp_kv8_decode_attn_kernel_kind(_desc(lib, **kw), 2)   # noqa: E731
    for kw in (dict(), dict(head_dim_qk=128, head_dim_v=128), dict(block_size=8), dict(block_size=128), dict(block_size=256),
               dict(q_len=100)):
        assert kind(**kw) == lib.DCP_KERNEL_GQA_TC
    for kw in (dict(head_dim_qk=72, head_dim_v=72), dict(block_size=48), dict(block_size=4),
               dict(kind="mla", num_kv_heads=1, head_dim_qk=576, head_dim_v=512)):
        assert kind(**kw) == lib.DCP_KERNEL_SIMT
    assert kind(batch=0) == lib.DCP_KERNEL_NONE
    d = _desc(lib)
    assert lib.dcp_kv8_decode_attn_launches(d, 2) == 2 and lib.dcp_kv8_decode_attn_workspace_size(d, 2) > 0
    assert lib.dcp_kv8_decode_attn_workspace_size(_desc(lib, batch=0), 2) == 0
    one = _desc(lib, batch=1, num_q_heads=4, num_kv_heads=1, max_local_blocks=1)
    assert lib.dcp_kv8_decode_attn_launches(one, 1) == 1          # one tile: nothing to join


# ---------------------------------------------------------------------------
# the oracle's pins
# ---------------------------------------------------------------------------

def test_codes_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    theirs = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(k8o.VALUES, theirs, equal_nan=True)
    g = np.random.default_rng(1)
    x = g.standard_normal(20000) * np.exp(g.uniform(-14, 7, 20000))
    x = np.concatenate([x, k8o.VALUES[:127], (k8o.VALUES[:126] + k8o.VALUES[1:127]) / 2, [0.0, -0.0, 2.0 ** -11]])
    x = torch.tensor(x).float().clamp(-448, 448)
    assert np.array_equal(k8o.encode(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert list(k8o.encode([1e9, -1e9, np.inf, np.nan])) == [126, 254, 127, 127]
    s = torch.arange(255, dtype=torch.uint8)
    assert np.array_equal(k8o.scale_values(s.numpy())[1:], s.view(torch.float8_e8m0fnu).double().numpy()[1:])


def test_exponent_for():
    for e in range(-40, 41):
        assert k8o.exponent_for(112.0 * 2.0 ** e) == e
        assert k8o.exponent_for(112.0 * 2.0 ** e * (1 + 1e-9)) == min(e + 1, 40)
    assert k8o.exponent_for(0.0) == -40 and k8o.exponent_for(1e300) == 40


def test_norm_against_torch():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((5, 3, 40), generator=g, dtype=torch.float64)
    w = torch.randn((32,), generator=g, dtype=torch.float64)
    want = torch.cat([torch.nn.functional.rms_norm(x[..., :32], (32,), w, 1e-5), x[..., 32:]], -1)
    assert np.abs(k8o.norm(x.numpy(), w.numpy(), 1e-5) - want.numpy()).max() < 1e-12


def test_append_oracle_keeps_grows_and_resets_scales():
    codes = np.full((1, 1, 4, 1, 8), 0x38, dtype=np.uint8).repeat(2, 0)          # 1.0 everywhere
    scales = np.full((2, 1, 1), 127, dtype=np.uint8)
    table, lens = np.zeros((1, 1, 1), dtype=np.int32), [3]
    run = lambda a, at: k8o.ref_kv8_append("gqa", codes, scales, np.full((1, 1, 1, 8), a), np.full((1, 1, 1, 8), a), table,   # noqa: E731
                                           [at + 1], 1, 4, 4)
    c, s, _ = run(448.0, 2)                      # fits: stays
    assert s[0, 0, 0] == 127 and (k8o.VALUES[c[0, 0, :2]] == 1.0).all() and (k8o.VALUES[c[0, 0, 2]] == 448.0).all()
    c, s, _ = run(449.0, 2)                      # does not: 2^3 >= 449 / 112, earlier rows / 8
    assert s[0, 0, 0] == 130 and (k8o.VALUES[c[0, 0, :2]] == 0.125).all() and (k8o.VALUES[c[0, 0, 3]] == 1.0).all()
    c, s, _ = run(2.0 ** -20, 0)                 # a new block: its scale starts over, rows behind stay
    assert s[0, 0, 0] == 127 - 26 and (k8o.VALUES[c[0, 0, 1:]] == 1.0).all()
    assert (k8o.dequantise(c, s)[0, 0, 0] == 2.0 ** -20).all()


def test_attention_oracle_is_the_causal_one_on_the_values():
    inst, codes, scales, _ = K.kv8_case("tiny_gqa", 3, None, lengths=("fixed", 40), batch=2)
    w = inst.w
    got = K.oracle_attn(inst, codes, scales)
    want = orc.ref_dcp_decode(w.kind, orc.to_f64(inst.q), k8o.dequantise(codes, scales), inst.block_tables.numpy(),
                              inst.seq_lens.numpy(), w.dcp_size, w.interleave, w.block_size, w.scale, 3, w.head_dim_v)
    assert np.abs(got["out"] - want["out"]).max() < 1e-12


def test_prepared_rows_rotate_as_the_append_oracle():
    inst = H.build_instance(H.small("tiny_gqa", batch=2, lengths=("fixed", 30)))
    w = inst.w
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 3, 2, 64)), rng.standard_normal((2, 3, 2, 64))
    freqs = tro.rope_freqs(64, 1e4)
    args = (inst.block_tables.numpy(), inst.seq_lens.numpy(), w.dcp_size, w.interleave)
    a, _ = tro.ref_append("gqa", orc.to_f64(inst.kv_cache), k, v, None, *args, w.block_size, freqs, "half", 0, 1.0)
    b, _ = k8o.ref_append_norm("gqa", orc.to_f64(inst.kv_cache), k, v, None, *args, w.block_size, (freqs, "half", 0, 1.0),
                               None, None, 1e-6)
    assert np.abs(a - b).max() < 1e-12


@pytest.mark.parametrize("dim,fits", [(584, True), (592, True), (600, False), (768, False)])
def test_heads_that_no_attention_kernel_takes_are_refused(lib, dim, fits):
    """The CUDA-core kernel's rows of long heads do not fit a CTA's shared memory: 384 bytes a dim and 2,304 for GQA."""
    assert (384 * dim + 2304 <= 227 * 1024) == fits
    d = _desc(lib, head_dim_qk=dim, head_dim_v=dim)
    kind = lib.DCP_KERNEL_SIMT if fits else lib.DCP_KERNEL_NONE
    assert lib.dcp_kv8_decode_attn_kernel_kind(d, 2) == lib.dcp_decode_attn_kernel_kind(d, 2) == kind
    assert lib.dcp_tree_attn_kernel_kind(d, 2) == kind
    assert (lib.dcp_kv8_decode_attn_launches(d, 2) > 0) == fits
    if not fits:
        assert lib.dcp_kv8_decode_attn_workspace_size(d, 2) == lib.dcp_decode_attn_workspace_size(d, 2) == 0
        assert _attn(lib, d) == lib.DCP_ERR_UNSUPPORTED


def test_shapes_past_the_cuda_core_kernels_grid_are_refused(lib):
    for kw in (dict(num_kv_heads=65536, num_q_heads=65536, head_dim_qk=8, head_dim_v=8),
               dict(q_len=1 << 20, num_q_heads=2, num_kv_heads=1, head_dim_qk=72, head_dim_v=72)):
        d = _desc(lib, **kw)
        assert lib.dcp_kv8_decode_attn_kernel_kind(d, 2) == lib.DCP_KERNEL_NONE
        assert _attn(lib, d, causal=d.q_len) == lib.DCP_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------
# what the header says of the query's split
# ---------------------------------------------------------------------------

def test_the_headers_bounds_of_the_query_split_hold():
    """A query row is scaled by a power of two so that its largest value lies in [128, 256), and each value becomes the sum
    of two codes: every bf16 value of that range, split so."""
    import os
    import re
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dcp.h")) as f:
        text = " ".join(f.read().replace("*", " ").split())
    said = re.search(r"two e4m3 terms, which is exact down to 2\^-(\d+) of the row's largest and an absolute error of at "
                     r"most 2\^-(\d+) of that below", text)
    exact, error = 2.0 ** -int(said.group(1)), 2.0 ** -int(said.group(2))
    x = torch.arange(0x4380, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()       # 0 up to 256
    assert x[-1] < 256.0 and bool((x[1:] > x[:-1]).all())
    hi = x.float().to(torch.float8_e4m3fn).double()
    rest = (x - hi - (x - hi).float().to(torch.float8_e4m3fn).double()).abs()
    inexact = x[rest > 0]
    # of a largest of 128, which is the least that rows are scaled to
    assert float(inexact.max()) < exact * 128 <= 2 * float(inexact.max())
    assert float(rest.max()) <= error * 128 < 2 * float(rest.max())
