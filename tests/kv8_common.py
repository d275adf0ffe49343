"""Shared pieces of the 8-bit cache's tests: seeded caches, calls and the oracle's answers."""

from __future__ import annotations

import numpy as np
import torch

import helpers as H
from oracle import dcp_oracle as orc
from oracle import kv8_oracle as k8o
from oracle import tree_oracle as tro


def kv8_case(name, Lq=1, q_lens=None, exps=(-6, -3), seed=17, std=None, **kw):
    """(instance, codes uint8, scales uint8, q_lens int32 or None): the workload with a cache of random codes
    and scales 2^e, e in [exps[0], exps[1]]."""
    inst = H.build_instance(H.small(name, q_len=Lq, **kw))
    rng = np.random.default_rng(seed)
    shape = tuple(inst.kv_cache.shape)
    codes = k8o.encode(rng.standard_normal(shape) * (28.0 if std is None else std))
    sshape = (2, shape[1], shape[3]) if inst.w.kind == "gqa" else (shape[0],)
    scales = (rng.integers(exps[0], exps[1] + 1, sshape) + 127).astype(np.uint8)
    return inst, codes, scales, None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32)


def chain(L):
    """The causal mask as packed words int32 [1][L][ceil(L / 32)]."""
    out = np.zeros((1, L, (L + 31) // 32), dtype=np.uint32)
    for i in range(L):
        for j in range(i + 1):
            out[0, i, j // 32] |= np.uint32(1 << (j % 32))
    return out.view(np.int32)


def oracle_attn(inst, codes, scales, q_lens=None):
    w = inst.w
    return tro.ref_tree(w.kind, orc.to_f64(inst.q), k8o.dequantise(codes, scales), inst.block_tables.numpy(),
                        inst.seq_lens.numpy(), chain(w.q_len), w.dcp_size, w.interleave, w.block_size, w.scale,
                        w.head_dim_v, None if q_lens is None else q_lens.tolist())


def run_attn(inst, codes, scales, q_lens=None, stream=None, types=("uint8", "uint8"), **kw):
    from context_decode_attention_paged_gb300 import binding as dcp
    w = inst.w
    on = lambda t: None if t is None else torch.as_tensor(t).cuda()   # noqa: E731
    q, bt, sl, ql = on(inst.q), on(inst.block_tables), on(inst.seq_lens), on(q_lens)
    c, s = on(codes).view(getattr(torch, types[0])), on(scales).view(getattr(torch, types[1]))
    torch.cuda.synchronize()
    po, lse = dcp.dcp_kv8_decode_attn(w.kind, q, c, s, bt, sl, w.dcp_size, w.interleave, w.scale, w.q_len, w.head_dim_v,
                                      q_lens=ql, stream=stream, **kw)
    out, out_lse = dcp.dcp_merge(po, lse, w.dcp_size, stream=stream)
    torch.cuda.synchronize()
    return {"partial_out": po.cpu().numpy(), "lse": lse.cpu().numpy(), "out": out.float().cpu().numpy(),
            "out_lse": out_lse.cpu().numpy(), "status": dcp.dcp_get_last_device_status(stream)}


def kind_of(inst):
    from context_decode_attention_paged_gb300 import binding as dcp
    return dcp.dcp_kv8_decode_attn_kernel_kind(
        dcp.desc_from_tensors(inst.w.kind, inst.q, inst.kv_cache, inst.block_tables, inst.w.head_dim_v), inst.w.dcp_size)


def check_attn(got, want, codes, scales, what=""):
    """Element by element.  A probability is rounded to fp16 once: 2^-11 of it, so 2^-11 max|v| of an output
    for weights that sum to 1; scores, exponentials and sums in fp32 (scores below 64: 2^-22 * 64 of a
    probability, a few times over) stay below another 2^-12.  The merged output is rounded to bf16 on top
    (2^-8 of it).  The LSE: fp32 scores and sums, 2^-22 * 64 and a few times 2^-24 |lse|: below 2e-4."""
    vals = k8o.dequantise(codes, scales)
    vmax = np.abs(vals[1] if vals.ndim == 5 else vals)
    vmax = vmax[np.isfinite(vmax)].max()
    for key, rel in (("partial_out", 0.0), ("out", 2.0 ** -8)):
        g, r = got[key].astype(np.float64), want[key]
        assert g.shape == r.shape
        nan = np.isnan(r)
        assert np.array_equal(np.isnan(g), nan), (what, key, "NaN pattern")
        err = np.abs(g - r)[~nan]
        tol = (2.0 ** -11 + 2.0 ** -12) * vmax + rel * np.abs(r[~nan])
        assert (err <= tol).all(), (what, key, float(err.max()), float(vmax))
    for key in ("lse", "out_lse"):
        g, r = got[key].astype(np.float64), want[key]
        assert np.array_equal(g == -np.inf, r == -np.inf) and np.array_equal(np.isnan(g), np.isnan(r)), (what, key)
        fin = np.isfinite(r)
        assert not fin.any() or np.abs(g[fin] - r[fin]).max() <= 2e-4, (what, key, float(np.abs(g[fin] - r[fin]).max()))


__all__ = ["kv8_case", "chain", "oracle_attn", "run_attn", "kind_of", "check_attn", "orc", "k8o", "tro"]
