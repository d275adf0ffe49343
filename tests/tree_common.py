"""Shared pieces of the speculative-verify tests: seeded trees and calls."""

from __future__ import annotations

import numpy as np
import torch

import helpers as H
from oracle import dcp_oracle as orc
from oracle import tree_oracle as tro


def random_parents(L, seed, trees=1):
    """[trees][L] parents, -1 at node 0 and now and then at another root."""
    rng = np.random.default_rng(seed)
    out = np.full((trees, L), -1, dtype=np.int64)
    for t in range(trees):
        for i in range(1, L):
            out[t, i] = rng.integers(-1 if rng.random() < 0.1 else 0, i)
    return out


def pack(sees):
    """bool [.][L][L] -> int32 words [.][L][ceil(L / 32)]."""
    L = sees.shape[-1]
    words = np.zeros((*sees.shape[:-1], (L + 31) // 32), dtype=np.uint32)
    for j in range(L):
        words[..., j // 32] |= sees[..., j].astype(np.uint32) << np.uint32(j % 32)
    return words.view(np.int32)


def tree_case(name, L, seed=3, shared=False, q_lens=None, mask="tree", **kw):
    """(instance of the workload with L nodes, mask int32, q_lens int32 or None).

    mask: "tree", "random" (any bits, rows of all zeros among them), "empty", "full"."""
    w = H.small(name, q_len=L, **kw)
    inst = H.build_instance(w)
    T = 1 if shared else w.batch
    if mask == "tree":
        par = random_parents(L, seed, T)
        sees = np.zeros((T, L, L), dtype=bool)
        for t in range(T):
            for i in range(L):
                sees[t, i, i] = True
                if par[t, i] >= 0:
                    sees[t, i] |= sees[t, par[t, i]]
    elif mask == "random":
        rng = np.random.default_rng(seed)
        sees = rng.random((T, L, L)) < 0.4
        sees[:, ::3] = False                     # rows that see no node
    else:
        sees = np.full((T, L, L), mask == "full")
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32)
    return inst, pack(sees), ql


def oracle_tree(inst, mask, q_lens=None):
    w = inst.w
    q, kv, bt, sl = H.oracle_inputs(inst)
    return tro.ref_tree(w.kind, q, kv, bt, sl, mask, w.dcp_size, w.interleave, w.block_size, w.scale, w.head_dim_v,
                        None if q_lens is None else q_lens.tolist())


def run_tree(inst, mask, q_lens=None, stream=None, **kw):
    from context_decode_attention_paged_gb300 import binding as dcp
    w = inst.w
    dev = torch.device("cuda:0")
    on = lambda t: None if t is None else torch.as_tensor(t).to(dev)   # noqa: E731
    q, kv, bt, sl = on(inst.q), on(inst.kv_cache), on(inst.block_tables), on(inst.seq_lens)
    m, ql = on(mask), on(q_lens)
    torch.cuda.synchronize()
    po, lse = dcp.dcp_tree_attn(w.kind, q, kv, bt, sl, m, w.dcp_size, w.interleave, w.scale, w.head_dim_v, q_lens=ql,
                                stream=stream, **kw)
    out, out_lse = dcp.dcp_merge(po, lse, w.dcp_size, stream=stream)
    torch.cuda.synchronize()
    return {"partial_out": po.cpu().numpy(), "lse": lse.cpu().numpy(), "out": out.float().cpu().numpy(),
            "out_lse": out_lse.cpu().numpy(), "status": dcp.dcp_get_last_device_status(stream)}


def cell(inst, b, t):
    """(block id, slot) that holds position t of request b."""
    w = inst.w
    return tro.cell_of(inst.block_tables.numpy(), b, t, w.interleave, w.dcp_size, w.block_size)


def append_inputs(w, n, seed, fused=True):
    """(new_k, new_v, q) bf16 on the CPU: slices of one fused row per token, or tensors of their own."""
    g = torch.Generator().manual_seed(seed)
    gqa = w.kind == "gqa"
    qw, kw_ = w.num_q_heads * w.head_dim_qk, w.num_kv_heads * w.head_dim_qk
    rows = torch.randn((w.batch, n, qw + kw_ * (2 if gqa else 1)), generator=g).to(torch.bfloat16)
    q = rows[..., :qw].unflatten(-1, (w.num_q_heads, w.head_dim_qk))
    k = rows[..., qw:qw + kw_]
    v = None
    if gqa:
        v = rows[..., qw + kw_:].unflatten(-1, (w.num_kv_heads, w.head_dim_qk))
        k = k.unflatten(-1, (w.num_kv_heads, w.head_dim_qk))
    if not fused:
        k, v, q = (None if x is None else x.contiguous() for x in (k, v, q))
    return k, v, q


def to_gpu(t):
    """On the GPU with the strides it has."""
    if t is None or t.is_contiguous():
        return None if t is None else t.cuda()
    buf = t.untyped_storage()
    flat = torch.empty((buf.nbytes() // t.element_size(),), dtype=t.dtype)
    flat.set_(buf, 0, flat.shape)
    return flat.cuda().as_strided(t.shape, t.stride(), t.storage_offset())


__all__ = ["random_parents", "pack", "tree_case", "oracle_tree", "run_tree", "cell", "append_inputs", "to_gpu", "orc",
           "tro"]


def oracle_rows(inst, mask, rows):
    """oracle_tree of some of the nodes: their queries and mask rows, over the whole cache."""
    w = inst.w
    q, kv, bt, sl = H.oracle_inputs(inst)
    return tro.ref_tree(w.kind, q, kv, bt, sl, mask, w.dcp_size, w.interleave, w.block_size, w.scale, w.head_dim_v,
                        rows=rows)
