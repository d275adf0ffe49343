"""Thin ctypes binding over libdcp.so (declared in include/dcp.h).

Argument marshalling only: tensors are passed as raw device pointers together
with ``torch.cuda.current_stream()``; every step of the computation runs in the
library's CUDA kernels.  Output tensors are allocated here with torch when the
caller does not pass them (torch is used for device memory only).

Importing this module loads the library and raises ``ImportError`` when it has
not been built: there is no other implementation to fall back to.
"""

from __future__ import annotations

import ctypes
import dataclasses
import functools
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdcp.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libdcp.so is not built ({LIB_PATH}); run "
                      "`python -m context_decode_attention_paged_gb300.build`")

_lib = ctypes.CDLL(LIB_PATH)

DCP_OK, DCP_ERR_INVALID_ARG, DCP_ERR_UNSUPPORTED, DCP_ERR_CUDA, DCP_ERR_TIMEOUT, DCP_ERR_BOUNDS = range(6)
DCP_ATTN_GQA, DCP_ATTN_MLA = 0, 1
DCP_KERNEL_NONE, DCP_KERNEL_MLA_TC, DCP_KERNEL_GQA_TC, DCP_KERNEL_SIMT = range(4)
KINDS = {"gqa": DCP_ATTN_GQA, "mla": DCP_ATTN_MLA}
DCP_TREE_MAX_NODES = 256
DCP_COMMIT_MAX_ACCEPT = 256
DCP_ROPE_MAX_DIM = 1024
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class DcpAttnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "kind", "batch", "q_len", "num_q_heads", "num_kv_heads", "head_dim_qk", "head_dim_v",
        "block_size", "num_blocks", "max_local_blocks")]


class DcpRopeDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rot_dim", "rot_offset", "layout", "scaling", "original_max_position")] + [
        ("mscale", ctypes.c_float)] + [(n, ctypes.c_double) for n in ("base", "factor", "beta_fast", "beta_slow")]


class DcpAppendStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("k_batch", "k_token", "v_batch", "v_token", "q_batch", "q_token")]


_vp, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_lib.dcp_build_slot_map.restype = _i32
_lib.dcp_build_slot_map.argtypes = [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp]
_lib.dcp_decode_attn_workspace_size.restype = _sz
_lib.dcp_decode_attn_workspace_size.argtypes = [ctypes.POINTER(DcpAttnDesc), _i32]
_lib.dcp_decode_attn.restype = _i32
_lib.dcp_decode_attn.argtypes = [ctypes.POINTER(DcpAttnDesc), _vp, _vp, _vp, _vp, _i32, _i32,
                                 _f32, _i32, _vp, _vp, _vp, _sz, _vp]
_lib.dcp_decode_attn_noalloc.restype = _i32
_lib.dcp_decode_attn_noalloc.argtypes = [ctypes.POINTER(DcpAttnDesc), _vp, _vp, _vp, _vp, _i32,
                                         _i32, _f32, _i32, _vp, _vp, _vp]
_lib.dcp_kv_cache_write.restype = _i32
_lib.dcp_kv_cache_write.argtypes = [ctypes.POINTER(DcpAttnDesc), _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                                    _i32, _vp]
_lib.dcp_merge.restype = _i32
_lib.dcp_merge.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]
_lib.dcp_decode_attn_kernel_kind.restype = _i32
_lib.dcp_decode_attn_kernel_kind.argtypes = [ctypes.POINTER(DcpAttnDesc), _i32]
_lib.dcp_decode_attn_launches.restype = _i32
_lib.dcp_decode_attn_launches.argtypes = [ctypes.POINTER(DcpAttnDesc), _i32]
_lib.dcp_get_last_device_status.restype = _i32
_lib.dcp_get_last_device_status.argtypes = [_vp]
_i64 = ctypes.c_int64
_lib.dcp_rope_steps.restype = _i32
_lib.dcp_rope_steps.argtypes = [ctypes.POINTER(DcpRopeDesc), _vp, _vp]
_lib.dcp_kv_cache_append.restype = _i32
_lib.dcp_kv_cache_append.argtypes = [ctypes.POINTER(DcpAttnDesc), ctypes.POINTER(DcpRopeDesc), _vp, _vp, _vp, _vp,
                                     ctypes.POINTER(DcpAppendStrides), _vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32,
                                     _vp]
_lib.dcp_tree_attn_workspace_size.restype = _sz
_lib.dcp_tree_attn_workspace_size.argtypes = [ctypes.POINTER(DcpAttnDesc), _i32]
_lib.dcp_tree_attn.restype = _i32
_lib.dcp_tree_attn.argtypes = [ctypes.POINTER(DcpAttnDesc), _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _f32, _vp,
                               _vp, _vp, _sz, _vp]
_lib.dcp_tree_attn_kernel_kind.restype = _i32
_lib.dcp_tree_attn_kernel_kind.argtypes = [ctypes.POINTER(DcpAttnDesc), _i32]
_lib.dcp_tree_attn_launches.restype = _i32
_lib.dcp_tree_attn_launches.argtypes = [ctypes.POINTER(DcpAttnDesc), _i32]
_lib.dcp_kv_cache_commit.restype = _i32
_lib.dcp_kv_cache_commit.argtypes = [ctypes.POINTER(DcpAttnDesc), _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32,
                                     _vp]
_lib.dcp_status_string.restype = ctypes.c_char_p
_lib.dcp_status_string.argtypes = [_i32]


class DcpError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)}")


def status_string(code: int) -> str:
    return _lib.dcp_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without a Stream object around it (3 us a call less)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None, device=None):
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device() if device is None else device)
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(code: int, what: str):
    if code != DCP_OK:
        raise DcpError(code, what)


def make_desc(kind, batch, q_len, num_q_heads, num_kv_heads, head_dim_qk, head_dim_v,
              block_size, num_blocks, max_local_blocks) -> DcpAttnDesc:
    return DcpAttnDesc(KINDS.get(kind, kind), batch, q_len, num_q_heads, num_kv_heads,
                       head_dim_qk, head_dim_v, block_size, num_blocks, max_local_blocks)


def desc_from_tensors(kind, q, kv_cache, block_tables, head_dim_v) -> DcpAttnDesc:
    B, Lq, Hq, Dqk = q.shape
    if KINDS.get(kind, kind) == DCP_ATTN_GQA:
        _, nb, bs, Hkv, _ = kv_cache.shape
    else:
        nb, bs, _ = kv_cache.shape
        Hkv = 1
    return make_desc(kind, B, Lq, Hq, Hkv, Dqk, head_dim_v, bs, nb, block_tables.shape[2])


def dcp_build_slot_map(seq_lens, block_size, interleave, dcp_size, max_seq=None, stream=None):
    """Returns (local_seq_lens [N][B], local_num_blocks [N][B], shard_of, local_pos);
    the last two are [B][max_seq] when ``max_seq`` is given, else None."""
    B = seq_lens.shape[0]
    dev = seq_lens.device
    lsl = torch.empty((dcp_size, B), dtype=torch.int32, device=dev)
    lnb = torch.empty((dcp_size, B), dtype=torch.int32, device=dev)
    shard_of = local_pos = None
    if max_seq is not None:
        shard_of = torch.empty((B, max_seq), dtype=torch.int32, device=dev)
        local_pos = torch.empty((B, max_seq), dtype=torch.int32, device=dev)
    _check(_lib.dcp_build_slot_map(_ptr(seq_lens), B, block_size, interleave, dcp_size,
                                   _ptr(lsl), _ptr(lnb), _ptr(shard_of), _ptr(local_pos),
                                   int(max_seq or 0), _stream(stream)), "dcp_build_slot_map")
    return lsl, lnb, shard_of, local_pos


def dcp_decode_attn_workspace_size(desc: DcpAttnDesc, dcp_size: int) -> int:
    return int(_lib.dcp_decode_attn_workspace_size(ctypes.byref(desc), dcp_size))


def dcp_decode_attn_launches(desc: DcpAttnDesc, dcp_size: int) -> int:
    """Kernels one dcp_decode_attn call enqueues for this shape (0: invalid)."""
    return int(_lib.dcp_decode_attn_launches(ctypes.byref(desc), dcp_size))


def dcp_decode_attn_kernel_kind(desc: DcpAttnDesc, dcp_size: int) -> int:
    """Which kernel dcp_decode_attn runs for this shape (DCP_KERNEL_*)."""
    return int(_lib.dcp_decode_attn_kernel_kind(ctypes.byref(desc), dcp_size))


def dcp_decode_attn(kind, q, kv_cache, block_tables, seq_lens, dcp_size, interleave, scale,
                    causal_q_len, head_dim_v, partial_out=None, lse=None, workspace=None,
                    stream=None):
    """Per-shard partial outputs fp32 [N][B][Lq][Hq][Dv] and lse fp32 [N][B][Lq][Hq]."""
    desc = desc_from_tensors(kind, q, kv_cache, block_tables, head_dim_v)
    B, Lq, Hq, _ = q.shape
    dev = q.device
    if partial_out is None:
        partial_out = torch.empty((dcp_size, B, Lq, Hq, head_dim_v), dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty((dcp_size, B, Lq, Hq), dtype=torch.float32, device=dev)
    ws_bytes = dcp_decode_attn_workspace_size(desc, dcp_size)
    if workspace is None and ws_bytes:
        workspace = torch.empty((ws_bytes,), dtype=torch.uint8, device=dev)
    _check(_lib.dcp_decode_attn(ctypes.byref(desc), _ptr(q), _ptr(kv_cache), _ptr(block_tables),
                                _ptr(seq_lens), dcp_size, interleave, float(scale),
                                causal_q_len, _ptr(partial_out), _ptr(lse), _ptr(workspace),
                                workspace.numel() if workspace is not None else 0,
                                _stream(stream)), "dcp_decode_attn")
    return partial_out, lse


def dcp_decode_attn_noalloc(kind, q, kv_cache, block_tables, seq_lens, dcp_size, interleave,
                            scale, causal_q_len, head_dim_v, partial_out, lse, stream=None):
    """dcp_decode_attn without a workspace argument: split scratch comes from the
    library's built-in array (for callers that may not allocate device memory).
    Outputs must be passed in; calls overlapping on the GPU share that array."""
    desc = desc_from_tensors(kind, q, kv_cache, block_tables, head_dim_v)
    _check(_lib.dcp_decode_attn_noalloc(ctypes.byref(desc), _ptr(q), _ptr(kv_cache),
                                        _ptr(block_tables), _ptr(seq_lens), dcp_size, interleave,
                                        float(scale), causal_q_len, _ptr(partial_out), _ptr(lse),
                                        _stream(stream)), "dcp_decode_attn_noalloc")
    return partial_out, lse


def dcp_kv_cache_write(kind, new_k, new_v, kv_cache, block_tables, seq_lens, dcp_size, interleave,
                       stream=None):
    """Store the newest n_new tokens of every request in their shards' cache cells
    (kv_cache is written in place).  new_k/new_v: GQA [B][n_new][Hkv][D];
    MLA new_k [B][n_new][Dqk] and new_v None."""
    B, n_new = new_k.shape[0], new_k.shape[1]
    if KINDS.get(kind, kind) == DCP_ATTN_GQA:
        _, nb, bs, Hkv, D = kv_cache.shape
    else:
        nb, bs, D = kv_cache.shape
        Hkv = 1
    desc = make_desc(kind, B, n_new, Hkv, Hkv, D, D, bs, nb, block_tables.shape[2])
    _check(_lib.dcp_kv_cache_write(ctypes.byref(desc), _ptr(new_k), _ptr(new_v), _ptr(kv_cache),
                                   _ptr(block_tables), _ptr(seq_lens), dcp_size, interleave, n_new,
                                   _stream(stream)), "dcp_kv_cache_write")
    return kv_cache


def dcp_merge(partial_out, lse, dcp_size, out=None, out_lse=None, want_lse=True, stream=None):
    """out bf16 [N][B][Lq][Hq/N][Dv] (+ out_lse fp32 [N][B][Lq][Hq/N])."""
    N, B, Lq, Hq, Dv = partial_out.shape
    assert N == dcp_size
    dev = partial_out.device
    if out is None:
        out = torch.empty((N, B, Lq, Hq // N, Dv), dtype=torch.bfloat16, device=dev)
    if out_lse is None and want_lse:
        out_lse = torch.empty((N, B, Lq, Hq // N), dtype=torch.float32, device=dev)
    _check(_lib.dcp_merge(_ptr(partial_out), _ptr(lse), dcp_size, B, Lq, Hq, Dv, _ptr(out),
                          _ptr(out_lse), _stream(stream)), "dcp_merge")
    return out, out_lse


# ---------------------------------------------------------------------------
# Speculative verify: rotary append, drafted-tree attention, commit
# ---------------------------------------------------------------------------

_bf16, _int32 = torch.bfloat16, torch.int32


def _refuse(call, what):
    raise DcpError(DCP_ERR_INVALID_ARG, f"{call}: {what}")


def _check_tensors(call, dtype, device, *tensors):
    """The tensors (None: skipped) are of ``dtype`` on ``device``, and contiguous."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != device or not t.is_contiguous()):
            _refuse(call, f"a tensor is not a contiguous {dtype} tensor on the current device")


def _check_lens(call, batch, device, *tensors):
    """The tensors (None: skipped) are contiguous int32 [batch] on ``device``."""
    shape = (batch,)
    for t in tensors:
        if t is not None:
            if t.shape != shape:
                _refuse(call, "lengths are [batch]")
            if t.dtype is not _int32 or t.get_device() != device or not t.is_contiguous():
                _refuse(call, f"a tensor is not a contiguous {_int32} tensor on the current device")


@functools.lru_cache(maxsize=1024)
def _cached_desc(*fields):
    """Pointer to the descriptor of a shape (descriptors are never written)."""
    return ctypes.pointer(DcpAttnDesc(*fields))


@functools.lru_cache(maxsize=1024)
def _cached_strides(*fields):
    return ctypes.pointer(DcpAppendStrides(*fields))


def _cache_fields(call, kind, kv_cache, block_tables, batch, dcp_size):
    """(kind, Hkv, Dqk, block_size, num_blocks, max_local_blocks) from the cache's tensors."""
    kind = KINDS.get(kind, kind)
    shape = kv_cache.shape
    if kind == DCP_ATTN_GQA:
        if len(shape) != 5 or shape[0] != 2:
            _refuse(call, "a GQA cache is [2][blocks][block_size][Hkv][D]")
        _, nb, bs, hkv, dim = shape
    else:
        if len(shape) != 3:
            _refuse(call, "an MLA cache is [blocks][block_size][Dqk]")
        (nb, bs, dim), hkv = shape, 1
    tables = block_tables.shape
    if len(tables) != 3 or tables[0] != dcp_size or tables[1] != batch:
        _refuse(call, "block_tables is [dcp_size][batch][max_local_blocks]")
    return kind, hkv, dim, bs, nb, tables[2]


@dataclasses.dataclass(frozen=True)
class RopeTable:
    """A rotation (``desc``) and its frequency table on the device (``steps``, int64 [rot_dim / 2])."""
    desc: DcpRopeDesc
    steps: torch.Tensor


def dcp_rope_table(rot_dim, base=10000.0, layout="half", rot_offset=0, scaling="none", factor=1.0,
                   original_max_position=0, beta_fast=32.0, beta_slow=1.0, mscale=None, inv_freq=None,
                   device="cuda") -> RopeTable:
    """The rotation of dims [rot_offset, rot_offset + rot_dim) of every head, made once and passed
    to every dcp_kv_cache_append.  ``scaling``: "none", "linear", "ntk" or "yarn", by ``factor``;
    ``mscale`` multiplies the rotated values (None: 1, and 0.1 ln(factor) + 1 for "yarn" with
    factor > 1); ``inv_freq`` (a float64 sequence of rot_dim / 2) replaces base and scaling."""
    call = "dcp_rope_table"
    if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
        _refuse(call, "layout or scaling")
    if mscale is None:
        mscale = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0
    desc = DcpRopeDesc(rot_dim, rot_offset, ROPE_LAYOUTS[layout], ROPE_SCALINGS[scaling], int(original_max_position or 0),
                       mscale, base, factor, beta_fast, beta_slow)
    steps = torch.empty((max(rot_dim // 2, 1),), dtype=torch.int64)
    freqs = None
    if inv_freq is not None:
        freqs = torch.as_tensor(inv_freq, dtype=torch.float64).cpu().contiguous()
        if freqs.dim() != 1 or freqs.numel() != rot_dim // 2:
            _refuse(call, "inv_freq is [rot_dim / 2]")
    _check(_lib.dcp_rope_steps(ctypes.byref(desc), _ptr(freqs), _ptr(steps)), call)
    return RopeTable(desc, steps.to(device))


def tree_mask(parents):
    """(mask int32 [.][L][ceil(L / 32)], depths int32 [.][L]) on the host of trees given by their
    nodes' parents, an integer array [L] or [.][L] with -1 at a root and parents before children:
    every node sees itself and its ancestors.  For trees that are the same from step to step;
    move both to the device once and pass them as ``tree_mask`` and ``pos_offsets``."""
    parents = torch.as_tensor(parents)
    flat = parents.reshape(-1, parents.shape[-1]).tolist()
    words = (parents.shape[-1] + 31) // 32
    masks, depths = [], []
    for row in flat:
        seen, depth = [], []
        for i, p in enumerate(row):
            if not -1 <= p < i:
                _refuse("tree_mask", "a parent comes before its child, -1 at a root")
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[p] + 1 if p >= 0 else 0)
        words_of = [[(s >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for s in seen]
        masks.append([[w - (1 << 32) if w >> 31 else w for w in ws] for ws in words_of])
        depths.append(depth)
    shape = parents.shape[:-1]
    return (torch.tensor(masks, dtype=torch.int32).view(*shape, -1, words),
            torch.tensor(depths, dtype=torch.int32).view(*shape, -1))


def _row_strides(call, t, device, shape):
    """(batch, token) strides in elements of rows [batch][n][...], each token's row contiguous."""
    if t.dtype is not _bf16 or t.get_device() != device:
        _refuse(call, "rows are bfloat16 on the current device")
    if t.shape != shape:
        _refuse(call, f"rows are {shape}, got {tuple(t.shape)}")
    stride = t.stride()
    width = shape[-1]
    if len(shape) == 4:
        if stride[2] != width and shape[2] > 1:
            _refuse(call, "a token's row is contiguous")
        width *= shape[2]
    if stride[-1] != 1:
        _refuse(call, "a token's row is contiguous")
    # the stride of a dimension of one entry says nothing: the contiguous one stands for it
    token = stride[1] if shape[1] > 1 else width
    return (stride[0] if shape[0] > 1 else token * shape[1]), token


def dcp_kv_cache_append(kind, new_k, new_v, kv_cache, block_tables, seq_lens, dcp_size, interleave, rope, q=None,
                        q_out=None, q_lens=None, pos_offsets=None, stream=None):
    """Store new tokens' rows in their shards' cache cells, keys rotated, and rotate their queries.

    new_k/new_v bf16: GQA [B][n][Hkv][D], MLA new_k [B][n][Dqk] and new_v None; q [B][n][Hq][Dqk] or
    None.  A token's row is contiguous, tokens may lie apart (slices of a fused projection).
    ``rope``: a RopeTable.  ``q_lens`` int32 [B]: tokens of each request (None: n).  ``pos_offsets``
    int32 [B or 1][n]: a token's rotary position relative to the request's first new token (None:
    0, 1, 2, ...; a tree passes its depths).  kv_cache and q_out are written in place, rows behind a
    request's q_lens are left alone.  Returns (kv_cache, q_out); q_out may be q, and without one a
    zeroed tensor is allocated."""
    call = "dcp_kv_cache_append"
    B, n = new_k.shape[:2]
    kind, hkv, dim, bs, nb, max_lb = _cache_fields(call, kind, kv_cache, block_tables, B, dcp_size)
    gqa = kind == DCP_ATTN_GQA
    rows = (B, n, hkv, dim) if gqa else (B, n, dim)
    if (new_v is not None) != gqa:
        _refuse(call, "GQA takes new_v, MLA none")
    device = torch.cuda.current_device()
    _check_tensors(call, _bf16, device, kv_cache, None if q_out is q else q_out)
    _check_tensors(call, _int32, device, block_tables, pos_offsets)
    _check_lens(call, B, device, seq_lens, q_lens)
    steps = rope.steps
    if steps.get_device() != device:
        _refuse(call, "the rope table is not on the current device")
    if steps.dtype is not torch.int64 or not steps.is_contiguous() or 2 * steps.numel() < rope.desc.rot_dim:
        _refuse(call, "the rope table is not contiguous int64 [rot_dim / 2]")
    k_batch, k_token = _row_strides(call, new_k, device, rows)
    v_batch, v_token = _row_strides(call, new_v, device, rows) if gqa else (0, 0)
    hq, q_batch, q_token = hkv, 0, 0
    if q is not None:
        if q.dim() != 4:
            _refuse(call, "q is [batch][n][Hq][Dqk]")
        hq = q.shape[2]
        q_batch, q_token = _row_strides(call, q, device, (B, n, hq, dim))
        if q_out is None:
            with torch.cuda.stream(stream):
                q_out = torch.zeros((B, n, hq, dim), dtype=torch.bfloat16, device=q.device)
        elif q_out.shape != q.shape:
            _refuse(call, "q_out is shaped as q")
    offsets_stride = 0
    if pos_offsets is not None:
        if pos_offsets.dim() != 2 or pos_offsets.shape[1] != n or pos_offsets.shape[0] not in (1, B):
            _refuse(call, "pos_offsets is [batch or 1][n]")
        offsets_stride = n if pos_offsets.shape[0] == B else 0
    code = _lib.dcp_kv_cache_append(
        _cached_desc(kind, B, n, hq, hkv, dim, dim, bs, nb, max_lb), rope.desc, steps.data_ptr(), new_k.data_ptr(),
        new_v.data_ptr() if gqa else None, None if q is None else q.data_ptr(),
        _cached_strides(k_batch, k_token, v_batch, v_token, q_batch, q_token), None if q is None else q_out.data_ptr(),
        None if pos_offsets is None else pos_offsets.data_ptr(), offsets_stride,
        None if q_lens is None else q_lens.data_ptr(), kv_cache.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
        dcp_size, interleave, _stream(stream, device))
    if code != DCP_OK:
        raise DcpError(code, call)
    return kv_cache, q_out


def dcp_tree_attn_workspace_size(desc: DcpAttnDesc, dcp_size: int) -> int:
    return int(_lib.dcp_tree_attn_workspace_size(ctypes.byref(desc), dcp_size))


def dcp_tree_attn_launches(desc: DcpAttnDesc, dcp_size: int) -> int:
    """Kernels one dcp_tree_attn call enqueues for this shape (0: invalid)."""
    return int(_lib.dcp_tree_attn_launches(ctypes.byref(desc), dcp_size))


def dcp_tree_attn_kernel_kind(desc: DcpAttnDesc, dcp_size: int) -> int:
    """Which kernel dcp_tree_attn runs for this shape (DCP_KERNEL_*)."""
    return int(_lib.dcp_tree_attn_kernel_kind(ctypes.byref(desc), dcp_size))


def dcp_tree_attn(kind, q, kv_cache, block_tables, seq_lens, tree_mask, dcp_size, interleave, scale, head_dim_v,
                  q_lens=None, partial_out=None, lse=None, workspace=None, stream=None):
    """Attention of a tree of drafted tokens over the sharded cache: per-shard partial outputs fp32
    [N][B][Lq][Hq][Dv] and lse fp32 [N][B][Lq][Hq], for dcp_merge.

    seq_lens count the nodes, which sit in a request's last q_lens positions (None: Lq each).
    tree_mask int32 [B or 1][Lq][ceil(Lq / 32)]: bit j % 32 of word j / 32 of row i set where node i
    sees node j; the context is seen by all (``tree_mask`` of this module packs parents)."""
    call = "dcp_tree_attn"
    if q.dim() != 4:
        _refuse(call, "q is [batch][Lq][Hq][Dqk]")
    B, Lq, Hq, Dqk = q.shape
    kind, hkv, dim, bs, nb, max_lb = _cache_fields(call, kind, kv_cache, block_tables, B, dcp_size)
    words = (Lq + 31) // 32
    if dim != Dqk:
        _refuse(call, "q and the cache differ in their head dim")
    trees = tree_mask.shape
    if len(trees) != 3 or trees[0] not in (1, B) or trees[1] != Lq or trees[2] != words:
        _refuse(call, "tree_mask is [batch or 1][Lq][ceil(Lq / 32)]")
    device = torch.cuda.current_device()
    _check_tensors(call, _bf16, device, q, kv_cache)
    _check_tensors(call, _int32, device, block_tables, tree_mask)
    _check_lens(call, B, device, seq_lens, q_lens)
    desc = _cached_desc(kind, B, Lq, Hq, hkv, Dqk, head_dim_v, bs, nb, max_lb)
    if partial_out is None or lse is None or workspace is None:
        # allocated for the stream that the kernels run on
        with torch.cuda.stream(stream):
            if partial_out is None:
                partial_out = torch.empty((dcp_size, B, Lq, Hq, head_dim_v), dtype=torch.float32, device=q.device)
            if lse is None:
                lse = torch.empty((dcp_size, B, Lq, Hq), dtype=torch.float32, device=q.device)
            size = int(_lib.dcp_tree_attn_workspace_size(desc, dcp_size))
            if workspace is None and size:
                workspace = torch.empty((size,), dtype=torch.uint8, device=q.device)
    _check_tensors(call, torch.float32, device, partial_out, lse)
    if partial_out.numel() != dcp_size * B * Lq * Hq * head_dim_v or lse.numel() != dcp_size * B * Lq * Hq:
        _refuse(call, "partial_out is [N][B][Lq][Hq][Dv] and lse [N][B][Lq][Hq]")
    ws_bytes = 0
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            _refuse(call, "the workspace is not contiguous on the current device")
        ws_bytes = workspace.numel() * workspace.element_size()
    code = _lib.dcp_tree_attn(
        desc, q.data_ptr(), kv_cache.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(),
        None if q_lens is None else q_lens.data_ptr(), tree_mask.data_ptr(), Lq * words if trees[0] == B else 0, dcp_size,
        interleave, scale, partial_out.data_ptr(), lse.data_ptr(), None if workspace is None else workspace.data_ptr(),
        ws_bytes, _stream(stream, device))
    if code != DCP_OK:
        raise DcpError(code, call)
    return partial_out, lse


def dcp_kv_cache_commit(kind, kv_cache, block_tables, seq_lens, q_len, accepted, num_accepted, dcp_size, interleave,
                        q_lens=None, new_seq_lens=None, stream=None):
    """Move the cache rows of each request's accepted nodes (accepted int32 [B][max_accept], strictly
    increasing, the first num_accepted[b] of them) to the positions right behind its context, in
    place; returns the new lengths int32 [B] (``new_seq_lens`` may be seq_lens itself)."""
    call = "dcp_kv_cache_commit"
    if accepted.dim() != 2:
        _refuse(call, "accepted is [batch][max_accept]")
    B, max_accept = accepted.shape
    kind, hkv, dim, bs, nb, max_lb = _cache_fields(call, kind, kv_cache, block_tables, B, dcp_size)
    if new_seq_lens is None:
        with torch.cuda.stream(stream):
            new_seq_lens = torch.empty((B,), dtype=torch.int32, device=kv_cache.device)
    device = torch.cuda.current_device()
    _check_tensors(call, _bf16, device, kv_cache)
    _check_tensors(call, _int32, device, block_tables, accepted)
    _check_lens(call, B, device, seq_lens, q_lens, num_accepted, new_seq_lens)
    code = _lib.dcp_kv_cache_commit(
        _cached_desc(kind, B, q_len, hkv, hkv, dim, dim, bs, nb, max_lb), kv_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), None if q_lens is None else q_lens.data_ptr(), accepted.data_ptr(), num_accepted.data_ptr(),
        max_accept, new_seq_lens.data_ptr(), dcp_size, interleave, _stream(stream, device))
    if code != DCP_OK:
        raise DcpError(code, call)
    return new_seq_lens


def dcp_get_last_device_status(stream=None) -> int:
    return int(_lib.dcp_get_last_device_status(_stream(stream)))


def raw_lib():
    """The ctypes library handle (for tests of the raw C ABI)."""
    return _lib
