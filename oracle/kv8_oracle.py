"""CPU oracle of the 8-bit cache and of the normalised append, in float64 numpy.

TEST INFRASTRUCTURE ONLY, as dcp_oracle: nothing in the product path imports it
and it shares no code or constants with the CUDA library.

Readings:
* an e4m3 code seeeemmm stands for (-1)^s 2^(e - 7) (1 + m / 8), of exponent field
  0 for (-1)^s 2^-6 m / 8; seeee = s1111 with m = 7 is NaN, there is no infinity;
* a scale byte s stands for 2^(s - 127), 255 for NaN;
* the new rows of one block, KV head and K or V have the largest finite magnitude
  a; a block without earlier rows gets the smallest 2^e >= a / 112 (e in -40 .. 40),
  one with them keeps its scale while a <= 448 of it and else gets that same 2^e,
  the earlier codes rounded to it.
"""

from __future__ import annotations

import numpy as np

from oracle import tree_oracle as tro


def code_values():
    """The 256 codes' values."""
    out = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = 2.0 ** -6 * m / 8 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8)
        out[c] = np.nan if c & 127 == 127 else v
        if c & 128:
            out[c] = -out[c]
    return out


VALUES = code_values()


def scale_values(s):
    s = np.asarray(s, dtype=np.int64)
    return np.where(s == 255, np.nan, 2.0 ** (np.minimum(s, 254) - 127.0))


def encode(x):
    """Codes (uint8) nearest to x, ties to the even code; beyond 448 the largest, not finite NaN."""
    x = np.asarray(x, dtype=np.float64)
    pos = VALUES[:127]                                          # 0 .. 448, increasing
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - pos[lo], pos[hi] - a
    take_lo = (down < up) | ((down == up) & (lo % 2 == 0))
    code = np.where(a >= 448.0, 126, np.where(take_lo, lo, hi)).astype(np.uint8)
    code = np.where(np.signbit(x), code | 128, code).astype(np.uint8)
    return np.where(np.isfinite(x), code, 127).astype(np.uint8)


def exponent_for(a):
    e = -40
    while e < 40 and a > 112.0 * 2.0 ** e:
        e += 1
    return e


def dequantise(codes, scales):
    """The cache's values: codes uint8 GQA [2][blocks][bs][Hkv][D] (MLA [blocks][bs][D]), scales uint8."""
    f = scale_values(scales)
    f = f[:, :, None, :, None] if codes.ndim == 5 else f[:, None, None]
    return VALUES[codes] * f


def norm(x, weight, eps):
    """RMS norm of the first len(weight) dims of every row x [..., D]."""
    if weight is None:
        return np.array(x, dtype=np.float64)
    y = np.array(x, dtype=np.float64)
    n = len(weight)
    mean = sum(y[..., d] ** 2 for d in range(n)) / n
    y[..., :n] = y[..., :n] / np.sqrt(mean + eps)[..., None] * np.asarray(weight, dtype=np.float64)
    return y


def prepared(x, weight, eps, seq_lens, q_lens, offsets, rope):
    """Rows x [B][n][...][D] normalised and rotated; rope (freqs, layout, rot_offset, mscale) or None."""
    y = norm(x, weight, eps)
    if rope is not None:
        freqs, layout, rot_offset, mscale = rope
        for b in range(x.shape[0]):
            n = x.shape[1] if q_lens is None else int(q_lens[b])
            for i in range(n):
                at = i if offsets is None else int(offsets[b if len(offsets) > 1 else 0][i])
                y[b, i] = tro.rotate(y[b, i], int(seq_lens[b]) - n + at, freqs, layout, rot_offset, mscale)
    return y


def ref_append_norm(kind, cache, new_k, new_v, q, table, seq_lens, N, interleave, bs, rope, k_weight, q_weight, eps,
                    q_lens=None, offsets=None, q_out=None):
    """(cache, q_out) of the bf16 cache, before any rounding."""
    args = (eps, seq_lens, q_lens, offsets, rope)
    k = prepared(new_k, k_weight, *args)
    none = np.zeros(0)                                          # (nothing left to rotate)
    cache, _ = tro.ref_append(kind, cache, k, new_v, None, table, seq_lens, N, interleave, bs, none, "half", 0, 1.0, q_lens)
    if q is None:
        return cache, None
    out = np.array(q_out)
    y = prepared(q, q_weight, *args)
    for b in range(q.shape[0]):
        n = q.shape[1] if q_lens is None else int(q_lens[b])
        out[b, :n] = y[b, :n]
    return cache, out


def ref_kv8_append(kind, codes, scales, k, new_v, table, seq_lens, N, interleave, bs, q_lens=None):
    """(codes, scales, touched): rows k [B][n][...] as they are stored (after norm and rotation).  touched
    [(pool, block, head, first slot, {slot: row})]."""
    codes, scales = np.array(codes), np.array(scales)
    mla = kind == "mla"
    view_c = codes[None, :, :, None] if mla else codes
    view_s = scales[None, :, None] if mla else scales
    touched = []
    for pool, rows in enumerate([k] if mla else [k, new_v]):
        cells = {}
        for b in range(rows.shape[0]):
            n = rows.shape[1] if q_lens is None else int(q_lens[b])
            for i in range(n):
                blk, slot = tro.cell_of(table, b, int(seq_lens[b]) - n + i, interleave, N, bs)
                cells.setdefault(blk, {})[slot] = rows[b, i].reshape(-1, rows.shape[-1])
        for blk, held in cells.items():
            first = min(held)
            for h in range(view_c.shape[3]):
                new = {s: r[h] for s, r in held.items()}
                finite = [np.abs(r[np.isfinite(r)]).max(initial=0.0) for r in new.values()]
                a = max(finite)
                s = float(scale_values(view_s[pool, blk, h]))
                if first == 0 or not a <= 448.0 * s:             # (a scale of NaN holds nothing)
                    e = exponent_for(a)
                    old = VALUES[view_c[pool, blk, :first, h]] * (s / 2.0 ** e)
                    view_c[pool, blk, :first, h] = encode(old)
                    view_s[pool, blk, h] = 127 + e
                    s = 2.0 ** e
                for slot, r in new.items():
                    view_c[pool, blk, slot, h] = encode(r / s)
                touched.append((pool, blk, h, first, new))
    return codes, scales, touched
