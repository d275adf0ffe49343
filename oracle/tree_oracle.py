"""CPU oracle of the speculative-verify operators, in float64 numpy.

TEST INFRASTRUCTURE ONLY, as dcp_oracle: nothing in the product path imports it
and it shares no code or constants with the CUDA library.

Readings (the vLLM DCP blog's roadmap, "未來發展藍圖", names speculative decoding
with several drafted tokens; its chain form is ``dcp_oracle``'s causal query):
* request b holds n_b nodes in its last n_b positions, node i at S_b - n_b + i;
* row i sees every position below S_b - n_b, and node j where its mask says so;
* a row that sees nothing, and every row i >= n_b, yields o = 0, lse = -inf;
* committing a path a_0 < a_1 < ... moves node a_k's row to S_b - n_b + k.
"""

from __future__ import annotations

import math

import numpy as np

from oracle import dcp_oracle as orc

NEG_INF = float("-inf")


def rope_freqs(rot_dim, base, scaling="none", factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0):
    """f_k, k < rot_dim / 2, in radians per position."""
    out = []
    for k in range(rot_dim // 2):
        b = base
        if scaling == "ntk":
            b = base * factor ** (rot_dim / (rot_dim - 2))
        f = 1.0 / b ** (2 * k / rot_dim)
        if scaling == "linear":
            f = f / factor
        if scaling == "yarn":
            def at(turns):
                return rot_dim * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
            lo, hi = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rot_dim - 1)
            r = min(max((k - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = f * (1 - r) + f / factor * r
        out.append(f)
    return np.array(out)


def rotate(x, position, freqs, layout="half", rot_offset=0, mscale=1.0):
    """Rows x [..., D] at one position."""
    y = np.array(x, dtype=np.float64)
    half = len(freqs)
    for k in range(half):
        i, j = (k, k + half) if layout == "half" else (2 * k, 2 * k + 1)
        i, j = i + rot_offset, j + rot_offset
        angle = math.fmod(float(position) * float(freqs[k]), 2 * math.pi)
        c, s = math.cos(angle) * mscale, math.sin(angle) * mscale
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def cell_of(table, b, t, interleave, dcp_size, block_size):
    """(block, slot) of position t of request b, by enumeration of its shard's tokens."""
    owner = (t // interleave) % dcp_size
    mine = orc.shard_token_lists(t + 1, interleave, dcp_size)[owner]
    j = len(mine) - 1
    assert mine[j] == t
    return int(table[owner][b][j // block_size]), j % block_size


def ref_append(kind, cache, new_k, new_v, q, table, seq_lens, dcp_size, interleave, block_size, freqs, layout, rot_offset,
               mscale, q_lens=None, offsets=None, q_out=None):
    """(cache, q_out) after the append; rows behind a request's q_lens keep what q_out holds."""
    cache = np.array(cache)
    q_out = None if q is None else np.zeros(q.shape) if q_out is None else np.array(q_out)
    B, L = new_k.shape[:2]
    for b in range(B):
        n = L if q_lens is None else int(q_lens[b])
        base = int(seq_lens[b]) - n
        for i in range(n):
            at = i if offsets is None else int(offsets[b if len(offsets) > 1 else 0][i])
            blk, slot = cell_of(table, b, base + i, interleave, dcp_size, block_size)
            row = rotate(new_k[b, i], base + at, freqs, layout, rot_offset, mscale)
            if kind == "gqa":
                cache[0, blk, slot], cache[1, blk, slot] = row, new_v[b, i]
            else:
                cache[blk, slot] = row
            if q is not None:
                q_out[b, i] = rotate(q[b, i], base + at, freqs, layout, rot_offset, mscale)
    return cache, q_out


def unpack(mask, L):
    """bool [.][L][L] of packed words int32 [.][L][ceil(L / 32)]."""
    words = np.asarray(mask).astype(np.int64) & 0xFFFFFFFF
    return np.stack([(words[..., j // 32] >> (j % 32)) & 1 for j in range(L)], axis=-1).astype(bool)


def ref_tree(kind, q, cache, table, seq_lens, mask, dcp_size, interleave, block_size, scale, dv, q_lens=None,
             rows=None):
    """partial_out [N][B][L][Hq][dv], lse [N][B][L][Hq] and the merged out / out_lse of dcp_oracle
    (``rows``: of these nodes alone, the others as empty)."""
    B, L, Hq, _ = q.shape
    sees = unpack(mask, L)
    o = np.zeros((dcp_size, B, L, Hq, dv))
    lse = np.full((dcp_size, B, L, Hq), NEG_INF)
    for b in range(B):
        S = int(seq_lens[b])
        n = L if q_lens is None else int(q_lens[b])
        lists = orc.shard_token_lists(S, interleave, dcp_size)
        for r, tokens in enumerate(lists):
            if not len(tokens):
                continue
            k, v = orc.gather_shard_kv(kind, cache, table[r][b], len(tokens), block_size)
            if kind == "mla":
                v = k[:, :, :dv]
            group = Hq // k.shape[1]
            for i in range(n) if rows is None else rows:
                keep = np.array([t < S - n or sees[b if len(sees) > 1 else 0, i, t - (S - n)] for t in tokens])
                if not keep.any():
                    continue
                for g in range(k.shape[1]):
                    heads = slice(g * group, (g + 1) * group)
                    x = scale * (q[b, i, heads] @ k[keep, g].T)
                    m = x.max(axis=1, keepdims=True)
                    w = np.exp(x - m)
                    o[r, b, i, heads] = w @ v[keep, g] / w.sum(axis=1, keepdims=True)
                    lse[r, b, i, heads] = m[:, 0] + np.log(w.sum(axis=1))
    out, out_lse = orc.ref_merge(o, lse)
    return {"partial_out": o, "lse": lse, "out": out, "out_lse": out_lse}


def ref_commit(kind, cache, table, seq_lens, L, accepted, num_accepted, dcp_size, interleave, block_size, q_lens=None):
    """(cache, new lengths)."""
    old, cache = np.array(cache), np.array(cache)
    lens = []
    for b in range(len(seq_lens)):
        n = L if q_lens is None else int(q_lens[b])
        base = int(seq_lens[b]) - n
        for k in range(int(num_accepted[b])):
            src = cell_of(table, b, base + int(accepted[b][k]), interleave, dcp_size, block_size)
            dst = cell_of(table, b, base + k, interleave, dcp_size, block_size)
            if kind == "gqa":
                cache[:, dst[0], dst[1]] = old[:, src[0], src[1]]
            else:
                cache[dst] = old[src]
        lens.append(base + int(num_accepted[b]))
    return cache, np.array(lens)
