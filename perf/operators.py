"""Cases of the speculative-verify operators: appending rotated rows to the sharded
paged cache, attention for a tree of drafted tokens over it, and committing the
accepted path.

``run`` computes a case either in its plain form (elementary torch operations in
32 bits; angles in 64) or, with ``own`` set, through the framework's calls.  A
case is a dict of plain values; sizes follow the repository's workloads (64 query
heads over 4 KV heads of 128 dims, 8 over 2 of 64, 128 heads over a 576-value
latent row) or are generic.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _gqa(**kw):
    c = dict(kind="gqa", heads=64, kv_heads=4, dim=128, dim_v=128, block=128, dcp=4, interleave=128)
    c.update(kw)
    return c


def _mla(**kw):
    c = dict(kind="mla", heads=128, kv_heads=1, dim=576, dim_v=512, block=128, dcp=8, interleave=128)
    c.update(kw)
    return c


def _rope(c, rot_dim, rot_offset=0, layout="half", base=10000.0, scaling="none", factor=1.0, original=0):
    c.update(rot_dim=rot_dim, rot_offset=rot_offset, layout=layout, base=base, scaling=scaling,
             factor=factor, original=original)
    return c


def listed():
    return [
        # a plain decode step: one new token per request, its query rotated on the way
        _rope(_gqa(name="append_step_gqa", op="append", batch=64, q_len=1, lo=8192, hi=32768, ragged=False), 128,
              base=1e6),
        # a decode step at high concurrency: long positions, the scaled rotation on the last 64 of 576 dims
        _rope(_mla(name="append_step_mla", op="append", batch=512, q_len=1, lo=4096, hi=200000, ragged=False), 64, 512,
              "interleaved", scaling="yarn", factor=40.0, original=4096),
        # drafted trees of different sizes, half of each head rotated, small blocks dealt token by token
        _rope(_gqa(name="append_tree_gqa", op="append", batch=33, q_len=24, heads=40, kv_heads=8, block=16, dcp=2,
                   interleave=1, lo=100, hi=9000, ragged=True, drafted=True), 64),
        # prompt chunks of up to 2048 tokens
        _rope(_gqa(name="append_prompt_gqa", op="append", batch=6, q_len=2048, lo=1, hi=60000, ragged=True), 128,
              scaling="linear", factor=4.0),
        # one request, a small model: what a call costs at the least
        _gqa(name="tree_tiny", op="tree", batch=1, q_len=8, heads=8, kv_heads=2, dim=64, dim_v=64, block=16, dcp=2,
             interleave=16, lo=1024, hi=1024, ragged=False, shared=True),
        # a batch without drafts: single tokens
        _gqa(name="tree_single", op="tree", batch=64, q_len=1, lo=1000, hi=16384, ragged=False, shared=True),
        # short drafts over long contexts: the cache's bytes bound it
        _gqa(name="tree_gqa_narrow", op="tree", batch=64, q_len=5, lo=8192, hi=32768, ragged=True, shared=False),
        # wide trees: 1024 query rows to each KV head
        _gqa(name="tree_gqa_wide", op="tree", batch=16, q_len=64, lo=8192, hi=32768, ragged=False, shared=False),
        # latent attention, a tree of eight for each of 32 requests
        _mla(name="tree_mla", op="tree", batch=32, q_len=8, lo=4096, hi=67000, ragged=True, shared=False),
        # one very long request, tokens dealt one by one
        _mla(name="tree_mla_long", op="tree", batch=1, q_len=32, interleave=1, lo=200000, hi=200000, ragged=False,
             shared=True),
        # the accepted paths of 64 requests
        _gqa(name="commit_gqa", op="commit", batch=64, q_len=32, accept=8, lo=8192, hi=32768, ragged=True),
        # and of 512, sixteen deep
        _mla(name="commit_mla", op="commit", batch=512, q_len=64, accept=16, lo=4096, hi=200000, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    limit = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["append", "tree", "tree", "commit"])
        if rng.random() < 0.6:
            kv = rng.choice([1, 2, 4, 8])
            dim = rng.choice([64, 128])
            c = _gqa(heads=8 * rng.randint(1, 10), kv_heads=kv, dim=dim, dim_v=dim)   # groups of 1 to 80 heads
            if rng.random() < 0.5:
                c.update(block=rng.choice([16, 32, 64, 128, 256]))
        else:
            c = _mla(heads=rng.choice([16, 32, 64, 128, 128, 128]))
            if rng.random() < 0.5:
                c.update(block=rng.choice([16, 32, 64, 128, 256]))
        c.update(op=op, dcp=rng.choice([1, 2, 4, 8]), ragged=rng.random() < 0.6)
        c.update(interleave=rng.choice([1, 3, 16, c["block"], 2 * c["block"]]))
        long = _log_int(rng, 500, 200000)
        c.update(lo=max(1, _log_int(rng, max(1, long // 40), long)), hi=long)
        if op == "append":
            c.update(batch=_log_int(rng, 1, 512), q_len=_log_int(rng, 1, 2048), drafted=rng.random() < 0.3)
            if c["batch"] * c["q_len"] > 16384 or c["drafted"] and c["q_len"] > 64:
                continue
            if c["kind"] == "mla":
                _rope(c, 64, 512)
            else:
                _rope(c, rng.choice([c["dim"], c["dim"] // 2]))
            c.update(layout=rng.choice(["half", "interleaved"]), base=rng.choice([1e4, 1e6]),
                     scaling=rng.choice(["none", "linear", "ntk", "yarn"]))
            if c["scaling"] != "none":
                c.update(factor=float(rng.choice([2, 4, 40])), original=4096)
        elif op == "tree":
            c.update(batch=_log_int(rng, 1, 128), q_len=_log_int(rng, 1, 64), shared=rng.random() < 0.4)
        else:
            q_len = _log_int(rng, 2, 64)
            c.update(batch=_log_int(rng, 1, 512), q_len=q_len, accept=rng.randint(1, min(q_len, 16)))
        # a pool of at most 24 GB, a cost within the largest listed case's
        if op == "tree" and _lengths(c).sum() * _row_bytes(c) > 24e9:
            continue
        if _cost(c) <= limit:
            return c


# ---------------------------------------------------------------------------
# what a case has to move and compute
# ---------------------------------------------------------------------------

def _row_bytes(c):
    return 2 * c["dim"] * c["kv_heads"] * (2 if c["kind"] == "gqa" else 1)


def _counts(c):
    """New tokens (tree nodes) of each request: all q_len, or spread over 1..q_len."""
    if not c["ragged"]:
        return np.full(c["batch"], c["q_len"], dtype=np.int64)
    return 1 + (np.arange(c["batch"], dtype=np.int64) * 7 + c["q_len"] - 1) % c["q_len"]


def _contexts(c):
    """Context length of each request before its new tokens: log-spaced over [lo, hi]."""
    n = c["batch"]
    x = np.linspace(1.0, 0.0, n) if n > 1 else np.ones(1)
    return np.rint(c["lo"] * (c["hi"] / c["lo"]) ** x).astype(np.int64)


def _lengths(c):
    return _contexts(c) + _counts(c)


def _accepts(c):
    # accepted nodes of each request, at most half of its tree
    n = _counts(c)
    return np.minimum(1 + (np.arange(c["batch"], dtype=np.int64) * 5) % c["accept"], (n + 1) // 2)


def work(c):
    n, S = _counts(c), _lengths(c)
    if c["op"] == "append":
        q_row = 2 * c["heads"] * c["dim"]
        values = c["heads"] * c["rot_dim"] + c["kv_heads"] * c["rot_dim"]
        return {"bytes": float(n.sum() * 2 * (_row_bytes(c) + q_row)), "flops": float(n.sum() * values * 3)}
    if c["op"] == "tree":
        io = 2 * c["heads"] * (c["dim"] + c["dim_v"])
        return {"bytes": float(S.sum() * _row_bytes(c) + n.sum() * io),
                "flops": float((2 * n * c["heads"] * (c["dim"] + c["dim_v"]) * S).sum())}
    return {"bytes": float(_accepts(c).sum() * 2 * _row_bytes(c) + 8 * c["batch"]), "flops": 0.0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _tables(c, S, first, rng):
    """Block tables int32 [dcp][B][max_blocks] (numpy) and the pool's block count.

    Blocks that hold a token at or behind ``first[b]`` are a request's own, dealt
    out of a shuffled pool; earlier ones (``first`` > 0: the call does not touch
    them) stand for a prefix that requests share and point at block 0."""
    N, I, bs, B = c["dcp"], c["interleave"], c["block"], c["batch"]
    held = lambda x, r: x // (I * N) * I + np.clip(x % (I * N) - r * I, 0, I)   # noqa: E731  tokens below x on shard r
    lo = np.stack([held(first, r) // bs for r in range(N)])
    hi = np.stack([(held(S, r) + bs - 1) // bs for r in range(N)])
    own_blocks = np.maximum(hi - lo, 0)
    total = int(own_blocks.sum()) + 1
    ids = rng.permutation(total - 1).astype(np.int32) + 1
    table = np.zeros((N, B, max(1, int(hi.max()))), dtype=np.int32)
    at = 0
    for r in range(N):
        for b in range(B):
            k = int(own_blocks[r, b])
            table[r, b, lo[r, b]:lo[r, b] + k] = ids[at:at + k]
            at += k
    return table, total


def _normal(shape, std, gen):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    for s in range(0, flat.numel(), 1 << 28):
        e = min(flat.numel(), s + (1 << 28))
        flat[s:e] = (torch.randn((e - s,), generator=gen, device=DEV) * std).to(torch.bfloat16)
    return out


def _trees(c, n, rng):
    """Random trees in the order of their nodes' parents: bit masks int32 [T][q_len][words] and
    node depths int32 [T][q_len]; T is 1 where the requests share one."""
    T = 1 if c.get("shared") else c["batch"]
    L = c["q_len"]
    words = (L + 31) // 32
    mask = np.zeros((T, L, words), dtype=np.uint32)
    depth = np.zeros((T, L), dtype=np.int32)
    for t in range(T):
        nodes = L if c.get("shared") else int(n[t])
        seen = [1]
        parents = [0] + sorted(int(rng.integers(0, i)) for i in range(1, nodes))
        for i in range(1, nodes):
            p = min(parents[i], i - 1)
            seen.append(seen[p] | 1 << i)
            depth[t, i] = depth[t, p] + 1
        for i in range(nodes):
            for w in range(words):
                mask[t, i, w] = seen[i] >> (32 * w) & 0xFFFFFFFF
    return mask.view(np.int32), depth


def prepare(case, seed):
    c = dict(case)
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    order = rng.permutation(c["batch"])                 # which request is how long
    n, ctx = _counts(c)[order], _contexts(c)[order]
    S = ctx + n
    first = np.zeros_like(S) if c["op"] == "tree" else ctx
    table, blocks = _tables(c, S, first, rng)
    shape = (blocks, c["block"], c["kv_heads"], c["dim"])
    std = 1.0 if c["kind"] == "gqa" else 0.5
    s = dict(case=c, n=n.tolist(), lengths=S.tolist(),
             cache=_normal((2, *shape) if c["kind"] == "gqa" else shape[:2] + shape[3:], std, gen),
             table=torch.from_numpy(table).to(DEV),
             seq_lens=torch.from_numpy(S.astype(np.int32)).to(DEV),
             q_lens=torch.from_numpy(n.astype(np.int32)).to(DEV) if c["ragged"] else None)
    B, L = c["batch"], c["q_len"]
    if c["op"] == "append":
        # the tokens' rows as a fused projection leaves them: queries, keys and values of a token side by side
        q_w, k_w = c["heads"] * c["dim"], c["kv_heads"] * c["dim"]
        wide = q_w + k_w * (2 if c["kind"] == "gqa" else 1)
        rows = _normal((B, L, wide), std, gen)
        s["q"] = rows[..., :q_w].unflatten(-1, (c["heads"], c["dim"]))
        k = rows[..., q_w:q_w + k_w]
        s["new_k"] = k.unflatten(-1, (c["kv_heads"], c["dim"])) if c["kind"] == "gqa" else k
        s["new_v"] = rows[..., q_w + k_w:].unflatten(-1, (c["kv_heads"], c["dim"])) if c["kind"] == "gqa" else None
        s["q_out"] = torch.zeros((B, L, c["heads"], c["dim"]), dtype=torch.bfloat16, device=DEV)
        s["depth"] = None
        if c.get("drafted"):
            s["depth"] = torch.from_numpy(_trees(c, n, rng)[1]).to(DEV)
        if own:
            from context_decode_attention_paged_gb300 import binding as dcp
            s["rope"] = dcp.dcp_rope_table(c["rot_dim"], base=c["base"], layout=c["layout"], rot_offset=c["rot_offset"],
                                           scaling=c["scaling"], factor=c["factor"], original_max_position=c["original"],
                                           device=DEV)
        else:
            s["freqs"], s["mscale"] = _frequencies(c)
    elif c["op"] == "tree":
        s["q"] = _normal((B, L, c["heads"], c["dim"]), 1.5 * std, gen)
        s["mask"] = torch.from_numpy(_trees(c, n, rng)[0]).to(DEV)
        s["scale"] = 1.0 / math.sqrt(c["dim"] if c["kind"] == "gqa" else 192)
        if own:
            from context_decode_attention_paged_gb300 import binding as dcp
            s["partial"] = torch.empty((c["dcp"], B, L, c["heads"], c["dim_v"]), device=DEV)
            s["lse"] = torch.empty((c["dcp"], B, L, c["heads"]), device=DEV)
            s["out"] = torch.empty((c["dcp"], B, L, c["heads"] // c["dcp"], c["dim_v"]), dtype=torch.bfloat16, device=DEV)
            desc = dcp.desc_from_tensors(c["kind"], s["q"], s["cache"], s["table"], c["dim_v"])
            size = dcp.dcp_tree_attn_workspace_size(desc, c["dcp"])
            s["workspace"] = torch.empty((max(size, 1),), dtype=torch.uint8, device=DEV)
    else:
        # accepted paths start at the root; deeper nodes lie behind the path's own slots, as they do in a
        # tree in breadth-first order that branches (and so a second pass over the same state changes nothing)
        take = _accepts(c)[order]
        path = np.zeros((B, c["accept"]), dtype=np.int32)
        for b in range(B):
            m = int(take[b])
            if m > 1:
                path[b, 1:m] = m + np.sort(rng.choice(int(n[b]) - m, m - 1, replace=False))
        s["path"] = torch.from_numpy(path).to(DEV)
        s["take"] = torch.from_numpy(take.astype(np.int32)).to(DEV)
        s["taken"] = take.tolist()
        s["new_lens"] = torch.empty((B,), dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _frequencies(c):
    """Inverse frequencies in 64 bits [rot_dim / 2] and the factor on the rotated values."""
    d, base, f = c["rot_dim"], c["base"], c["factor"]
    i = torch.arange(0, d, 2, dtype=torch.float64, device=DEV)
    if c["scaling"] == "ntk":
        base = base * f ** (d / (d - 2))
    freqs = base ** (-i / d)
    if c["scaling"] == "linear":
        return freqs / f, 1.0
    if c["scaling"] != "yarn":
        return freqs, 1.0
    turn = lambda beta: d * math.log(c["original"] / (beta * 2 * math.pi)) / (2 * math.log(base))   # noqa: E731
    lo, hi = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), d - 1)
    ramp = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return freqs / f * ramp + freqs * (1 - ramp), 0.1 * math.log(f) + 1.0 if f > 1 else 1.0


def _cells(s, b, t):
    """Rows of the flattened pool that hold positions t of requests b (tensors)."""
    c = s["case"]
    N, I, bs = c["dcp"], c["interleave"], c["block"]
    j = t // (I * N) * I + t % I
    return s["table"][t // I % N, b, j // bs].long() * bs + j % bs


def _valid(s):
    """(request, node) index pairs of the tokens that are there."""
    c = s["case"]
    b = torch.arange(c["batch"], device=DEV).view(-1, 1).expand(c["batch"], c["q_len"])
    i = torch.arange(c["q_len"], device=DEV).expand_as(b)
    if s["q_lens"] is None:
        return b.reshape(-1), i.reshape(-1), torch.full((c["batch"],), c["q_len"], device=DEV)
    n = s["q_lens"].long()
    live = i < n.view(-1, 1)
    return b[live], i[live], n


def _rotated(c, x, cos, sin):
    """The rotation of rows x [tokens][heads][dim], in 32 bits."""
    x = x.float()
    a, d = c["rot_offset"], c["rot_dim"]
    first, second = ((slice(a, a + d // 2), slice(a + d // 2, a + d)) if c["layout"] == "half"
                     else (slice(a, a + d, 2), slice(a + 1, a + d, 2)))
    y = x.clone()
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return y.to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    b, i, n = _valid(s)
    base = s["seq_lens"].long() - n
    at = i if s["depth"] is None else s["depth"].long()[b, i]
    angle = (base[b] + at).double().view(-1, 1) * s["freqs"]
    cos = (angle.cos() * s["mscale"]).float().unsqueeze(1)
    sin = (angle.sin() * s["mscale"]).float().unsqueeze(1)
    cell = _cells(s, b, base[b] + i)
    k = s["new_k"][b, i].view(-1, c["kv_heads"], c["dim"])
    if c["kind"] == "gqa":
        s["cache"][0].view(-1, c["kv_heads"], c["dim"])[cell] = _rotated(c, k, cos, sin)
        s["cache"][1].view(-1, c["kv_heads"], c["dim"])[cell] = s["new_v"][b, i]
    else:
        s["cache"].view(-1, 1, c["dim"])[cell] = _rotated(c, k, cos, sin)
    s["q_out"][b, i] = _rotated(c, s["q"][b, i], cos, sin)
    return s["cache"], s["q_out"]


def _plain_tree(s):
    c = s["case"]
    B, L, H, Hkv, Dv = c["batch"], c["q_len"], c["heads"], c["kv_heads"], c["dim_v"]
    out = torch.zeros((B, L, H, Dv), dtype=torch.bfloat16, device=DEV)
    node = torch.arange(L, device=DEV)
    seen = (s["mask"][:, :, node // 32] >> (node % 32) & 1).bool()       # [T][L][L]
    pools = s["cache"] if c["kind"] == "gqa" else (s["cache"], s["cache"][..., :Dv])
    for b in range(B):
        S, n = s["lengths"][b], s["n"][b]
        cell = _cells(s, b, torch.arange(S, device=DEV))
        k = pools[0].reshape(-1, Hkv, c["dim"])[cell].float().transpose(0, 1)      # [Hkv][S][dim]
        v = pools[1].flatten(0, 1).view(-1, Hkv, Dv)[cell].float().transpose(0, 1) if c["kind"] == "gqa" else k[..., :Dv]
        q = s["q"][b, :n].float().view(n, Hkv, H // Hkv, c["dim"]).permute(1, 0, 2, 3).reshape(Hkv, -1, c["dim"])
        x = torch.matmul(q, k.transpose(1, 2)).mul_(s["scale"])                   # [Hkv][n * group][S]
        hidden = ~seen[b if len(seen) > 1 else 0, :n, :n]
        x[..., S - n:].masked_fill_(hidden.repeat_interleave(H // Hkv, 0), -math.inf)
        p = x.sub_(x.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
        out[b, :n] = o.view(Hkv, n, H // Hkv, Dv).permute(1, 0, 2, 3).reshape(n, H, Dv).to(torch.bfloat16)
    N = c["dcp"]
    return out.view(B, L, N, H // N, Dv).permute(2, 0, 1, 3, 4).contiguous()


def _plain_commit(s):
    c = s["case"]
    take, n = s["take"].long(), s["q_lens"].long() if s["q_lens"] is not None else c["q_len"]
    base = s["seq_lens"].long() - n
    k = torch.arange(c["accept"], device=DEV).expand(c["batch"], -1)
    b = torch.arange(c["batch"], device=DEV).view(-1, 1).expand_as(k)
    live = k < take.view(-1, 1)
    b, k = b[live], k[live]
    to, of = _cells(s, b, base[b] + k), _cells(s, b, base[b] + s["path"].long()[b, k])
    for pool in (s["cache"] if c["kind"] == "gqa" else (s["cache"],)):
        rows = pool.flatten(0, 1)
        rows[to] = rows[of]
    return s["cache"], (base + take).int()


def _own(s):
    from context_decode_attention_paged_gb300 import binding as dcp
    c = s["case"]
    if c["op"] == "append":
        dcp.dcp_kv_cache_append(c["kind"], s["new_k"], s["new_v"], s["cache"], s["table"], s["seq_lens"], c["dcp"],
                                c["interleave"], s["rope"], q=s["q"], q_out=s["q_out"], q_lens=s["q_lens"],
                                pos_offsets=s["depth"])
        return s["cache"], s["q_out"]
    if c["op"] == "tree":
        dcp.dcp_tree_attn(c["kind"], s["q"], s["cache"], s["table"], s["seq_lens"], s["mask"], c["dcp"],
                          c["interleave"], s["scale"], c["dim_v"], q_lens=s["q_lens"], partial_out=s["partial"],
                          lse=s["lse"], workspace=s["workspace"])
        dcp.dcp_merge(s["partial"], s["lse"], c["dcp"], out=s["out"], want_lse=False)
        return s["out"]
    dcp.dcp_kv_cache_commit(c["kind"], s["cache"], s["table"], s["seq_lens"], c["q_len"], s["path"], s["take"], c["dcp"],
                            c["interleave"], q_lens=s["q_lens"], new_seq_lens=s["new_lens"])
    return s["cache"], s["new_lens"]


def run(s):
    if own:
        return _own(s)
    return {"append": _plain_append, "tree": _plain_tree, "commit": _plain_commit}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _slot(c, table, b, t):
    """(block, row) that holds position t of request b, one token at a time."""
    turn, rest = divmod(int(t), c["interleave"] * c["dcp"])
    shard, inside = divmod(rest, c["interleave"])
    local = turn * c["interleave"] + inside
    return int(table[shard, b, local // c["block"]]), local % c["block"]


def _exact_rotation(c, x, p):
    """Rows x (64 bits, [heads][dim]) at position p, as products of complex numbers."""
    d, f, base = c["rot_dim"], c["factor"], c["base"]
    if c["scaling"] == "ntk":
        base *= f ** (d / (d - 2))
    rate = np.array([base ** (-2.0 * i / d) for i in range(d // 2)])
    gain = 1.0
    if c["scaling"] == "linear":
        rate = rate / f
    if c["scaling"] == "yarn":
        at = [d * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
        share = np.clip((np.arange(d // 2) - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        rate = rate * (1 - share) + rate / f * share
        gain = 1.0 + 0.1 * math.log(f) if f > 1 else 1.0
    turn = gain * np.exp(1j * (p * rate))
    y = x.copy()
    part = x[:, c["rot_offset"]:c["rot_offset"] + d]
    z = part[:, :d // 2] + 1j * part[:, d // 2:] if c["layout"] == "half" else part[:, 0::2] + 1j * part[:, 1::2]
    z = z * turn
    r = np.empty_like(part)
    if c["layout"] == "half":
        r[:, :d // 2], r[:, d // 2:] = z.real, z.imag
    else:
        r[:, 0::2], r[:, 1::2] = z.real, z.imag
    y[:, c["rot_offset"]:c["rot_offset"] + d] = r
    return y


def exact(case, seed):
    c = dict(case)
    w = work(c)
    if w["flops"] > 4e12 or c["op"] == "tree" and c["batch"] * c["q_len"] * c["kv_heads"] > 40000:
        return None
    s = prepare(case, seed)
    table = s["table"].cpu().numpy()
    B, L = c["batch"], c["q_len"]
    if c["op"] == "append":
        cache, q_out = s["cache"].double().cpu().numpy(), s["q_out"].double().cpu().numpy()
        k, q = s["new_k"].double().cpu().numpy(), s["q"].double().cpu().numpy()
        v = s["new_v"].double().cpu().numpy() if s["new_v"] is not None else None
        for b in range(B):
            base = s["lengths"][b] - s["n"][b]
            for i in range(s["n"][b]):
                p = base + (i if s["depth"] is None else int(s["depth"][b, i]))
                blk, row = _slot(c, table, b, base + i)
                new = _exact_rotation(c, k[b, i].reshape(c["kv_heads"], c["dim"]), p)
                if c["kind"] == "gqa":
                    cache[0, blk, row], cache[1, blk, row] = new, v[b, i]
                else:
                    cache[blk, row] = new[0]
                q_out[b, i] = _exact_rotation(c, q[b, i], p)
        return torch.from_numpy(cache), torch.from_numpy(q_out)
    if c["op"] == "commit":
        cache = s["cache"].double()
        old = cache.clone()
        lens = []
        path = s["path"].cpu().numpy()
        for b in range(B):
            base = s["lengths"][b] - s["n"][b]
            for k in range(s["taken"][b]):
                (b0, r0), (b1, r1) = _slot(c, table, b, base + k), _slot(c, table, b, base + path[b, k])
                if c["kind"] == "gqa":
                    cache[:, b0, r0] = old[:, b1, r1]
                else:
                    cache[b0, r0] = old[b1, r1]
            lens.append(base + s["taken"][b])
        return cache, torch.tensor(lens, dtype=torch.int32)
    out = torch.zeros((c["dcp"], B, L, c["heads"] // c["dcp"], c["dim_v"]), dtype=torch.float64, device=DEV)
    group, per = c["heads"] // c["kv_heads"], c["heads"] // c["dcp"]
    mask = s["mask"].cpu().numpy().view(np.uint32)
    N, I = c["dcp"], c["interleave"]
    for b in range(B):
        S, n = s["lengths"][b], s["n"][b]
        base = S - n
        # the request's rows in the order of its tokens, gathered shard by shard
        rows = torch.empty((2, S, c["kv_heads"], c["dim"]), dtype=torch.float64, device=DEV)
        pos = np.arange(S)
        for r in range(N):
            mine = pos[pos // I % N == r]
            if not len(mine):
                continue
            local = np.arange(len(mine))
            blk = torch.from_numpy(table[r, b, local // c["block"]].astype(np.int64)).to(DEV)
            off = torch.from_numpy(local % c["block"]).to(DEV)
            at = torch.from_numpy(mine).to(DEV)
            if c["kind"] == "gqa":
                rows[0, at], rows[1, at] = s["cache"][0, blk, off].double(), s["cache"][1, blk, off].double()
            else:
                rows[0, at] = s["cache"][blk, off].double().unsqueeze(1)
        bits = mask[b if len(mask) > 1 else 0]
        for i in range(n):
            sees = np.ones(S, dtype=bool)
            sees[base:] = [bits[i, j // 32] >> (j % 32) & 1 for j in range(n)]
            sees = torch.from_numpy(sees).to(DEV)
            for g in range(c["kv_heads"]):
                heads = slice(g * group, (g + 1) * group)
                x = s["q"][b, i, heads].double() @ rows[0, :, g].T * s["scale"]
                weights = torch.softmax(x.masked_fill(~sees, -math.inf), -1)
                values = rows[1, :, g] if c["kind"] == "gqa" else rows[0, :, g, :c["dim_v"]]
                o = weights @ values
                for k in range(group):
                    h = g * group + k
                    out[h // per, b, i, h % per] = o[k]
        del rows
    return out
