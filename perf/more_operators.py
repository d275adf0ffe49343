"""Cases of the 8-bit cache's operators and of the normalised append: RMS norms of
query and key heads with the rotary position on the way to the cache, the same into
a cache held as e4m3 codes with one power-of-two scale per block of tokens and KV
head, reading such a cache back, and decode attention over it.

``run`` computes a case either in its plain form (elementary torch operations in
32 bits; angles in 64) or, with ``own`` set, through the framework's calls.  A case
is a dict of plain values; sizes follow the repository's workloads (64 query heads
over 4 KV heads of 128 dims, 8 over 2 of 64, a 576-value latent row) or are generic.

The stored form: a block's scale is 2^e.  A block that gets rows from its first slot
on takes e(a) = the smallest e with a <= 112 2^e (at least -40, at most 40), a being
the largest magnitude of the new rows; one that held rows before keeps its scale while
a <= 448 2^e and otherwise takes e(a), its old codes rounded to the new scale.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _gqa(**kw):
    c = dict(kind="gqa", heads=64, kv_heads=4, dim=128, dim_v=128, norm=128, block=128, dcp=4, interleave=128)
    c.update(kw)
    return c


def _mla(**kw):
    c = dict(kind="mla", heads=128, kv_heads=1, dim=576, dim_v=512, norm=512, block=128, dcp=8, interleave=128)
    c.update(kw)
    return c


def _rope(c, rot_dim, rot_offset=0, layout="half", base=10000.0, scaling="none", factor=1.0, original=0):
    c.update(rot_dim=rot_dim, rot_offset=rot_offset, layout=layout, base=base, scaling=scaling,
             factor=factor, original=original)
    return c


def listed():
    return [
        # a decode step of a model that normalises its query and key heads, bf16 cache
        _rope(_gqa(name="norm_step", op="norm", batch=64, q_len=1, lo=8192, hi=32768, ragged=False), 128, base=1e6),
        # its prompt chunks of up to 2048 tokens
        _rope(_gqa(name="norm_prompt", op="norm", batch=6, q_len=2048, lo=1, hi=60000, ragged=True), 128, base=1e6),
        # a decode step into the 8-bit cache: one row per request, block and head, a few blocks rescaled
        _rope(_gqa(name="store_step", op="store", batch=64, q_len=1, lo=8192, hi=32768, ragged=False), 128, base=1e6),
        # drafted tokens into small blocks dealt token by token, half of each head rotated, no norms
        _rope(_gqa(name="store_drafts", op="store", batch=33, q_len=24, heads=40, kv_heads=8, norm=0, block=16, dcp=2,
                   interleave=1, lo=100, hi=9000, ragged=True), 64),
        # prompt chunks into the 8-bit cache
        _rope(_gqa(name="store_prompt", op="store", batch=6, q_len=2048, lo=1, hi=60000, ragged=True), 128, base=1e6),
        # latent rows of a prompt: the first 512 of 576 values normalised, the last 64 rotated
        _rope(_mla(name="store_latent", op="store", batch=16, q_len=512, lo=4096, hi=67000, ragged=True), 64, 512,
              "interleaved", scaling="yarn", factor=40.0, original=4096),
        # the context of a prompt chunk read back, as an attention without paging wants it
        _gqa(name="read_context", op="read", batch=8, q_len=4096, lo=2000, hi=30000, ragged=True),
        # the last tokens of many requests, latent rows
        _mla(name="read_latent", op="read", batch=32, q_len=100, lo=50, hi=67000, ragged=True),
        # one request, a small model: what a call costs at the least
        _gqa(name="attn_tiny", op="attn", batch=1, q_len=1, heads=8, kv_heads=2, dim=64, dim_v=64, block=16, dcp=2,
             interleave=16, lo=1024, hi=1024, ragged=False),
        # several tokens of a request at once, ragged, small blocks dealt token by token
        _gqa(name="attn_verify", op="attn", batch=33, q_len=4, heads=40, kv_heads=8, block=16, dcp=2, interleave=1,
             lo=500, hi=20000, ragged=True),
        # one very long request
        _gqa(name="attn_long", op="attn", batch=1, q_len=1, heads=64, kv_heads=8, dcp=8, interleave=1, lo=200000,
             hi=200000, ragged=False),
        # a large batch of long requests
        _gqa(name="attn_batch", op="attn", batch=256, q_len=1, lo=8192, hi=32768, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    limit = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["norm", "store", "store", "read", "attn", "attn"])
        if op == "attn" or rng.random() < 0.6:
            kv = rng.choice([1, 2, 4, 8])
            dim = rng.choice([64, 128])
            group = rng.choice([1, 2, 3, 4, 5, 7, 8, 10, 16])
            c = _gqa(heads=8 * rng.randint(1, 10) if op != "attn" else kv * group, kv_heads=kv, dim=dim, dim_v=dim,
                     norm=dim)
        else:
            c = _mla(heads=rng.choice([16, 32, 64, 128]))
        c.update(block=rng.choice([16, 32, 64, 128, 128, 256]), op=op, ragged=rng.random() < 0.6)
        shards = [n for n in (1, 2, 4, 8) if c["heads"] % n == 0]
        c.update(dcp=rng.choice(shards))
        c.update(interleave=rng.choice([1, 3, 16, c["block"], 2 * c["block"]]))
        long = _log_int(rng, 500, 200000)
        c.update(lo=max(1, _log_int(rng, max(1, long // 40), long)), hi=long)
        if op in ("norm", "store"):
            c.update(batch=_log_int(rng, 1, 512), q_len=_log_int(rng, 1, 2048))
            if c["batch"] * c["q_len"] > 16384:
                continue
            if c["kind"] == "mla":
                _rope(c, 64, 512)
            else:
                _rope(c, rng.choice([c["dim"], c["dim"] // 2]))
            c.update(layout=rng.choice(["half", "interleaved"]), base=rng.choice([1e4, 1e6]),
                     scaling=rng.choice(["none", "linear", "ntk", "yarn"]))
            if c["scaling"] != "none":
                c.update(factor=float(rng.choice([2, 4, 40])), original=4096)
            if op == "store" and rng.random() < 0.3:
                c.update(norm=0)
        elif op == "read":
            c.update(batch=_log_int(rng, 1, 256), q_len=_log_int(rng, 1, 8192))
            if c["batch"] * c["q_len"] > 65536:
                continue
        else:
            c.update(batch=_log_int(rng, 1, 256), q_len=_log_int(rng, 1, 8))
        # a pool of at most 12 GB, a cost within the largest listed case's
        if op in ("read", "attn") and _lengths(c).sum() * _values(c) > 12e9:
            continue
        if _cost(c) <= limit:
            return c


# ---------------------------------------------------------------------------
# what a case has to move and compute
# ---------------------------------------------------------------------------

def _values(c):
    """Values of a token in the cache."""
    return c["dim"] * c["kv_heads"] * (2 if c["kind"] == "gqa" else 1)


def _counts(c):
    """New tokens of each request (read: tokens wanted): all q_len, or spread over 1..q_len."""
    if not c["ragged"] or c["op"] == "read":
        return np.full(c["batch"], c["q_len"], dtype=np.int64)
    return 1 + (np.arange(c["batch"], dtype=np.int64) * 7 + c["q_len"] - 1) % c["q_len"]


def _contexts(c):
    """Context length of each request before its new tokens: log-spaced over [lo, hi]."""
    n = c["batch"]
    x = np.linspace(1.0, 0.0, n) if n > 1 else np.ones(1)
    return np.rint(c["lo"] * (c["hi"] / c["lo"]) ** x).astype(np.int64)


def _lengths(c):
    return _contexts(c) if c["op"] == "read" else _contexts(c) + _counts(c)


def _starts(c):
    """First position that a read wants: the last q_len tokens', or (ragged) one that leaves it short."""
    S = _lengths(c)
    start = np.maximum(S - c["q_len"], 0)
    if c["ragged"]:
        start = np.minimum(start + (np.arange(c["batch"]) * 13) % (c["q_len"] // 2 + 1), S - 1)
    return start


def work(c):
    n, S = _counts(c), _lengths(c)
    if c["op"] in ("norm", "store"):
        size = 2 if c["op"] == "norm" else 1
        q = c["heads"] * c["dim"]
        ops = (c["heads"] + c["kv_heads"]) * (c["rot_dim"] * 3 + c["norm"] * 4)
        return {"bytes": float(n.sum() * ((2 + size) * _values(c) + 4 * q)), "flops": float(n.sum() * ops)}
    if c["op"] == "read":
        rows = np.minimum(S, _starts(c) + c["q_len"]) - _starts(c)
        return {"bytes": float(rows.sum() * 3 * _values(c)), "flops": float(rows.sum() * _values(c))}
    io = 2 * c["heads"] * (c["dim"] + c["dim_v"])
    return {"bytes": float(S.sum() * _values(c) + n.sum() * io),
            "flops": float((2 * n * c["heads"] * (c["dim"] + c["dim_v"]) * S).sum())}


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
    counts = np.maximum(hi - lo, 0)
    total = int(counts.sum()) + 1
    ids = rng.permutation(total - 1).astype(np.int32) + 1
    table = np.zeros((N, B, max(1, int(hi.max()))), dtype=np.int32)
    ends = np.cumsum(counts.reshape(-1))
    for r in range(N):
        for b in range(B):
            k, e = int(counts[r, b]), int(ends[r * B + b])
            table[r, b, lo[r, b]:lo[r, b] + k] = ids[e - k:e]
    return table, total


def _normal(shape, std, gen, dtype):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for s in range(0, flat.numel(), 1 << 28):
        e = min(flat.numel(), s + (1 << 28))
        flat[s:e] = (torch.randn((e - s,), generator=gen, device=DEV) * std).to(dtype)
    return out


def prepare(case, seed):
    c = dict(case)
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    order = rng.permutation(c["batch"])                 # which request is how long
    n, S, gqa = _counts(c)[order], _lengths(c)[order], c["kind"] == "gqa"
    first = _starts(c)[order] if c["op"] == "read" else np.zeros_like(S) if c["op"] == "attn" else S - n
    table, blocks = _tables(c, S, first, rng)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)   # noqa: E731
    s = dict(case=c, n=n.tolist(), lengths=S.tolist(), starts=first.tolist(), table=i32(table), seq_lens=i32(S),
             q_lens=i32(n) if c["ragged"] and c["op"] != "read" else None)
    shape = (blocks, c["block"], c["kv_heads"], c["dim"])
    shape = (2, *shape) if gqa else shape[:2] + shape[3:]
    if c["op"] == "norm":
        s["cache"] = _normal(shape, 1.0, gen, torch.bfloat16)
    else:
        # codes of normal values: a block's largest magnitude near 112, its scale between 2^-6 and 2^-4 (a value of
        # about 1); one block in sixteen holds much smaller values, as behind a run of quiet tokens
        s["cache"] = _normal(shape, 28.0, gen, torch.float8_e4m3fn)
        scales = rng.integers(121, 124, (2, blocks, c["kv_heads"]) if gqa else (blocks,))
        quiet = rng.random(scales.shape) < 1 / 16
        s["scales"] = torch.from_numpy(np.where(quiet, scales - 4, scales).astype(np.uint8)).to(DEV)
    B, L = c["batch"], c["q_len"]
    if c["op"] in ("norm", "store"):
        # the tokens' rows as a fused projection leaves them: queries, keys and values of a token side by side
        q_w, k_w = c["heads"] * c["dim"], c["kv_heads"] * c["dim"]
        rows = _normal((B, L, q_w + k_w * (2 if gqa else 1)), 1.0, gen, torch.bfloat16)
        s["q"] = rows[..., :q_w].unflatten(-1, (c["heads"], c["dim"]))
        k = rows[..., q_w:q_w + k_w]
        s["new_k"] = k.unflatten(-1, (c["kv_heads"], c["dim"])) if gqa else k
        s["new_v"] = rows[..., q_w + k_w:].unflatten(-1, (c["kv_heads"], c["dim"])) if gqa else None
        s["q_out"] = torch.zeros((B, L, c["heads"], c["dim"]), dtype=torch.bfloat16, device=DEV)
        # (request, index) of the tokens that are there
        b = np.repeat(np.arange(B), n)
        s["b"], s["i"] = torch.from_numpy(b).to(DEV), torch.from_numpy(np.concatenate([np.arange(x) for x in n])).to(DEV)
        weight = lambda: 1.0 + 0.2 * torch.randn((c["norm"],), generator=gen, device=DEV)   # noqa: E731
        s["k_weight"] = weight() if c["norm"] else None
        s["q_weight"] = weight() if c["norm"] and gqa else None       # (latent queries come absorbed)
        s["freqs"], s["mscale"] = _frequencies(c)
        if own:
            from context_decode_attention_paged_gb300 import binding as dcp
            s["rope"] = dcp.dcp_rope_table(c["rot_dim"], base=c["base"], layout=c["layout"], rot_offset=c["rot_offset"],
                                           scaling=c["scaling"], factor=c["factor"], original_max_position=c["original"],
                                           device=DEV)
    elif c["op"] == "read":
        s["first"] = i32(first)
        row = (B, L, c["kv_heads"], c["dim"]) if gqa else (B, L, c["dim"])
        s["out_k"] = torch.zeros(row, dtype=torch.bfloat16, device=DEV)
        s["out_v"] = torch.zeros(row, dtype=torch.bfloat16, device=DEV) if gqa else None
        take = np.minimum(S, first + L) - first
        s["b"] = torch.from_numpy(np.repeat(np.arange(B), take)).to(DEV)
        s["i"] = torch.from_numpy(np.concatenate([np.arange(x) for x in take])).to(DEV)
    else:
        s["q"] = _normal((B, L, c["heads"], c["dim"]), 1.0, gen, torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(c["dim"])
        s["groups"] = [torch.from_numpy(g).to(DEV) for g in _padded_groups(c, S)]
        s["longest"] = [int(S[g.cpu().numpy()].max()) for g in s["groups"]]
        if own:
            from context_decode_attention_paged_gb300 import binding as dcp
            s["partial"] = torch.empty((c["dcp"], B, L, c["heads"], c["dim_v"]), device=DEV)
            s["lse"] = torch.empty((c["dcp"], B, L, c["heads"]), device=DEV)
            s["out"] = torch.empty((c["dcp"], B, L, c["heads"] // c["dcp"], c["dim_v"]), dtype=torch.bfloat16, device=DEV)
            desc = dcp.desc_from_tensors(c["kind"], s["q"], s["cache"], s["table"], c["dim_v"])
            size = dcp.dcp_kv8_decode_attn_workspace_size(desc, c["dcp"])
            s["workspace"] = torch.empty((max(size, 1),), dtype=torch.uint8, device=DEV)
    return s


def _padded_groups(c, S):
    """Requests in groups of like lengths, padded to the longest: up to 2^29 values of keys each."""
    groups, most = [], (1 << 29) // (c["kv_heads"] * c["dim"])
    for b in np.argsort(-S, kind="stable"):
        if groups and S[groups[-1][0]] * (len(groups[-1]) + 1) <= most and S[b] > 0.7 * S[groups[-1][0]]:
            groups[-1].append(b)
        else:
            groups.append([b])
    return [np.array(g) for g in groups]


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
    """(block, slot) of positions t of requests b (tensors)."""
    c = s["case"]
    N, I, bs = c["dcp"], c["interleave"], c["block"]
    j = t // (I * N) * I + t % I
    return s["table"][t // I % N, b, j // bs].long(), j % bs


def _prepared(s, x, weight):
    """Rows x [tokens][heads][dim] normalised and rotated, in 32 bits."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        part = x[..., :c["norm"]]
        part = part * torch.rsqrt(part.square().mean(-1, keepdim=True) + EPS) * weight
        x = torch.cat([part, x[..., c["norm"]:]], -1)
    base = s["seq_lens"].long()[s["b"]] - (s["q_lens"].long()[s["b"]] if s["q_lens"] is not None else c["q_len"])
    angle = (base + s["i"]).double().view(-1, 1) * s["freqs"]
    cos = (angle.cos() * s["mscale"]).float().unsqueeze(1)
    sin = (angle.sin() * s["mscale"]).float().unsqueeze(1)
    a, d = c["rot_offset"], c["rot_dim"]
    first, second = ((slice(a, a + d // 2), slice(a + d // 2, a + d)) if c["layout"] == "half"
                     else (slice(a, a + d, 2), slice(a + 1, a + d, 2)))
    y = x.clone()
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return y


def _new_cells(s):
    c = s["case"]
    base = s["seq_lens"].long()[s["b"]] - (s["q_lens"].long()[s["b"]] if s["q_lens"] is not None else c["q_len"])
    return _cells(s, s["b"], base + s["i"])


def _plain_norm(s):
    c = s["case"]
    blk, slot = _new_cells(s)
    k = _prepared(s, s["new_k"][s["b"], s["i"]].view(-1, c["kv_heads"], c["dim"]), s["k_weight"]).to(torch.bfloat16)
    if c["kind"] == "gqa":
        s["cache"][0, blk, slot], s["cache"][1, blk, slot] = k, s["new_v"][s["b"], s["i"]]
    else:
        s["cache"][blk, slot] = k.squeeze(1)
    s["q_out"][s["b"], s["i"]] = _prepared(s, s["q"][s["b"], s["i"]], s["q_weight"]).to(torch.bfloat16)
    return s["cache"], s["q_out"]


def _code(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _store_pool(pool, scales, rows, blk, slot):
    """New rows [tokens][heads][dim] (32 bits) into one pool [blocks][block][heads][dim], its scales [blocks][heads]."""
    most = torch.zeros(scales.shape, device=DEV).index_reduce_(0, blk, rows.abs().amax(-1), "amax")
    first = torch.full((len(pool),), pool.shape[1], device=DEV).index_reduce_(0, blk, slot, "amin").view(-1, 1)
    m, x = torch.frexp(most)                                  # most = m 2^x, m in [0.5, 1); 112 = 0.875 2^7
    wanted = torch.where(most > 0, x - 6 - (m <= 0.875).int(), -40).clamp(-40, 40)
    old = scales.int() - 127
    keep = (first == pool.shape[1]) | (first > 0) & (most <= torch.exp2(old.float()) * 448.0)
    e = torch.where(keep, old, wanted)
    before = torch.arange(pool.shape[1], device=DEV).view(1, -1, 1) < torch.where(keep, 0, first).unsqueeze(1)
    ratio = torch.exp2((old - e).float()).view(len(pool), 1, -1, 1)
    pool.copy_(torch.where(before.unsqueeze(-1), _code(pool.float() * ratio), pool))
    pool.view(torch.uint8)[blk, slot] = _code(rows * torch.exp2(-e.float())[blk].unsqueeze(-1)).view(torch.uint8)
    scales.copy_(e + 127)


def _pools(s):
    """(pool [blocks][block][heads][dim], scales [blocks][heads]) of keys and values, or of latent rows."""
    if s["case"]["kind"] == "gqa":
        return [(s["cache"][0], s["scales"][0]), (s["cache"][1], s["scales"][1])]
    return [(s["cache"].unsqueeze(2), s["scales"].unsqueeze(1))]


def _plain_store(s):
    c = s["case"]
    blk, slot = _new_cells(s)
    rows = [_prepared(s, s["new_k"][s["b"], s["i"]].view(-1, c["kv_heads"], c["dim"]), s["k_weight"])]
    if c["kind"] == "gqa":
        rows.append(s["new_v"][s["b"], s["i"]].float())
    for (pool, scales), new in zip(_pools(s), rows):
        _store_pool(pool, scales, new, blk, slot)
    s["q_out"][s["b"], s["i"]] = _prepared(s, s["q"][s["b"], s["i"]], s["q_weight"]).to(torch.bfloat16)
    return s["cache"], s["scales"].view(torch.float8_e8m0fnu), s["q_out"]


def _plain_read(s):
    blk, slot = _cells(s, s["b"], s["first"].long()[s["b"]] + s["i"])
    for (pool, scales), out in zip(_pools(s), (s["out_k"], s["out_v"])):
        rows = pool.view(torch.uint8)[blk, slot].view(torch.float8_e4m3fn).float()
        rows = rows * torch.exp2(scales[blk].float() - 127).unsqueeze(-1)
        out[s["b"], s["i"]] = rows.view(-1, *out.shape[2:]).to(torch.bfloat16)
    return s["out_k"], s["out_v"]


def _plain_attn(s):
    c = s["case"]
    B, L, H, Hkv, D = c["batch"], c["q_len"], c["heads"], c["kv_heads"], c["dim"]
    out = torch.zeros((B, L, H, D), dtype=torch.bfloat16, device=DEV)
    S = s["seq_lens"].long()
    n = s["q_lens"].long() if s["q_lens"] is not None else torch.full_like(S, L)
    node = torch.arange(L, device=DEV)
    for g, longest in zip(s["groups"], s["longest"]):         # (requests of like lengths, padded)
        t = torch.arange(longest, device=DEV)
        blk, slot = _cells(s, g.view(-1, 1), torch.minimum(t, S[g].view(-1, 1) - 1))
        k, v = (pool.view(torch.uint8)[blk, slot].view(torch.float8_e4m3fn).float().mul_(
            torch.exp2(scales[blk].float() - 127).unsqueeze(-1)) for pool, scales in _pools(s))   # [g][S][Hkv][D]
        q = s["q"][g].float().view(len(g), L, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(len(g), Hkv, -1, D)
        x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"])           # [g][Hkv][L * group][S]
        last = (S[g] - n[g]).view(-1, 1) + node                               # [g][L]: the position of a query
        hidden = t > last.unsqueeze(-1)
        x.masked_fill_(hidden.repeat_interleave(H // Hkv, 1).unsqueeze(1), -math.inf)
        p = x.sub_(x.amax(-1, keepdim=True)).exp_()
        o = torch.matmul(p, v.transpose(1, 2)) / p.sum(-1, keepdim=True)
        o = o.view(len(g), Hkv, L, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(len(g), L, H, D)
        out[g] = torch.where((node < n[g].view(-1, 1)).view(len(g), L, 1, 1), o, 0.0).to(torch.bfloat16)
    N = c["dcp"]
    return out.view(B, L, N, H // N, D).permute(2, 0, 1, 3, 4).contiguous()


def _own(s):
    from context_decode_attention_paged_gb300 import binding as dcp
    c = s["case"]
    if c["op"] == "norm":
        dcp.dcp_kv_cache_append_norm(c["kind"], s["new_k"], s["new_v"], s["cache"], s["table"], s["seq_lens"], c["dcp"],
                                     c["interleave"], s["rope"], k_weight=s["k_weight"], q_weight=s["q_weight"], eps=EPS,
                                     q=s["q"], q_out=s["q_out"], q_lens=s["q_lens"])
        return s["cache"], s["q_out"]
    if c["op"] == "store":
        dcp.dcp_kv8_append(c["kind"], s["new_k"], s["new_v"], s["cache"], s["scales"], s["table"], s["seq_lens"], c["dcp"],
                           c["interleave"], s["rope"], k_weight=s["k_weight"], q_weight=s["q_weight"], eps=EPS,
                           q=s["q"], q_out=s["q_out"], q_lens=s["q_lens"])
        return s["cache"], s["scales"].view(torch.float8_e8m0fnu), s["q_out"]
    if c["op"] == "read":
        return dcp.dcp_kv8_read(c["kind"], s["cache"], s["scales"], s["table"], s["seq_lens"], c["q_len"], c["dcp"],
                                c["interleave"], starts=s["first"], out_k=s["out_k"], out_v=s["out_v"])
    dcp.dcp_kv8_decode_attn(c["kind"], s["q"], s["cache"], s["scales"], s["table"], s["seq_lens"], c["dcp"],
                            c["interleave"], s["scale"], c["q_len"], c["dim_v"], q_lens=s["q_lens"],
                            partial_out=s["partial"], lse=s["lse"], workspace=s["workspace"])
    dcp.dcp_merge(s["partial"], s["lse"], c["dcp"], out=s["out"], want_lse=False)
    return s["out"]


def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "store": _plain_store, "read": _plain_read, "attn": _plain_attn}[s["case"]["op"]](s)


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


def _exact_norm(c, x, weight):
    if weight is None:
        return x
    y = x.copy()
    for h in range(len(x)):
        part = x[h, :c["norm"]]
        y[h, :c["norm"]] = part / math.sqrt(float(part @ part) / c["norm"] + EPS) * weight
    return y


def _e4m3(x):
    """Nearest value with 4 significant bits at or above 2^-6, a multiple of 2^-9 below; ties to even, at most 448."""
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def _exact_store(c, s, table, k, v):
    """(codes' values, scales) after the rows k (and v), lists of (request, position, rows [heads][dim]), are stored."""
    codes, scales = s["cache"].double().cpu().numpy(), s["scales"].cpu().numpy().astype(np.int64) - 127
    if c["kind"] == "mla":
        codes, scales = codes[None, :, :, None], scales[None, :, None]
    for pool, new in enumerate((k, v) if v is not None else (k,)):
        held = {}
        for b, t, rows in new:
            blk, at = _slot(c, table, b, t)
            held.setdefault(blk, {})[at] = rows
        for blk, rows in held.items():
            first = min(rows)
            for h in range(c["kv_heads"]):
                most = max(float(np.abs(r[h]).max()) for r in rows.values())
                e = int(scales[pool, blk, h])
                if first == 0 or most > 448.0 * 2.0 ** e:
                    new_e = -40
                    while new_e < 40 and most > 112.0 * 2.0 ** new_e:
                        new_e += 1
                    codes[pool, blk, :first, h] = _e4m3(codes[pool, blk, :first, h] * 2.0 ** (e - new_e))
                    scales[pool, blk, h] = e = new_e
                for at, r in rows.items():
                    codes[pool, blk, at, h] = _e4m3(r[h] * 2.0 ** -e)
    if c["kind"] == "mla":
        codes, scales = codes[0, :, :, 0], scales[0, :, 0]
    return torch.from_numpy(codes), torch.from_numpy(2.0 ** scales.astype(np.float64))


def exact(case, seed):
    c = dict(case)
    n, w = _counts(c), work(c)
    if c["op"] in ("norm", "store") and n.sum() * (c["heads"] + 4 * c["kv_heads"] * c["dim"] / 128) > 3e5:
        return None
    if c["op"] == "read" and w["bytes"] > 3e8 or c["op"] == "attn" and (w["bytes"] > 5e9 or w["flops"] > 1e12):
        return None
    s = prepare(case, seed)
    table = s["table"].cpu().numpy()
    B, L, gqa = c["batch"], c["q_len"], c["kind"] == "gqa"
    if c["op"] in ("norm", "store"):
        q_out = s["q_out"].double().cpu().numpy()
        new_k, q = s["new_k"].double().cpu().numpy(), s["q"].double().cpu().numpy()
        new_v = s["new_v"].double().cpu().numpy() if gqa else None
        kw, qw = (None if s[x] is None else s[x].double().cpu().numpy() for x in ("k_weight", "q_weight"))
        k, v = [], []
        for b in range(B):
            base = s["lengths"][b] - s["n"][b]
            for i in range(s["n"][b]):
                rows = _exact_norm(c, new_k[b, i].reshape(c["kv_heads"], c["dim"]), kw)
                k.append((b, base + i, _exact_rotation(c, rows, base + i)))
                if gqa:
                    v.append((b, base + i, new_v[b, i]))
                q_out[b, i] = _exact_rotation(c, _exact_norm(c, q[b, i], qw), base + i)
        if c["op"] == "store":
            return (*_exact_store(c, s, table, k, v if gqa else None), torch.from_numpy(q_out))
        cache = s["cache"].double().cpu().numpy()
        for j, (b, t, rows) in enumerate(k):
            blk, at = _slot(c, table, b, t)
            if gqa:
                cache[0, blk, at], cache[1, blk, at] = rows, v[j][2]
            else:
                cache[blk, at] = rows[0]
        return torch.from_numpy(cache), torch.from_numpy(q_out)
    codes, scales = s["cache"].view(torch.uint8), 2.0 ** (s["scales"].double() - 127)
    if c["op"] == "read":
        codes, scales = s["cache"].double().cpu().numpy(), scales.cpu().numpy()
        out = np.zeros((2, *s["out_k"].shape))
        for b in range(B):
            for i in range(min(s["lengths"][b] - s["starts"][b], L)):
                blk, at = _slot(c, table, b, s["starts"][b] + i)
                if gqa:
                    out[:, b, i] = codes[:, blk, at] * scales[:, blk, :, None]
                else:
                    out[0, b, i] = codes[blk, at] * scales[blk]
        return torch.from_numpy(out[0]), torch.from_numpy(out[1]) if gqa else None
    out = torch.zeros((c["dcp"], B, L, c["heads"] // c["dcp"], c["dim_v"]), dtype=torch.float64, device=DEV)
    group, per, N, I = c["heads"] // c["kv_heads"], c["heads"] // c["dcp"], c["dcp"], c["interleave"]
    for b in range(B):
        S, n_b = s["lengths"][b], s["n"][b]
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
            values = codes[:, blk, off].view(torch.float8_e4m3fn).double()
            rows[:, torch.from_numpy(mine).to(DEV)] = values * scales[:, blk].unsqueeze(-1)
        for i in range(n_b):
            seen = S - n_b + i + 1
            for g in range(c["kv_heads"]):
                x = s["q"][b, i, g * group:(g + 1) * group].double() @ rows[0, :seen, g].T * s["scale"]
                o = torch.softmax(x, -1) @ rows[1, :seen, g]
                h = torch.arange(g * group, (g + 1) * group, device=DEV)
                out[h // per, b, i, h % per] = o
        del rows
    return out
