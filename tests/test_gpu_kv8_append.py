"""GPU parity of the normalised append (bf16 and 8-bit cache) and of reading the 8-bit cache back.

A prepared value y = m (x0 c - x1 s) w / sqrt(mean x^2 + eps) in fp32: c and s within 2^-22, the
norm's factor within 2^-20 (a sum of up to 576 squares in fp32, each term once rounded, in a tree of
shuffles over at most 24 terms a lane: below 32 * 2^-24; the square root 2^-22), the products and the
sum 5 * 2^-24: together below 2^-18 of m (|x0| + |x1|) after the norm.  A bf16 value is rounded once
more (2^-8 of it), a code to half a step (2^-4 of it, or half of 2^-9 scales below 2^-6 scales)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import helpers as H
import tree_common as T
from oracle import dcp_oracle as orc
from oracle import kv8_oracle as k8o
from oracle import tree_oracle as tro

pytestmark = pytest.mark.gpu

SLACK = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from context_decode_attention_paged_gb300 import build
    build.build()


HALF, INTER = dict(rot_dim=64), dict(rot_dim=64, layout="interleaved")
LATENT = dict(rot_dim=64, rot_offset=512, layout="interleaved")
CASES = [
    # (workload, overrides, new tokens, rope, norm dims of keys and of queries, q_lens, offsets)
    ("tiny_gqa", dict(batch=3, lengths=("uniform", 20, 700), dcp_size=4, interleave=3), 7, HALF, 64, 64, None, None),
    ("tiny_gqa", dict(batch=3, lengths=("uniform", 20, 700), dcp_size=4, interleave=3), 7, INTER, 64, 0, [7, 0, 3], None),
    ("tiny_gqa", dict(batch=2, lengths=("uniform", 20, 700)), 3, dict(rot_dim=32, rot_offset=16), 0, 64, None, [[0, 1, 1]]),
    ("tiny_gqa", dict(batch=2, lengths=("uniform", 20, 700)), 3, dict(rot_dim=20, rot_offset=6), 32, 64, None, None),
    ("tiny_gqa", dict(batch=2, lengths=("uniform", 20, 700)), 3, dict(rot_dim=6, rot_offset=5, layout="interleaved"), 64, 64,
     None, [[3, 1, 2], [0, 0, 9]]),
    ("tiny_gqa", dict(batch=2, lengths=("uniform", 20, 700)), 2, None, 64, 64, None, None),
    ("tiny_gqa", dict(batch=2, lengths=("uniform", 20, 700)), 2, None, 0, 0, None, None),
    ("tiny_gqa", dict(batch=1, lengths=("fixed", 1), interleave=1), 1, HALF, 64, 64, None, None),
    ("tiny_gqa", dict(batch=2, lengths=("fixed", 5), interleave=1), 5, HALF, 64, 64, None, None),
    ("tiny_gqa", dict(batch=2, num_q_heads=10, num_kv_heads=5, head_dim_qk=72, head_dim_v=72, block_size=24,
                      lengths=("uniform", 40, 300)), 3, HALF, 72, 72, None, None),
    ("tiny_gqa", dict(batch=2, num_q_heads=4, num_kv_heads=2, head_dim_qk=256, head_dim_v=256, lengths=("uniform", 40, 300)),
     9, dict(rot_dim=128), 256, 256, None, None),
    ("tiny_gqa", dict(batch=2, num_q_heads=2, num_kv_heads=1, head_dim_qk=264, head_dim_v=264, lengths=("uniform", 40, 300)),
     9, dict(rot_dim=128, rot_offset=8), 264, 264, None, None),
    ("qwen_gqa", dict(batch=2, num_q_heads=10, lengths=("uniform", 400, 1500)), 300, dict(rot_dim=128, base=1e6), 128, 128,
     None, None),
    ("qwen_gqa", dict(batch=2, num_q_heads=8, block_size=512, dcp_size=1, lengths=("uniform", 400, 1500)), 390,
     dict(rot_dim=128), 128, 128, [390, 201], None),
    ("qwen_gqa", dict(batch=70, lengths=("uniform", 1, 4000)), 1, dict(rot_dim=64, scaling="yarn", factor=40.0,
                                                                      original_max_position=4096), 128, 128, None, None),
    ("mla_32", dict(batch=3, num_q_heads=16, lengths=("uniform", 129, 3000), interleave=1), 5, LATENT, 512, 0, None, None),
    ("mla_32", dict(batch=2, num_q_heads=4, dcp_size=2, lengths=("uniform", 300, 900)), 250,
     dict(rot_dim=64, rot_offset=512), 512, 0, [250, 131], None),
    # the longest heads, all dims rotated in halves: most shared memory, for few rows a block and for many
    ("tiny_gqa", dict(batch=1, num_q_heads=2, num_kv_heads=1, head_dim_qk=768, head_dim_v=768, lengths=("fixed", 90)), 20,
     dict(rot_dim=768), 768, 768, None, None),
    ("tiny_gqa", dict(batch=1, num_q_heads=2, num_kv_heads=1, head_dim_qk=768, head_dim_v=768, block_size=256, dcp_size=1,
                      lengths=("fixed", 400)), 200, dict(rot_dim=768), 768, 768, None, None),
    ("tiny_gqa", dict(batch=1, num_q_heads=2, num_kv_heads=1, head_dim_qk=8, head_dim_v=8, lengths=("fixed", 90)), 20,
     dict(rot_dim=8, layout="interleaved"), 8, 8, None, None),
]


def _call(which, inst, n, rope_kw, kdim, qdim, q_lens, offsets, codes=None, scales=None, in_place=False, seed=5, eps=1e-6,
          scale_rows=1.0, stream=None, fused=True, change=None):
    """Runs the append and returns (cache, scales or None, q_out, the oracle's prepared k, v, q_out, the inputs)."""
    from context_decode_attention_paged_gb300 import binding as dcp
    w = inst.w
    k, v, q = T.append_inputs(w, n, seed, fused)
    for t in (k, v, q):
        if t is not None:
            t.mul_(scale_rows)
    if change is not None:
        change(k, v, q)
    rng = np.random.default_rng(seed)
    wk, wq = (None if not d else (1 + 0.3 * rng.standard_normal(d)).astype(np.float32) for d in (kdim, qdim))
    on = lambda x: None if x is None else torch.as_tensor(x).cuda()   # noqa: E731
    rope = None if rope_kw is None else dcp.dcp_rope_table(**rope_kw)
    gq = T.to_gpu(q)
    q_out = gq if in_place else torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    # (more than one norm dim length at a time is two calls' worth: the shorter one's weights are 1 behind it)
    if wk is not None and wq is not None and len(wk) != len(wq):
        wk = wk if len(wk) > len(wq) else wk[:len(wq)]
        wq = wq[:len(wk)]
    args = (T.to_gpu(k), T.to_gpu(v))
    kw = dict(k_weight=on(wk), q_weight=on(wq), eps=eps, q=gq, q_out=q_out, q_lens=on(ql), pos_offsets=on(off), stream=stream)
    tail = (on(inst.block_tables), on(inst.seq_lens), w.dcp_size, w.interleave, rope)
    torch.cuda.synchronize()
    if which == "norm":
        cache = inst.kv_cache.cuda()
        dcp.dcp_kv_cache_append_norm(w.kind, *args, cache, *tail, **kw)
        sc = None
    else:
        cache, sc = on(codes), on(scales)
        torch.cuda.synchronize()
        dcp.dcp_kv8_append(w.kind, *args, cache, sc, *tail, **kw)
    torch.cuda.synchronize()
    freqs = None
    if rope_kw is not None:
        freqs = (tro.rope_freqs(rope_kw["rot_dim"], rope_kw.get("base", 10000.0), rope_kw.get("scaling", "none"),
                                rope_kw.get("factor", 1.0), rope_kw.get("original_max_position", 0)),
                 rope_kw.get("layout", "half"), rope_kw.get("rot_offset", 0), rope.desc.mscale)
    pk = k8o.prepared(orc.to_f64(k), wk, eps, inst.seq_lens.numpy(), q_lens, offsets, freqs)
    pq = k8o.prepared(orc.to_f64(q), wq, eps, inst.seq_lens.numpy(), q_lens, offsets, freqs)
    want_q = orc.to_f64(q) if in_place else np.full(q.shape, 7.0)
    for b in range(w.batch):
        m = n if q_lens is None else q_lens[b]
        want_q[b, :m] = pq[b, :m]
    return cache, sc, q_out, pk, None if v is None else orc.to_f64(v), want_q


def _near_bf16(got, want, what):
    err = np.abs(got - want)
    tol = 2.0 ** -8 * np.abs(want) + SLACK * 2 * np.abs(want).max(-1, keepdims=True)
    assert (err <= tol).all(), (what, float((err - tol).max()))


@pytest.mark.parametrize("name,kw,n,rope,kdim,qdim,q_lens,offsets", CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_append_norm(name, kw, n, rope, kdim, qdim, q_lens, offsets, in_place):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small(name, **kw))
    w = inst.w
    cache, _, q_out, k, v, want_q = _call("norm", inst, n, rope, kdim, qdim, q_lens, offsets, in_place=in_place,
                                          fused=not in_place)
    want, _ = tro.ref_append(w.kind, orc.to_f64(inst.kv_cache), k, v, None, inst.block_tables.numpy(),
                             inst.seq_lens.numpy(), w.dcp_size, w.interleave, w.block_size, np.zeros(0), "half", 0, 1.0, q_lens)
    got = orc.to_f64(cache)
    same = want == orc.to_f64(inst.kv_cache)                 # (untouched rows bit for bit)
    same = same.all(-1, keepdims=True) & np.ones_like(same)
    assert np.array_equal(got[same], want[same])
    _near_bf16(got, want, "cache")
    if w.kind == "gqa":
        assert np.array_equal(got[1], want[1])
    _near_bf16(orc.to_f64(q_out), want_q, "queries")
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK


def _cache8(inst, seed=3, exps=(-8, -4)):
    rng = np.random.default_rng(seed)
    shape = tuple(inst.kv_cache.shape)
    codes = rng.integers(0, 256, shape).astype(np.uint8)
    codes[(codes & 127) == 127] ^= 1                         # (no NaN)
    sshape = (2, shape[1], shape[3]) if inst.w.kind == "gqa" else (shape[0],)
    return codes, (rng.integers(exps[0], exps[1] + 1, sshape) + 127).astype(np.uint8)


def _check_codes(inst, codes, scales, cache, sc, k, v, q_lens):
    w = inst.w
    want, want_s, touched = k8o.ref_kv8_append(w.kind, codes, scales, k, v, inst.block_tables.numpy(), inst.seq_lens.numpy(),
                                               w.dcp_size, w.interleave, w.block_size, q_lens)
    got, got_s = cache.cpu().numpy(), sc.cpu().numpy()
    gc, gs, wc = (x[None, :, :, None] if w.kind == "mla" else x for x in (got, got[:0], want))
    ss = want_s[None, :, None] if w.kind == "mla" else want_s
    # no largest magnitude lies within the arithmetic's slack of a scale's border, so the scales are equal
    for pool, blk, h, first, rows in touched:
        a = max(np.abs(r[np.isfinite(r)]).max(initial=0.0) for r in rows.values())
        for border in [112.0 * 2.0 ** e for e in range(-40, 41)] + [448.0 * 2.0 ** (e - 127.0) for e in (int(scales.min()), int(scales.max()))]:
            assert pool == 1 or a == 0 or abs(a / border - 1) > 2 * SLACK, "choose another seed"
    assert np.array_equal(got_s, want_s)
    new = np.zeros(wc.shape, dtype=bool)
    for pool, blk, h, first, rows in touched:
        s = 2.0 ** (int(ss[pool, blk, h]) - 127)
        for slot, y in rows.items():
            new[pool, blk, slot, h] = True
            if pool == 1 or not np.isfinite(y).all():
                assert np.array_equal(gc[pool, blk, slot, h], wc[pool, blk, slot, h])     # values are exact
                continue
            g = k8o.VALUES[gc[pool, blk, slot, h]] * s
            y = np.clip(y, -448.0 * s, 448.0 * s)            # (beyond the largest code: that one)
            slack = 2 * SLACK * np.abs(y).max()
            assert (np.abs(g - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s) + slack).all()
            # and the oracle's code, unless the value is a border's slack away from the next one
            other = gc[pool, blk, slot, h] != wc[pool, blk, slot, h]
            mid = (g + k8o.VALUES[wc[pool, blk, slot, h]] * s) / 2
            assert (np.abs(y - mid)[other] <= slack).all()
    assert np.array_equal(gc[~new], wc[~new])                # earlier rows rounded to the scale, all others untouched


@pytest.mark.parametrize("name,kw,n,rope,kdim,qdim,q_lens,offsets", CASES)
@pytest.mark.parametrize("size", [1.0, 0.02, 40.0])
def test_kv8_append(name, kw, n, rope, kdim, qdim, q_lens, offsets, size):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small(name, **kw))
    codes, scales = _cache8(inst)
    cache, sc, q_out, k, v, want_q = _call("kv8", inst, n, rope, kdim, qdim, q_lens, offsets, codes, scales, scale_rows=size)
    _check_codes(inst, codes, scales, cache, sc, k, v, q_lens)
    _near_bf16(orc.to_f64(q_out), want_q, "queries")
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK


@pytest.mark.parametrize("name,kw,n,starts", [
    ("tiny_gqa", dict(batch=4, lengths=("uniform", 1, 700), dcp_size=4, interleave=3), 50, [0, 3, 600, 5000]),
    ("tiny_gqa", dict(batch=3, num_q_heads=10, num_kv_heads=5, head_dim_qk=72, head_dim_v=72, block_size=24,
                      lengths=("uniform", 40, 300)), 1, None),
    ("qwen_gqa", dict(batch=3, lengths=("uniform", 300, 3000)), 700, [0, 100, 299]),
    ("mla_32", dict(batch=3, lengths=("uniform", 300, 3000), interleave=1), 333, [0, 100, 299]),
])
@pytest.mark.parametrize("parts", ["kv", "k", "v", "none"])
def test_read_back(name, kw, n, starts, parts):
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small(name, **kw))
    w = inst.w
    if w.kind == "mla" and parts == "v":
        return
    codes, scales = _cache8(inst, exps=(-40, 40))
    shape = (w.batch, n, w.num_kv_heads, w.head_dim_qk) if w.kind == "gqa" else (w.batch, n, w.head_dim_qk)
    fill = lambda: torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    ok = fill() if parts in ("kv", "k") else None
    ov = fill() if w.kind == "gqa" and parts in ("kv", "v") else None
    on = lambda x: None if x is None else torch.as_tensor(x).cuda()   # noqa: E731
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32)
    ok, ov = dcp.dcp_kv8_read(w.kind, on(codes), on(scales), on(inst.block_tables), on(inst.seq_lens), n, w.dcp_size,
                              w.interleave, starts=on(st), out_k=ok, out_v=ov)
    values = k8o.dequantise(codes, scales)
    for pool, out in enumerate((ok, ov)):
        if out is None:
            continue
        want = np.full(shape, 0.0 if parts == "none" else 7.0)
        for b in range(w.batch):
            s0 = 0 if starts is None else starts[b]
            for i in range(max(0, min(n, int(inst.seq_lens[b]) - s0))):
                blk, slot = tro.cell_of(inst.block_tables.numpy(), b, s0 + i, w.interleave, w.dcp_size, w.block_size)
                want[b, i] = values[pool, blk, slot] if w.kind == "gqa" else values[blk, slot]
        assert np.array_equal(orc.to_f64(out), want)         # (codes times powers of two are bf16 values)
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK
