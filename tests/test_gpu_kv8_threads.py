"""Calls of the 8-bit cache's operators from two host threads at once, each on its own stream and tensors: a call's set-up
is its own, whatever shape the other thread asks for."""

from __future__ import annotations

import ctypes
import threading

import pytest
import torch

import helpers as H
import kv8_common as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from context_decode_attention_paged_gb300 import build
    build.build()


def _both(calls, rounds):
    """Runs every call `rounds` times in a thread of its own, all at once; what they raised."""
    raised, start = [], threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        handle = ctypes.c_void_p(stream.cuda_stream)
        stream.synchronize()
        start.wait()
        for k in range(rounds):
            try:
                call(handle)
            except Exception as e:                               # noqa: BLE001
                raised.append(e)
            if k % 50 == 49:
                stream.synchronize()                             # (no call waits for room in the stream's queue)
        stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return raised


def _append(name, n, seed, kw):
    """An append of n rows into a cache of its own, with buffers given: () -> what it left (cache, scales, queries)."""
    from context_decode_attention_paged_gb300 import binding as dcp
    inst = H.build_instance(H.small(name, batch=2, lengths=("uniform", n, 2 * n), **kw))
    w = inst.w
    mla = w.kind == "mla"
    g = torch.Generator().manual_seed(seed)
    k, v, q = (torch.randn((2, n, h, w.head_dim_qk), generator=g).to(torch.bfloat16).cuda()
               for h in (w.num_kv_heads, w.num_kv_heads, w.num_q_heads))
    cache = torch.zeros(inst.kv_cache.shape, dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, cache.shape[1], cache.shape[3]) if not mla else (cache.shape[0],), dtype=torch.uint8, device="cuda")
    rope = dcp.dcp_rope_table(64, rot_offset=w.head_dim_qk - 64)
    table, lens, out = inst.block_tables.cuda(), inst.seq_lens.cuda(), torch.empty_like(q)

    desc = dcp.make_desc(w.kind, 2, n, w.num_q_heads, 1 if mla else w.num_kv_heads, w.head_dim_qk, w.head_dim_v, w.block_size,
                         cache.shape[0 if mla else 1], table.shape[2])
    at = lambda t: ctypes.c_void_p(t.data_ptr())                 # noqa: E731
    k = k[:, :, 0].contiguous() if mla else k
    args = (ctypes.byref(desc), rope.desc, at(rope.steps), None, at(k), None if mla else at(v), at(q), None, at(out), None, 0,
            None, at(cache), at(scales), at(table), at(lens), w.dcp_size, w.interleave)
    held = (desc, rope, k, v, q, table, lens)
    fn = dcp.raw_lib().dcp_kv8_append

    def call(stream=None):                                       # (the C call alone: threads meet in it)
        code = fn(*args, stream)
        assert code == dcp.DCP_OK and held, dcp.status_string(code)

    return call, (cache, scales, out)


@pytest.mark.parametrize("name,one,other", [
    # rows of one instance that need 96 KB of shared memory and 48 KB; latent rows: 144 and 96
    ("qwen_gqa", (300, dict(block_size=256, interleave=256, dcp_size=1)), (90, dict(block_size=96, interleave=96, dcp_size=1))),
    ("mla_32", (200, dict(block_size=128, interleave=128, dcp_size=1, num_q_heads=4)),
     (40, dict(block_size=48, interleave=48, dcp_size=1, num_q_heads=4))),
])
def test_appends_of_two_shapes_from_two_threads(name, one, other):
    from context_decode_attention_paged_gb300 import binding as dcp
    made = [_append(name, n, seed, kw) for seed, (n, kw) in enumerate((one, other))]
    for call, _ in made:
        call()
    torch.cuda.synchronize()
    want = [[t.clone() for t in held] for _, held in made]
    for _, held in made:
        for t in held:
            t.zero_()
    raised = _both([call for call, _ in made], 10000)
    assert not raised, (len(raised), raised[0])
    for (_, held), copy in zip(made, want):
        assert all(torch.equal(a, b) for a, b in zip(held, copy))
    assert dcp.dcp_get_last_device_status() == dcp.DCP_OK


def _attention(which, dim, L, name="tiny_gqa", **kw):
    """An attention call with buffers of its own: (the C call on a stream, its outputs)."""
    from context_decode_attention_paged_gb300 import binding as dcp
    dims = {} if name == "mla_32" else dict(head_dim_qk=dim, head_dim_v=dim)
    inst, codes, scales, _ = K.kv8_case(name, L, None, batch=2, lengths=("fixed", 80), **dims, **kw)
    w = inst.w
    q, table, lens = inst.q.cuda(), inst.block_tables.cuda(), inst.seq_lens.cuda()
    cache = torch.from_numpy(codes).cuda() if which == "kv8" else inst.kv_cache.cuda()
    sc, mask = torch.from_numpy(scales).cuda(), torch.from_numpy(K.chain(L)).cuda()
    shape = (w.dcp_size, 2, L, w.num_q_heads)
    po, lse = torch.empty((*shape, w.head_dim_v), device="cuda"), torch.empty(shape, device="cuda")
    ws = torch.empty((1 << 24,), dtype=torch.uint8, device="cuda")
    desc = dcp.desc_from_tensors(w.kind, inst.q, inst.kv_cache, inst.block_tables, w.head_dim_v)
    at = lambda t: ctypes.c_void_p(t.data_ptr())                 # noqa: E731
    head, out = (ctypes.byref(desc), at(q), at(cache)), (at(po), at(lse), at(ws), ws.numel())
    if which == "kv8":
        fn, args = dcp.raw_lib().dcp_kv8_decode_attn, (*head, at(sc), at(table), at(lens), None, w.dcp_size, w.interleave,
                                                       w.scale, L, *out)
    elif which == "bf16":
        fn, args = dcp.raw_lib().dcp_decode_attn, (*head, at(table), at(lens), w.dcp_size, w.interleave, w.scale, L, *out)
    else:
        fn, args = dcp.raw_lib().dcp_tree_attn, (*head, at(table), at(lens), None, at(mask), 0, w.dcp_size, w.interleave,
                                                 w.scale, *out)
    held = (desc, q, cache, sc, mask, table, lens, ws)

    def call(stream=None):
        code = fn(*args, stream)
        assert code == dcp.DCP_OK and held, dcp.status_string(code)

    return call, (po, lse)


@pytest.mark.parametrize("which,one,other", [
    # (head dim, tokens a request): the CUDA cores; the decode kernel; row blocks of one and of two tiles of a drafted tree
    ("kv8", (72, 1), (512, 1)), ("bf16", (72, 1), (512, 1)), ("bf16", (64, 1), (128, 1)), ("tree", (128, 4), (128, 64)),
])
def test_attention_of_two_shapes_from_two_threads(which, one, other):
    made = [_attention(which, *one), _attention(which, *other)]
    for call, _ in made:
        call()
    torch.cuda.synchronize()
    want = [[t.clone() for t in held] for _, held in made]
    raised = _both([call for call, _ in made], 10000)
    assert not raised, (len(raised), raised[0])
    for (_, held), copy in zip(made, want):
        assert all(torch.equal(a, b) for a, b in zip(held, copy))


@pytest.mark.parametrize("which,dim,name,kw", [("kv8", 64, "tiny_gqa", {}), ("kv8", 128, "tiny_gqa", {}), ("kv8", 72, "tiny_gqa", {}),
                                               ("bf16", 128, "tiny_gqa", {}), ("tree", 128, "tiny_gqa", {}),
                                               ("bf16", 576, "mla_32", dict(num_q_heads=64))])
def test_the_first_call_of_a_host_thread(which, dim, name, kw):
    """A thread that has made no CUDA call yet, so that no context is current in it."""
    call, held = _attention(which, dim, 2, name, **kw)
    call()
    torch.cuda.synchronize()
    want, raised = [t.clone() for t in held], []
    for t in held:
        t.zero_()
    torch.cuda.synchronize()

    def work():
        try:
            call()
        except Exception as e:                                   # noqa: BLE001
            raised.append(e)

    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not raised, raised
    assert all(torch.equal(a, b) for a, b in zip(held, want))
