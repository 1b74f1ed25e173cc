"""The serving operators on a stream that is not the current one: given as a torch stream or as a
raw handle, with results whose memory no pending work of the current stream still writes."""
import ctypes
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
from chunked_kda_delta_gb300.inputs import custom, make_inputs
from chunked_kda_delta_gb300.kda import KdaScratchAllocator

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def calls():
    """name -> function of stream that runs an operator and returns its results; on inputs that
    are made here, alike in every call."""
    gen = torch.Generator("cuda").manual_seed(5)
    draw = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    tables, refs = i32([[0, 1], [2, -1]]), i32([1, 1, 1, 0, 0])
    pool = draw(5, 64)
    x, scores = draw(2, 3, 700), draw(2, 3)
    codes = [torch.zeros(5, 2, 16, 64, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    scales = [torch.zeros(5, 2, device="cuda") for _ in range(2)]
    k, v, q = (draw(20, h, 64).bfloat16() for h in (2, 2, 4))
    lens, cu = i32([17, 3]), i32([0, 17, 20])
    cache = (*codes, *scales, tables)
    K.kda_kvcache_append(k, v, *cache, i32([0, 0]), cu_tokens=cu)
    inp = make_inputs(custom([1, 1], 2, False, 6, dense=True), "cuda")
    tok = [inp[n].view(2, 1, *inp[n].shape[1:]) for n in ("q", "k", "v", "g", "beta")]
    state = draw(3, 2, 128, 128) * 0.1
    two, zeros, kept, pages = i32([2, 2]), i32([0, 0]), i32([20, 0]), i32([2, 0])
    drop = torch.tensor([True, False], device="cuda")
    return {
        "alloc": lambda s: K.kda_pages_alloc(tables, refs, two, stream=s),
        "free": lambda s: K.kda_pages_free(tables, refs, drop, stream=s),
        "fork": lambda s: K.kda_pages_fork(tables, refs, zeros, lens=kept, page_tokens=16, pools=[pool], stream=s),
        "compact": lambda s: K.kda_pages_compact(tables, refs, [pool], stream=s),
        "attend": lambda s: (K.kda_kvcache_attention(q, *cache, lens, cu_tokens=cu, stream=s),),
        "beam": lambda s: K.kda_beam_select(x, scores, stream=s),
        "decode": lambda s: (K.kda_decode_paged(*tok, state, pages, stream=s),),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["alloc", "free", "fork", "compact", "attend", "beam", "decode"])
def test_given_stream(name, raw):
    want = calls()[name](None)
    call = calls()[name]
    side = torch.cuda.Stream()
    # A block of each result's size with a write to it pending on the current stream, given back
    # to the allocator.  The inputs are there already, so the call runs ahead of that write.
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    held = [torch.empty_like(t) for t in want]
    for _ in range(8):
        busy = busy @ busy * 1e-3
    for t in held:
        t.fill_(1)
    del held, t
    got = call(side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_legacy_handles():
    call = calls()["beam"]
    want = call(None)
    for handle in (0, 1):
        got = call(handle)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_capture_after_other_work():
    # Launches that may be set up early, captured behind a copy, behind another stream's work and
    # first of all.
    call = calls()["beam"]
    want = call(None)
    x = torch.zeros(1 << 20, device="cuda")
    y = torch.zeros(1 << 20).pin_memory()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other.wait_stream(torch.cuda.current_stream())
    call(other)  # (each stream has its workspace before the capture)
    with torch.cuda.stream(side):
        call(None)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = [call(None)]
            x.copy_(y, non_blocking=True)
            got.append(call(None))
            other.wait_stream(side)
            with torch.cuda.stream(other):
                x.add_(1)
                got.append(call(None))
            side.wait_stream(other)
            got.append(call(None))
    g.replay()
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_chains_of_calls_without_waits():
    # Each call reads what the one before it wrote: appends of a token, attention over it, forks
    # of both, with nothing between them that would hold the stream up.
    def run(wait):
        gen = torch.Generator("cuda").manual_seed(11)
        rows, page = 4, 16
        tables, refs = torch.full((rows, 8), -1, dtype=torch.int32, device="cuda"), torch.zeros(64, dtype=torch.int32, device="cuda")
        codes = [torch.zeros(64, 2, page, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.zeros(64, 2, device="cuda") for _ in range(2)]
        k, v, q, logits = (torch.randn(100, rows, *s, device="cuda", generator=gen) for s in ((2, 64), (2, 64), (4, 64), (300,)))
        k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
        lens = [torch.full((rows,), n, dtype=torch.int32, device="cuda") for n in range(102)]
        scores, outs = torch.zeros(2, 2, device="cuda"), []
        torch.cuda.synchronize()
        for i in range(100):
            tables, refs = K.kda_pages_alloc(tables, refs, lens[i // page + 1])
            wait()
            K.kda_kvcache_append(k[i], v[i], *codes, *scales, tables, lens[i])
            wait()
            outs.append(K.kda_kvcache_attention(q[i], *codes, *scales, tables, lens[i + 1]))
            wait()
            scores, tok, parents = K.kda_beam_select(logits[i].view(2, 2, 300), scores)
            wait()
            tables, refs = K.kda_pages_fork(tables, refs, parents.view(-1), lens=lens[i + 1], page_tokens=page, pools=codes + scales)
            wait()
            outs += [tok, parents, tables]
        return outs
    want = run(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))
    assert K.kda_get_device_status() == 0


def graph_of(call):
    """A graph of the call, captured on torch's own capture stream with no call before it there."""
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = call(None)
    return g, out


def attend_and_beam(seed):
    """Calls whose launches hand results on through scratch: parts of attention, candidates, copies."""
    gen = torch.Generator("cuda").manual_seed(seed)
    draw = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, scores = draw(2, 4, 50000), draw(2, 4)
    codes = [draw(64, 2, 64, 64).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.rand(64, 2, device="cuda", generator=gen) + 0.5 for _ in range(2)]
    tables = torch.randperm(64, device="cuda", generator=gen).to(torch.int32).view(2, 32)
    q1, q2 = draw(2, 16, 64).bfloat16(), draw(140, 16, 64).bfloat16()
    lens, cu = i32([2048, 1999]), i32([0, 70, 140])
    pool, refs, two = draw(64, 1000), torch.ones(64, dtype=torch.int32, device="cuda"), i32([1, 1])
    more = torch.cat([refs, torch.zeros(64, dtype=torch.int32, device="cuda")])
    big = torch.cat([pool, torch.zeros_like(pool)])

    def call(s):
        copy = big.clone()
        return [K.kda_kvcache_attention(q1, *codes, *scales, tables, lens, stream=s),
                K.kda_kvcache_attention(q2, *codes, *scales, tables, lens, cu_tokens=cu, stream=s),
                *K.kda_beam_select(x, scores, stream=s),
                *K.kda_pages_fork(tables, more, two, pools=[copy], stream=s), copy]
    return call


def test_capture_without_a_call_before_it():
    call = attend_and_beam(1)
    g, out = graph_of(call)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, call(None)))


def test_graphs_of_one_capture_stream_share_no_scratch():
    # replayed side by side on two streams, with calls on a third and on the capture stream's handle
    calls_ = [attend_and_beam(s) for s in (2, 3, 4)]
    want = [[t.clone() for t in c(None)] for c in calls_]
    graphs = [graph_of(c) for c in calls_[:2]]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(50):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            got = calls_[2](None)
    torch.cuda.synchronize()
    for (_, out), w in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    assert all(torch.equal(a, b) for a, b in zip(got, want[2]))


def test_graphs_outlive_calls_on_many_streams():
    call, other = attend_and_beam(5), attend_and_beam(6)
    want = [t.clone() for t in call(None)]
    g, out = graph_of(call)
    wide = torch.cuda.Stream(priority=-1)
    streams = [torch.cuda.Stream() for _ in range(40)] + [torch.cuda.Stream(priority=-1) for _ in range(40)] + [wide]
    handles = {s.cuda_stream for s in streams}
    assert len(handles) > 33
    keep = [other(s) for s in streams]
    torch.cuda.synchronize()
    fill = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and (fill == 0xFF).all()
    assert all(torch.equal(a, b) for k in keep for a, b in zip(k, keep[0]))


def beam_call(lib, x, scores, out, stream):
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    b, w, v = x.shape
    return lib.kda_beam_select(b, w, v, w, P(x), 0, v, P(scores), None, -1, P(out[0]), P(out[1]), P(out[2]), None, ctypes.c_void_p(stream))


def beam_out(b, w):
    return torch.empty(b, w, device="cuda"), *(torch.empty(b, w, dtype=torch.int32, device="cuda") for _ in range(2))


def test_threads_on_one_stream_share_no_scratch():
    # through the C ABI, whose calls run at the same time: the launches of two calls in any order
    lib = K.load_library()
    gen = torch.Generator("cuda").manual_seed(7)
    xs, scores = torch.randn(4, 1, 4, 20000, device="cuda", generator=gen), torch.zeros(1, 4, device="cuda")
    want = [K.kda_beam_select(x, scores) for x in xs]
    outs = [[beam_out(1, 4) for _ in range(300)] for _ in xs]
    stream = torch.cuda.Stream().cuda_stream
    torch.cuda.synchronize()

    def work(i):
        for o in outs[i]:
            assert beam_call(lib, xs[i], scores, o, stream) == 0

    with ThreadPoolExecutor(len(xs)) as pool:
        list(pool.map(work, range(len(xs))))
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for x in o for a, b in zip(x, w))


def test_scratch_of_a_callers_allocator():
    lib = K.load_library()
    x, scores = torch.randn(1, 4, 20000, device="cuda"), torch.zeros(1, 4, device="cuda")
    want, out = K.kda_beam_select(x, scores), beam_out(1, 4)
    stream = torch.cuda.current_stream().cuda_stream
    held, log = {}, []

    def allocate(context, size, s):
        if context == 7:
            return None
        t = torch.empty(size, dtype=torch.uint8, device="cuda")
        held[t.data_ptr()] = t
        log.append((size, s or 0))
        return t.data_ptr()

    def release(context, p, size, s):
        assert held.pop(p).numel() == size and log[-1] == (size, s or 0)

    a = KdaScratchAllocator(KdaScratchAllocator._fields_[0][1](allocate), KdaScratchAllocator._fields_[1][1](release), 0)
    before = KdaScratchAllocator()
    assert lib.kda_set_scratch_allocator(ctypes.byref(a), None) == 0
    try:
        assert beam_call(lib, x, scores, out, stream) == 0
        assert len(log) == 1 and not held and log[0][1] == stream
        assert all(torch.equal(p, q) for p, q in zip(K.kda_beam_select(x, scores), want))  # (torch's, and back)
        a.context = 7
        lib.kda_set_scratch_allocator(ctypes.byref(a), None)
        assert beam_call(lib, x, scores, out, stream) == 4 and b"scratch" in lib.kda_last_error_message()
    finally:
        assert lib.kda_set_scratch_allocator(None, ctypes.byref(before)) == 0
    assert before.context == 7
    assert beam_call(lib, x, scores, out, stream) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_per_thread_default_streams_share_no_scratch():
    # one handle for the streams of all threads
    lib = K.load_library()
    gen = torch.Generator("cuda").manual_seed(8)
    xs, scores = torch.randn(4, 1, 4, 20000, device="cuda", generator=gen), torch.zeros(1, 4, device="cuda")
    want = [K.kda_beam_select(x, scores) for x in xs]
    outs = [[beam_out(1, 4) for _ in range(300)] for _ in xs]
    torch.cuda.synchronize()

    def work(i):
        for o in outs[i]:
            assert beam_call(lib, xs[i], scores, o, 2) == 0

    with ThreadPoolExecutor(len(xs)) as pool:
        list(pool.map(work, range(len(xs))))
    got = K.kda_beam_select(xs[0], scores, stream=2)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for x in o for a, b in zip(x, w))
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
