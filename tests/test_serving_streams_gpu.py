"""The serving operators on a stream that is not the current one: given as a torch stream or as a
raw handle, with results whose memory no pending work of the current stream still writes."""
import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
from chunked_kda_delta_gb300.inputs import custom, make_inputs

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
