"""Host-side refusals of the serving operators: bad arguments are rejected with the documented
status before any device work."""
import ctypes

import pytest
import torch

import chunked_kda_delta_gb300 as K
from chunked_kda_delta_gb300 import build as kbuild
from chunked_kda_delta_gb300.kda import KdaKvCache, KdaPageShape, KdaPool, KdaShape
from chunked_kda_delta_gb300.kda import KdaScratchAllocator

# Calls that pass validation go on with made-up addresses: they must not reach a GPU.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses")

INVALID, ALIAS = 1, 2
P = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return K.load_library()


def fork(lib, shape=(4, 3, 10), pools=(), num_pools=None, page_tokens=16, **over):
    a = dict(tables=0x1000, refs=0x2000, parents=0x3000, lens=0x4000, nt=0x5000, nr=0x6000)
    a.update(over)
    arr = (KdaPool * max(1, len(pools)))(*pools)
    return lib.kda_pages_fork(None if shape is None else ctypes.byref(KdaPageShape(*shape)), P(a["tables"]), P(a["refs"]),
                              P(a["parents"]), P(a["lens"]), page_tokens, arr,
                              len(pools) if num_pools is None else num_pools, P(a["nt"]), P(a["nr"]), None)


def test_fork_rules(lib):
    assert fork(lib) not in (INVALID, ALIAS)
    assert fork(lib, shape=None) == INVALID
    for shape in ((-1, 3, 10), (4, 0, 10), (4, 3, -1), (1 << 20, 1 << 20, 10)):
        assert fork(lib, shape=shape) == INVALID
    for name in ("tables", "refs", "parents", "lens", "nt", "nr"):
        assert fork(lib, **{name: None}) == INVALID
        assert fork(lib, **{name: 0x7002}) == INVALID
    assert fork(lib, lens=None, page_tokens=0) not in (INVALID, ALIAS)
    assert fork(lib, page_tokens=-1) == INVALID
    assert fork(lib, nt=0x1004) == ALIAS
    assert fork(lib, nr=0x3000) == ALIAS
    assert fork(lib, nt=0x6008) == ALIAS
    assert b"overlaps" in lib.kda_last_error_message()


def test_pool_rules(lib):
    good = KdaPool(0x100000, 64, 64, 640, 2)
    assert fork(lib, pools=[good]) not in (INVALID, ALIAS)
    for bad in (KdaPool(None, 64, 64, 640, 1), KdaPool(0x100000, 64, 32, 640, 1), KdaPool(0x100000, -1, 64, 640, 1),
                KdaPool(0x100000, 64, 64, 640, -1), KdaPool(0x100000, 64, 64, 320, 2),
                KdaPool(0x100000, 64, 1 << 46, 640, 1), KdaPool(0x100000, 64, 64, 1 << 50, 2), KdaPool(0x100000, 64, 64, -640, 2)):
        assert fork(lib, pools=[bad]) == INVALID
    # layers inside the page stride ([pages][layers] order) are fine
    assert fork(lib, pools=[KdaPool(0x100000, 64, 128, 64, 2)]) not in (INVALID, ALIAS)
    assert fork(lib, pools=[KdaPool(0x5000, 64, 64, 640, 1)]) == ALIAS
    assert fork(lib, pools=[good], num_pools=65) == INVALID
    assert fork(lib, pools=[good], num_pools=-1) == INVALID


def test_other_page_rules(lib):
    s = ctypes.byref(KdaPageShape(4, 3, 10))
    assert lib.kda_pages_alloc(s, P(0x1000), P(0x2000), None, P(0x5000), P(0x6000), None) == INVALID
    assert lib.kda_pages_free(s, P(0x1000), P(0x2000), None, P(0x5000), P(0x6000), None) == INVALID
    assert lib.kda_pages_free(s, P(0x1000), P(0x2000), P(0x5001), P(0x5000), P(0x6000), None) == ALIAS
    pool = (KdaPool * 1)(KdaPool(0x100000, 64, 64, 0, 1))
    call = lambda pm, nl: lib.kda_pages_compact(s, P(0x1000), P(0x2000), pool, 1, P(0x5000), P(0x6000), P(pm), P(nl), None)  # noqa: E731
    assert call(0x7000, 0x8000) not in (INVALID, ALIAS)
    assert call(None, 0x8000) == INVALID and call(0x7000, None) == INVALID
    assert call(0x7000, 0x7004) == ALIAS and call(0x2000, 0x8000) == ALIAS
    assert lib.kda_pages_copy(-1, 1, P(0x1000), P(0x2000), pool, 1, None) == INVALID
    assert lib.kda_pages_copy(10, 1, None, P(0x2000), pool, 1, None) == INVALID
    assert lib.kda_pages_copy(10, 1, P(0x100040), P(0x2000), pool, 1, None) == ALIAS


def cache(**over):
    a = dict(k=0x10000000, v=0x20000000, ks=0x30000000, vs=0x40000000, pages=8, page=16, heads=2, dim=64, tables=0x50000000, rows=3, width=4)
    a.update(over)
    return KdaKvCache(a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["page"], a["heads"], a["dim"], a["tables"], a["rows"], a["width"])


def attend(lib, c=None, q=0x60000000, hq=4, act=0, qs=256, n=3, lens=0x70000000, cu=None, scale=0.1, out=0x71000000, os=256):
    return lib.kda_kvcache_attention(ctypes.byref(c or cache()), P(q), hq, act, qs, n, P(lens), P(cu), ctypes.c_float(scale), P(out), os, None)


def append(lib, c=None, k=0x60000000, v=0x61000000, act=0, ks=128, vs=128, n=3, lens=0x70000000, cu=None):
    return lib.kda_kvcache_append(ctypes.byref(c or cache()), P(k), P(v), act, ks, vs, n, P(lens), P(cu), None)


@pytest.mark.parametrize("call", [attend, append])
def test_cache_rules(lib, call):
    assert call(lib) not in (INVALID, ALIAS)
    for bad in (dict(page=24), dict(dim=96), dict(heads=0), dict(pages=-1), dict(rows=-1), dict(width=0), dict(k=None),
                dict(v=0x20000008), dict(ks=None), dict(vs=0x40000002), dict(tables=None)):
        assert call(lib, c=cache(**bad)) == INVALID, bad
    assert call(lib, n=4) == INVALID            # one token for each of the three rows
    assert call(lib, n=4, cu=0x72000000) not in (INVALID, ALIAS)
    assert call(lib, n=-1, cu=0x72000000) == INVALID
    assert call(lib, cu=0x72000002) == INVALID
    assert call(lib, act=2) == INVALID
    assert call(lib, lens=None) == INVALID
    assert lib.kda_kvcache_append(None, None, None, 0, 128, 128, 0, None, None, None) == INVALID


def test_attention_rules(lib):
    assert attend(lib, hq=3) == INVALID and attend(lib, hq=0) == INVALID
    assert attend(lib, qs=252) == INVALID and attend(lib, qs=128) == INVALID and attend(lib, os=8) == INVALID
    assert attend(lib, q=None) == INVALID and attend(lib, q=0x60000008) == INVALID and attend(lib, out=None) == INVALID
    assert attend(lib, scale=float("nan")) == INVALID and attend(lib, scale=float("inf")) == INVALID
    assert attend(lib, out=0x60000100) == ALIAS and attend(lib, out=0x10000000) == ALIAS and attend(lib, out=0x70000000) == ALIAS


def test_append_rules(lib):
    assert append(lib, k=None) == INVALID and append(lib, v=0x61000002) == INVALID
    assert append(lib, ks=64) == INVALID and append(lib, vs=132) == INVALID
    assert append(lib, k=0x10000000) == ALIAS and append(lib, c=cache(v=0x10000000)) == ALIAS
    assert append(lib, c=cache(vs=0x50000000)) == ALIAS


def beam(lib, batch=2, beams=3, vocab=100, k=3, logits=0x10000000, dt=0, stride=100, scores=0x20000000, done=None, eos=-1,
         ns=0x30000000, tok=0x40000000, par=0x50000000, nd=None):
    return lib.kda_beam_select(batch, beams, vocab, k, P(logits), dt, stride, P(scores), P(done), eos, P(ns), P(tok), P(par), P(nd), None)


def test_beam_rules(lib):
    assert beam(lib) not in (INVALID, ALIAS)
    for bad in (dict(batch=-1), dict(beams=0), dict(beams=65), dict(k=0), dict(k=65), dict(vocab=0), dict(stride=99), dict(dt=3),
                dict(beams=64, vocab=1 << 26, stride=1 << 26), dict(eos=100), dict(eos=-2), dict(done=0x60000000),
                dict(logits=None), dict(logits=0x10000002), dict(scores=None), dict(ns=None), dict(tok=0x40000001), dict(par=None)):
        assert beam(lib, **bad) == INVALID, bad
    assert beam(lib, dt=1, logits=0x10000002) not in (INVALID, ALIAS)
    assert beam(lib, done=0x60000000, eos=0, nd=0x61000000) not in (INVALID, ALIAS)
    assert beam(lib, ns=0x20000004) == ALIAS and beam(lib, tok=0x10000100) == ALIAS and beam(lib, par=0x40000004) == ALIAS


def test_paged_decode_rules(lib):
    def call(shape=(2, 1, 0, 2, 128, 0), states=0x70000000, pages=4, stride=32768, at=0x78000000, dt=0, out=0x60000000):
        return lib.kda_decode_paged(ctypes.byref(KdaShape(*shape)), P(0x10000000), P(0x20000000), P(0x30000000), P(0x40000000),
                                    P(0x50000000), ctypes.c_float(0.1), P(states), pages, stride, P(at), dt, P(out), None)

    assert call() not in (INVALID, ALIAS)
    assert call(shape=(2, 1, 0, 2, 128, 4)) == INVALID       # grouped query heads
    assert call(shape=(2, 1, 0, 4, 128, 2), stride=65536) not in (INVALID, ALIAS)
    assert call(states=None) == INVALID and call(states=0x70000008) == INVALID and call(pages=-1) == INVALID
    assert call(stride=16384) == INVALID and call(stride=32772) == INVALID and call(stride=1 << 46) == INVALID
    assert call(at=None) == INVALID and call(at=0x78000002) == INVALID and call(dt=2) == INVALID
    assert call(out=0x70000100) == ALIAS and call(at=0x70000000) == ALIAS


def test_binding_refuses_cpu_tensors_and_wrong_types():
    t = torch.zeros(2, 2, dtype=torch.int32)
    r = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        K.kda_pages_fork(t, r, r[:2])
    with pytest.raises(ValueError):
        K.kda_pages_compact(t, r)
    with pytest.raises(ValueError):
        K.kda_beam_select(torch.zeros(1, 2, 10), torch.zeros(1, 2))
    c = torch.zeros(4, 1, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        K.kda_kvcache_attention(torch.zeros(1, 1, 64), c, c, torch.zeros(4, 1), torch.zeros(4, 1), t[:1], r[:1])


def test_scratch_allocator_rules(lib):
    fields = KdaScratchAllocator._fields_
    one = KdaScratchAllocator(fields[0][1](lambda c, n, s: None), fields[1][1](), 5)
    assert lib.kda_set_scratch_allocator(ctypes.byref(one), None) == INVALID
    both = KdaScratchAllocator(fields[0][1](lambda c, n, s: None), fields[1][1](lambda c, p, n, s: None), 5)
    before = KdaScratchAllocator()
    assert lib.kda_set_scratch_allocator(ctypes.byref(both), ctypes.byref(before)) == 0 and not before.context
    assert lib.kda_set_scratch_allocator(None, ctypes.byref(before)) == 0 and before.context == 5
    assert lib.kda_set_scratch_allocator(None, None) == 0
