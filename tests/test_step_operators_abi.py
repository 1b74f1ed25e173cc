"""Host-side refusals of a decoding step's operators: bad arguments are rejected with the documented
status before any device work."""
import ctypes

import pytest
import torch

import chunked_kda_delta_gb300 as K
from chunked_kda_delta_gb300 import build as kbuild
from chunked_kda_delta_gb300.kda import KdaKvCache, KdaLogitsRules

# Calls that pass validation go on with made-up addresses: they must not reach a GPU.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses")

INVALID, ALIAS = 1, 2
P = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return K.load_library()


def cache(**over):
    a = dict(k=0x10000000, v=0x20000000, ks=0x30000000, vs=0x40000000, pages=8, page=16, heads=2, dim=64, tables=0x50000000, rows=3, width=4)
    a.update(over)
    return KdaKvCache(a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["page"], a["heads"], a["dim"], a["tables"], a["rows"], a["width"])


def rotary(lib, c=None, q=0x60000000, k=0x61000000, v=0x62000000, hq=4, act=0, qs=256, ks=128, vs=128, n=3, lens=0x70000000, cu=None,
           table=0x71000000, positions=100, rot=64, inter=0, at=None, out=0x72000000, os=256):
    return lib.kda_kvcache_append_rotary(ctypes.byref(c or cache()), P(q), P(k), P(v), hq, act, qs, ks, vs, n, P(lens), P(cu), P(table), positions,
                                         rot, inter, P(at), P(out), os, None)


def test_rotary_rules(lib):
    assert rotary(lib) not in (INVALID, ALIAS)
    for bad in (dict(page=24), dict(dim=96), dict(heads=0), dict(pages=-1), dict(rows=-1), dict(width=0), dict(k=None), dict(v=0x20000008),
                dict(ks=None), dict(vs=0x40000002), dict(tables=None)):
        assert rotary(lib, c=cache(**bad)) == INVALID, bad
    for bad in (dict(act=2), dict(hq=0), dict(hq=1 << 17), dict(n=4), dict(n=-1, cu=0x73000000), dict(cu=0x73000002), dict(lens=None), dict(q=None),
                dict(q=0x60000008), dict(qs=128), dict(qs=260), dict(ks=64), dict(vs=132), dict(k=None), dict(v=0x62000002), dict(out=None),
                dict(out=0x72000008), dict(os=128), dict(table=None), dict(table=0x71000004), dict(rot=0), dict(rot=24), dict(rot=80), dict(rot=-16),
                dict(positions=-1), dict(positions=1 << 40), dict(at=0x73000002)):
        assert rotary(lib, **bad) == INVALID, bad
    assert rotary(lib, hq=5, qs=320, os=320) not in (INVALID, ALIAS)       # any number of query heads
    assert rotary(lib, table=None, positions=0) not in (INVALID, ALIAS)


def test_rotary_overlaps(lib):
    assert rotary(lib, out=0x60000000) not in (INVALID, ALIAS)              # in place
    assert rotary(lib, out=0x60000000, os=264) == ALIAS                     # at another stride
    for bad in (dict(out=0x60000010), dict(out=0x61000000), dict(out=0x62000010), dict(out=0x10000000), dict(out=0x30000000), dict(out=0x50000000),
                dict(out=0x70000000), dict(out=0x71000000), dict(at=0x73000000, out=0x73000000), dict(k=0x10000000), dict(q=0x20000000),
                dict(table=0x10000000), dict(at=0x30000000)):
        assert rotary(lib, **bad) == ALIAS, bad
    # heads of one fused projection [tokens][q 4, k 2, v 2]: q in place between its neighbours
    fused = dict(q=0x60000000, k=0x60000000 + 512, v=0x60000000 + 768, qs=512, ks=512, vs=512, os=512)
    assert rotary(lib, out=0x60000000, **fused) not in (INVALID, ALIAS)
    assert rotary(lib, out=0x60000000 + 128, **fused) == ALIAS
    assert rotary(lib, out=0x60000000 - 128, **fused) == ALIAS
    assert rotary(lib, out=0x60000000 - 512, **dict(fused, os=1024)) == ALIAS


def logits(lib, rows=4, vocab=100, x=0x10000000, dt=0, stride=100, out=0x20000000, os=100, **rules):
    r = dict(history=0x30000000, lens=0x31000000, prompt_lens=0x32000000, repetition=0x33000000, presence=0x34000000, frequency=0x35000000,
             bias_tokens=0x36000000, bias=0x37000000, mask=0x38000000, mask_stride=4, history_width=20, num_bias=5)
    r.update(rules)
    s = KdaLogitsRules(**r)
    return lib.kda_logits_penalize(ctypes.byref(s), rows, vocab, P(x), dt, stride, P(out), os, None)


def test_logits_rules(lib):
    assert logits(lib) not in (INVALID, ALIAS)
    assert logits(lib, **{k: None for k in ("lens", "prompt_lens", "repetition", "presence", "frequency", "mask")}) not in (INVALID, ALIAS)
    assert logits(lib, history=None, history_width=0, bias=None, bias_tokens=None, num_bias=0) not in (INVALID, ALIAS)
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(vocab=0), dict(vocab=(1 << 30) + 1, stride=1 << 31, os=1 << 31), dict(dt=3),
                dict(stride=99), dict(os=99), dict(stride=1 << 33), dict(x=None), dict(x=0x10000002), dict(out=None), dict(out=0x20000001), dict(history=None),
                dict(history=0x30000002), dict(history_width=-1), dict(num_bias=-1), dict(bias=None), dict(bias_tokens=0x36000001), dict(lens=0x31000002),
                dict(repetition=0x33000001), dict(mask=0x38000002), dict(mask_stride=3)):
        assert logits(lib, **bad) == INVALID, bad
    assert lib.kda_logits_penalize(None, 1, 100, P(0x10000000), 0, 100, P(0x20000000), 100, None) == INVALID
    assert logits(lib, dt=1, x=0x10000002, out=0x20000002) not in (INVALID, ALIAS)


def test_logits_overlaps(lib):
    assert logits(lib, out=0x10000000) not in (INVALID, ALIAS)               # in place
    for bad in (dict(out=0x10000004), dict(out=0x10000000, os=104), dict(out=0x30000000), dict(out=0x31000000), dict(out=0x34000000), dict(out=0x36000008),
                dict(out=0x37000008), dict(out=0x38000010)):
        assert logits(lib, **bad) == ALIAS, bad


def attend(lib, c=None, q=0x60000000, hq=4, act=0, qs=256, n=3, lens=0x70000000, cu=None, rows=0x73000000, groups=2, scale=0.1, out=0x71000000, os=256):
    return lib.kda_kvcache_attention_shared(ctypes.byref(c or cache()), P(q), hq, act, qs, n, P(lens), P(cu), P(rows), groups, ctypes.c_float(scale), P(out),
                                            os, None)


def test_shared_attention_rules(lib):
    assert attend(lib) not in (INVALID, ALIAS)
    for bad in (dict(page=24), dict(dim=96), dict(heads=0), dict(pages=-1), dict(rows=-1), dict(width=0), dict(k=None), dict(tables=None)):
        assert attend(lib, c=cache(**bad)) == INVALID, bad
    for bad in (dict(rows=None), dict(rows=0x73000002), dict(groups=0), dict(groups=-1), dict(groups=1 << 25), dict(hq=3), dict(hq=0), dict(qs=252),
                dict(qs=128), dict(os=8), dict(q=None), dict(out=None), dict(n=4), dict(n=-1, cu=0x72000000), dict(act=2), dict(lens=None),
                dict(scale=float("nan"))):
        assert attend(lib, **bad) == INVALID, bad
    for bad in (dict(out=0x60000100), dict(out=0x10000000), dict(out=0x70000000), dict(out=0x73000000), dict(out=0x50000000)):
        assert attend(lib, **bad) == ALIAS, bad
    assert lib.kda_kvcache_attention_shared(None, None, 1, 0, 64, 0, None, None, P(0x73000000), 0, ctypes.c_float(1), None, 64, None) == INVALID
