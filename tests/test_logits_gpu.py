"""Penalties, biases and masks on logits against 64 bits.

Allowed: the rounding to the logits' type (half a step), and for the fp32 steps before it (a quotient or
product, two subtractions, the biases' additions) 2^-24 of what each of them works on: twice the sum of
the magnitudes that enter, for each step.  Logits that no rule touches keep their bits."""
import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
from step_testutil import DT, ints

pytestmark = pytest.mark.gpu


def reference(x, rules):
    """(values, sum of magnitudes, touched) in 64 bits; x [R, V]."""
    y, size, touched = x.astype(np.float64).copy(), np.abs(x).astype(np.float64), np.zeros(x.shape, bool)
    rows, vocab = x.shape
    for r in range(rows):
        if "history" in rules:
            h = rules["history"][r]
            n = int(np.clip(rules["lens"][r], 0, len(h))) if "lens" in rules else len(h)
            p = int(np.clip(rules["prompt_lens"][r], 0, n)) if "prompt_lens" in rules else 0
            g = [float(rules[k][r]) if k in rules else d for k, d in (("repetition", 1.0), ("presence", 0.0), ("frequency", 0.0))]
            if not (np.isfinite(g).all() and g[0] > 0):
                g = [1.0, 0.0, 0.0]
            behind = np.bincount([t for t in h[p:n].tolist() if 0 <= t < vocab], minlength=vocab)
            for t in set(h[:n].tolist()):
                if not 0 <= t < vocab:
                    continue
                c = int(behind[t])
                y[r, t] = y[r, t] / g[0] if y[r, t] > 0 else y[r, t] * g[0]
                size[r, t] += abs(y[r, t]) + abs(g[2] * c) + abs(g[1])
                y[r, t] -= (g[2] * c + g[1]) if c else 0.0
                touched[r, t] = True
        if "bias" in rules:
            for t, b in zip(rules["bias_tokens"][r].tolist(), rules["bias"][r].tolist()):
                if 0 <= t < vocab:
                    y[r, t] += b
                    size[r, t] += abs(b)
                    touched[r, t] = True
        if "mask" in rules:
            bits = np.unpackbits(rules["mask"][r].view(np.uint8), bitorder="little")[:vocab]
            y[r, bits == 0] = -np.inf
    return y, size, touched


def make(rng, rows, vocab, width=0, biases=0, mask=None, lens=True):
    rules = {}
    if width:
        rules["history"] = (vocab * rng.random((rows, width)) ** 3).astype(np.int64).clip(0, vocab - 1)
        rules["history"][:, ::17] = -1
        if lens:
            rules["lens"] = rng.integers(0, width + 1, rows)
            rules["prompt_lens"] = (rules["lens"] * rng.random(rows)).astype(np.int64)
        rules["repetition"], rules["presence"], rules["frequency"] = (f(rng.random(rows)).astype(np.float32) for f in (
            lambda u: 0.7 + u, lambda u: 2 * u - 0.5, lambda u: u - 0.3))
    if biases:
        rules["bias_tokens"] = rng.integers(-1, vocab, (rows, biases))
        rules["bias"] = rng.standard_normal((rows, biases)).astype(np.float32) * 5
    if mask is not None:
        bits = (rng.random((rows, (vocab + 31) // 32 * 32)) < mask).astype(np.uint8)
        rules["mask"] = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
    return rules


def call(x, rules, **kw):
    t = {k: ints(v) if v.dtype == np.int64 else torch.as_tensor(v).cuda() for k, v in rules.items()}
    return K.kda_logits_penalize(x, **t, **kw)


def check(got, x, rules, dtype, adds=0):
    want, size, touched = reference(x.double().numpy().reshape(-1, x.shape[-1]), rules)
    got = got.cpu()
    flat = got.reshape(want.shape)
    masked = np.isneginf(want)
    g = flat.double().numpy()
    assert np.isneginf(g[masked]).all()
    same = torch.as_tensor(~touched & ~masked)
    assert torch.equal(flat[same], x.reshape(want.shape)[same])
    eps = torch.finfo(DT[dtype]).eps / 2
    ok = touched & ~masked
    allowed = eps * np.abs(want) + (4 + adds) * 2.0 ** -23 * size + (2.0 ** -24 if dtype == "fp16" else 0)
    with np.errstate(invalid="ignore"):
        off = np.abs(g - want) > allowed
    assert not (off & ok).any(), np.max((np.abs(g - want) / allowed)[ok])


@pytest.mark.parametrize("vocab", [1, 7, 32, 33, 500, 4097, 32001, 70000])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_everything_together(vocab, dtype):
    rng = np.random.default_rng(vocab)
    rules = make(rng, 6, vocab, width=100, biases=33, mask=0.6)
    x = torch.as_tensor(rng.standard_normal((2, 3, vocab)) * 5).to(DT[dtype])
    got = call(x.cuda(), rules)
    assert got.shape == x.shape and got.dtype == x.dtype and got.is_contiguous()
    check(got, x, rules, dtype, adds=33)
    y = x.cuda()
    assert call(y, rules, out=y).data_ptr() == y.data_ptr()
    assert torch.equal(y, got)


@pytest.mark.parametrize("rules", [dict(width=1), dict(width=5000, lens=False), dict(biases=1), dict(biases=700), dict(mask=0.0), dict(mask=0.02),
                                   dict(mask=0.98), dict(mask=1.0), dict(width=40, mask=0.5), dict()])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("place", [False, True])
def test_rules_alone(rules, dtype, place):
    rng = np.random.default_rng(3)
    made = make(rng, 5, 12345, **rules)
    x = torch.as_tensor(rng.standard_normal((5, 12345)) * 5).to(DT[dtype])
    y = x.cuda()
    check(call(y, made, out=y if place else None), x, made, dtype, adds=rules.get("biases", 0))


@pytest.mark.parametrize("rows,vocab", [(1, 300000), (3, 131072), (40, 50257), (300, 9000)])
def test_large(rows, vocab):
    rng = np.random.default_rng(rows)
    made = make(rng, rows, vocab, width=300, biases=20, mask=0.9)
    x = torch.as_tensor(rng.standard_normal((rows, vocab)).astype(np.float32) * 5).to(torch.bfloat16)
    check(call(x.cuda(), made), x, made, "bf16", adds=20)


# Rows enough that a row is one segment, of several chunks: with edges outside of 16-byte loads, and all touched tokens
# in one chunk.
@pytest.mark.parametrize("dtype,vocab", [("bf16", 25003), ("fp16", 8201), ("fp32", 8193)])
@pytest.mark.parametrize("pad,skip", [(0, 0), (1, 1), (24, 3)])
@pytest.mark.parametrize("rules", [dict(width=300, biases=20, mask=0.9), dict(width=64, biases=600), dict(mask=0.3), dict(width=7000, lens=False)])
def test_segments_of_several_chunks(dtype, vocab, pad, skip, rules):
    rng = np.random.default_rng(vocab + pad)
    rows = 300
    made = make(rng, rows, vocab, **rules)
    if rules.get("biases") == 600:
        made["history"] = np.where(made["history"] >= 0, 8192 - made["history"] % 90, -1)
        made["bias_tokens"] %= 100
    whole = torch.as_tensor(rng.standard_normal((rows, vocab + pad)).astype(np.float32) * 5).to(DT[dtype])
    x = whole[:, skip: skip + vocab]
    target = torch.zeros(rows, vocab + pad, device="cuda", dtype=DT[dtype])
    call(whole.cuda()[:, skip: skip + vocab], made, out=target[:, skip: skip + vocab])
    check(target[:, skip: skip + vocab], x, made, dtype, adds=rules.get("biases", 0))
    assert (target[:, :skip] == 0).all() and (target[:, skip + vocab:] == 0).all()


def test_vocabularies_past_a_segments_chunks():
    rng = np.random.default_rng(4)
    made = make(rng, 300, 600_001, width=50, biases=3, mask=0.9)
    x = torch.randn(300, 600_001, device="cuda").to(torch.bfloat16)
    assert torch.equal(call(x, made), call(x.clone(), made, out=x))


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
@pytest.mark.parametrize("pad,skip", [(24, 0), (1, 0), (7, 3), (64, 1)])
def test_padded_and_shifted_rows(dtype, pad, skip):
    rng = np.random.default_rng(pad)
    vocab, rows = 5001, 7
    made = make(rng, rows, vocab, width=64, biases=5, mask=0.5)
    whole = torch.as_tensor(rng.standard_normal((rows, vocab + pad)) * 5).to(DT[dtype])
    x, dev = whole[:, skip: skip + vocab], whole.cuda()
    view = dev[:, skip: skip + vocab]
    check(call(view, made), x, made, dtype, adds=5)
    target = torch.zeros(rows, vocab + 3, device="cuda", dtype=DT[dtype])
    call(view, made, out=target[:, 2: 2 + vocab])
    check(target[:, 2: 2 + vocab], x, made, dtype, adds=5)
    assert (target[:, :2] == 0).all() and (target[:, vocab + 2:] == 0).all()
    assert torch.equal(dev.cpu(), whole)
    call(view, made, out=view)
    check(view, x, made, dtype, adds=5)
    edges = torch.ones(vocab + pad, dtype=torch.bool)
    edges[skip: skip + vocab] = False
    assert torch.equal(dev.cpu()[:, edges], whole[:, edges])


def test_lengths_and_tokens_out_of_range_are_recorded():
    rng = np.random.default_rng(5)
    base = make(rng, 4, 1000, width=50, biases=6)
    x = torch.as_tensor(rng.standard_normal((4, 1000)).astype(np.float32))
    K.kda_get_device_status()
    check(call(x.cuda(), base), x, base, "fp32", adds=6)
    assert K.kda_get_device_status() == 0
    for key, at, value in (("history", (1, 1), 1000), ("history", (1, 1), 2 ** 31 - 1), ("bias_tokens", (2, 0), 1000), ("lens", 3, 51), ("lens", 3, -1),
                           ("repetition", 0, 0.0), ("repetition", 0, float("nan")), ("repetition", 0, float("inf")), ("presence", 1, float("inf")),
                           ("frequency", 2, float("nan"))):
        rules = {k: v.copy() for k, v in base.items()}
        rules["lens"][1] = 50
        rules[key][at] = value
        check(call(x.cuda(), rules), x, rules, "fp32", adds=6)
        assert K.kda_get_device_status() == 1, (key, value)
    rules = {k: v.copy() for k, v in base.items()}  # prompts of any length are taken as the history's
    rules["prompt_lens"][:2] = [-5, 10 ** 6]
    check(call(x.cuda(), rules), x, rules, "fp32", adds=6)
    assert K.kda_get_device_status() == 0


def test_logits_that_are_not_finite():
    x = torch.tensor([[float("inf"), -float("inf"), float("nan"), 1.0, -1.0, 60000.0, -0.0, 5.0]]).half()
    h = np.arange(8)[None].repeat(3, 1)[:1]
    got = call(x.cuda(), dict(history=h, repetition=np.float32([0.5]), presence=np.float32([1.0]))).cpu()[0]
    assert got[0] == float("inf") and got[1] == -float("inf") and torch.isnan(got[2])
    assert got[3] == 1.0 and got[4] == -1.5 and got[5] == float("inf") and got[6] == -1.0 and got[7] == 9.0
    got = call(x.cuda(), dict(mask=np.int32([[0b01000000]]))).cpu()[0]
    assert torch.isneginf(got[[0, 1, 2, 3, 4, 5, 7]]).all() and got[6] == 0
    got = call(x.cuda(), dict(bias_tokens=np.int64([[3, 3, 4]]), bias=np.float32([[float("-inf"), 2.0, 1e30]]))).cpu()[0]
    assert got[3] == -float("inf") and got[4] == float("inf")


def test_biases_of_one_token_are_added_in_order():
    n = 1000
    rng = np.random.default_rng(9)
    bias = (rng.standard_normal((1, n)) * 10.0 ** rng.integers(-3, 4, (1, n))).astype(np.float32)
    tokens = np.where(rng.random((1, n)) < 0.7, 77, rng.integers(0, 100, (1, n)))
    x = torch.zeros(1, 5000)
    got = call(x.cuda(), dict(bias_tokens=tokens, bias=bias)).cpu()[0]
    want = np.zeros(5000, np.float32)
    for t, b in zip(tokens[0], bias[0]):
        want[t] = np.float32(want[t] + b)
    assert np.array_equal(got.numpy(), want)  # (x is 0: the sum alone)


def test_empty_calls():
    x = torch.randn(2, 3, 100, device="cuda")
    assert torch.equal(K.kda_logits_penalize(x), x)
    none = torch.zeros(2, 3, 0, dtype=torch.int32, device="cuda")
    one = torch.ones(2, 3, device="cuda")
    assert torch.equal(K.kda_logits_penalize(x, history=none, lens=none.sum(2, dtype=torch.int32), repetition=2 * one), x)
    assert K.kda_logits_penalize(x[:0]).shape == (0, 3, 100)
    assert torch.equal(K.kda_logits_penalize(x[0, 0]), x[0, 0])
    # rows in one dimension or in logits' own
    h = torch.randint(0, 100, (2, 3, 9), dtype=torch.int32, device="cuda")
    a = K.kda_logits_penalize(x, history=h, repetition=2 * one)
    assert torch.equal(a, K.kda_logits_penalize(x, history=h.view(6, 9), repetition=2 * one.view(6)))


def test_streams_and_graphs():
    rng = np.random.default_rng(11)
    made = make(rng, 6, 30011, width=200, biases=10, mask=0.7)
    x = torch.as_tensor(rng.standard_normal((6, 30011)).astype(np.float32)).cuda()
    want = call(x, made)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t = {k: ints(v) if v.dtype == np.int64 else torch.as_tensor(v).cuda() for k, v in made.items()}
    torch.cuda.synchronize()
    got = K.kda_logits_penalize(x, **t, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    moved = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = K.kda_logits_penalize(moved, **t)
    moved.copy_(x)
    graph.replay()
    graph.replay()
    assert torch.equal(got, want)


def test_refusals():
    x = torch.zeros(4, 100, device="cuda")
    h, n, f = torch.zeros(4, 9, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(4, device="cuda")
    words = torch.zeros(4, 4, dtype=torch.int32, device="cuda")
    for bad in (dict(logits=x.double()), dict(logits=x.cpu()), dict(logits=x.t()), dict(history=h.long()), dict(history=h[:3]), dict(history=h.t()),
                dict(lens=n), dict(repetition=f), dict(history=h, lens=f), dict(history=h, repetition=f.double()), dict(history=h, presence=f[:2]),
                dict(bias_tokens=h), dict(bias=f.view(4, 1)), dict(bias_tokens=h, bias=f.view(4, 1)), dict(mask=words[:, :3].contiguous()),
                dict(mask=words.long()), dict(mask=words.cpu()), dict(out=x.half()), dict(out=x[:3]), dict(out=x.cpu())):
        a = dict(logits=x, **bad) if "logits" not in bad else bad
        with pytest.raises(ValueError):
            K.kda_logits_penalize(**a)
    whole = torch.zeros(8, 100, device="cuda")
    with pytest.raises(K.KdaError):
        K.kda_logits_penalize(whole[:4], out=whole[1:5])
    with pytest.raises(K.KdaError):
        K.kda_logits_penalize(x[:1].expand(4, 100))
