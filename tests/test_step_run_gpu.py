"""The operators of a decoding step one after another, as a server runs them: prompts into the cache with their
rotation, then steps of penalised beam selection, forked pages, rotating appends and attention over the prefixes that
the beams share.  Every call is held against 64 bits on what the calls before it left; the bounds are those of
the operators' own tests."""
import os
import sys

import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
import serving_testutil as ref
from step_testutil import F8, check_quantised, cu_of, ints, rotary_table, rotate
from test_logits_gpu import check as check_logits

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


class Run:
    """`requests` of `beams` rows; tables wide enough that sharing pays."""

    def __init__(self, requests=2, beams=8, hq=8, hkv=2, d=64, page=16, vocab=500, rot=32, interleaved=False):
        self.rng = np.random.default_rng(beams + d)
        self.requests, self.beams, self.rows, self.page, self.vocab, self.inter = requests, beams, requests * beams, page, vocab, interleaved
        g = torch.Generator(device="cuda").manual_seed(1)
        self.embed = torch.randn(vocab, hq + 2 * hkv, d, generator=g, device="cuda").to(torch.bfloat16)
        self.head = torch.randn(hq * d, vocab, generator=g, device="cuda").to(torch.bfloat16)
        self.split, self.d = [hq, hkv, hkv], d
        width, pages = 250_000 // page, 40 * self.rows
        self.cache = [torch.zeros(pages, hkv, page, d, dtype=F8, device="cuda") for _ in range(2)] + [torch.zeros(pages, hkv, device="cuda") for _ in range(2)]
        self.tables = torch.full((self.rows, width), -1, dtype=torch.int32, device="cuda")
        self.refs, self.lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (pages, self.rows))
        self.rotary = rotary_table(700, rot)
        self.groups = cu_of([beams] * requests)

    def append(self, tokens, counts, shared):
        """Appends tokens (int64, all rows' one after another) and returns attention's output, both checked."""
        after = self.lens + ints(counts)
        self.tables, self.refs = K.kda_pages_alloc(self.tables, self.refs, -(-after // self.page))
        x = self.embed[tokens]
        q, k, v = x.split(self.split, 1)
        before = [c.view(torch.uint8).cpu().numpy().copy() if c.dtype == F8 else c.cpu().numpy().copy() for c in self.cache]
        cu = None if all(n == 1 for n in counts) else cu_of(counts)
        turned = K.kda_kvcache_append_rotary(q, k, v, torch.as_tensor(self.rotary).cuda(), *self.cache, self.tables, self.lens, cu_tokens=cu,
                                             interleaved=self.inter)
        call = K.kda_kvcache_attention_shared if shared else K.kda_kvcache_attention
        o = call(turned, *self.cache, self.tables, after, *([self.groups] if shared else []), cu_tokens=cu)
        lens, tables = self.lens.cpu().numpy(), self.tables.cpu().numpy()
        rows = self.rotary[np.concatenate([np.arange(a, a + n) for a, n in zip(lens, counts)])]
        want = [rotate(t.double().cpu().numpy(), rows, self.inter) for t in (q, k)] + [v.double().cpu().numpy()]
        assert (np.abs(turned.double().cpu().numpy() - want[0]) <= (2.0 ** -8 + 2.0 ** -21) * np.abs(want[0]) + 2.0 ** -25).all()
        now = [c.view(torch.uint8).cpu().numpy() if c.dtype == F8 else c.cpu().numpy() for c in self.cache]
        for i in range(2):
            check_quantised(want[1 + i], before[i], now[i], before[2 + i], now[2 + i], tables, lens, counts, self.page)
        want, weight = ref.attention(turned.double().cpu().numpy(), *now, tables, after.cpu().numpy(), counts, self.page, self.d ** -0.5)
        assert (np.abs(o.double().cpu().numpy() - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -10 * weight + 1e-6).all()
        self.lens = after
        return o

    def logits(self, o):
        return (o.reshape(o.shape[0], -1) @ self.head).float()

    def fork(self, parents):
        self.tables, self.refs = K.kda_pages_fork(self.tables, self.refs, parents, lens=self.lens, page_tokens=self.page, pools=self.cache)
        self.lens = self.lens[parents.long()]


@pytest.mark.parametrize("sizes", [dict(), dict(requests=3, beams=4, hq=6, hkv=1, d=128, page=64, rot=128, interleaved=True)])
def test_steps(sizes):
    run = Run(**sizes)
    rng, rows, beams = run.rng, run.rows, run.beams
    K.kda_get_device_status()
    prompts = [rng.integers(0, run.vocab, n) for n in (300, 411, 129)[: run.requests]]
    counts = [len(prompts[r // beams]) if r % beams == 0 else 0 for r in range(rows)]
    o = run.append(torch.as_tensor(np.concatenate(prompts)).cuda(), counts, shared=False)
    last = o[(cu_of([len(p) for p in prompts])[1:] - 1).long()]
    logits = torch.zeros(run.requests, beams, run.vocab, device="cuda")
    logits[:, 0] = run.logits(last)
    scores = torch.full((run.requests, beams), float("-inf"), device="cuda")
    scores[:, 0] = 0
    history = np.full((rows, 420), -1, np.int64)
    for r in range(rows):
        history[r, : len(prompts[r // beams])] = prompts[r // beams]
    prompt_lens = np.array([len(prompts[r // beams]) for r in range(rows)])
    lens = prompt_lens.copy()
    for step in range(4):
        mask = np.packbits((rng.random((rows, (run.vocab + 31) // 32 * 32)) < 0.9).astype(np.uint8), axis=1, bitorder="little").view(np.int32)
        rules = dict(history=history, lens=lens, prompt_lens=prompt_lens, repetition=np.full(rows, 1.2, np.float32),
                     presence=np.full(rows, 0.5, np.float32), frequency=np.full(rows, 0.25, np.float32),
                     bias_tokens=rng.integers(0, run.vocab, (rows, 7)), bias=rng.standard_normal((rows, 7)).astype(np.float32), mask=mask)
        raw = logits.cpu()
        K.kda_logits_penalize(logits, **{k: ints(a) if a.dtype == np.int64 else torch.as_tensor(a).cuda() for k, a in rules.items()}, out=logits)
        check_logits(logits, raw, rules, "fp32", adds=7)
        scores, tokens, parents = K.kda_beam_select(logits, scores)
        tokens, parents = tokens.view(rows), parents.view(rows)
        assert all(mask[p, t // 32] >> (t % 32) & 1 for p, t in zip(parents.tolist(), tokens.tolist()))
        run.fork(parents)
        history, lens = history[parents.cpu().numpy()], lens[parents.cpu().numpy()]
        history[np.arange(rows), lens] = tokens.cpu().numpy()
        lens = lens + 1
        logits = run.logits(run.append(tokens.long(), [1] * rows, shared=True)).view(run.requests, beams, run.vocab)
    assert K.kda_get_device_status() == 0
    assert int(run.lens.min()) == min(len(p) for p in prompts) + 4


def test_a_captured_step():
    # the same step from the same cache, eager and out of a graph that was captured before
    run = Run()
    rows = run.rows
    run.append(torch.arange(300, device="cuda"), [300] + [0] * (rows - 1), shared=False)
    run.fork(torch.zeros(rows, dtype=torch.int32, device="cuda"))
    after = run.lens + 1
    run.tables, run.refs = K.kda_pages_alloc(run.tables, run.refs, -(-after // run.page))
    rotary = torch.as_tensor(run.rotary).cuda()
    history = torch.randint(0, run.vocab, (rows, 300), dtype=torch.int32, device="cuda")
    repetition = torch.full((rows,), 1.5, device="cuda")
    scores = torch.zeros(run.requests, run.beams, device="cuda")
    tokens = torch.zeros(rows, dtype=torch.int64, device="cuda")

    def step():
        q, k, v = run.embed[tokens].split(run.split, 1)
        q = K.kda_kvcache_append_rotary(q, k, v, rotary, *run.cache, run.tables, run.lens)
        o = K.kda_kvcache_attention_shared(q, *run.cache, run.tables, after, run.groups)
        x = run.logits(o).view(run.requests, run.beams, -1)
        return (o, *K.kda_beam_select(K.kda_logits_penalize(x, history=history, repetition=repetition, out=x), scores))

    saved = [c.clone() for c in run.cache]

    def restore():
        for c, s in zip(run.cache, saved):
            c.copy_(s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        tokens.copy_(torch.randint(0, run.vocab, (rows,), generator=torch.Generator().manual_seed(seed)))
        restore()
        want, cache = step(), [c.clone() for c in run.cache]
        restore()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(run.cache, cache))
    assert K.kda_get_device_status() == 0


def test_example_with_rotation_and_penalties():
    import hybrid_beam_decode as ex
    answers, _ = ex.decode(requests=2, beams=3, steps=5, rotary=True, repetition=1.3)
    assert answers == ex.decode(requests=2, beams=3, steps=5, rotary=True, repetition=1.3)[0]
    assert [[len(t) for _, t in beams] for beams in answers] == [[5] * 3] * 2
