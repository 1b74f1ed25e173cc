"""The hybrid beam-decoding example: the paged, reordered, quantised path against the same model
run from scratch on whole sequences."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def scratch_scores(model, prompt, tokens, eos):
    """Log-probability of `tokens` after `prompt`: every layer over the whole sequence at once, with
    the full-attention layers in plain 32-bit torch on unquantised keys and values."""
    import chunked_kda_delta_gb300 as K
    seq = torch.cat([prompt.cuda(), torch.tensor(tokens, device="cuda")])
    x = model.embed[seq]
    for i, kind in enumerate(model.layers):
        q, k, v = model.project(i, x)
        if kind == "kda":
            g, beta = model.gates(i, x)
            o, _ = K.kda_prefill(q, k, v, g, beta)
        else:
            r = model.heads // model.kv_heads
            kk, vv = (t.float().repeat_interleave(r, 1) for t in (k, v))
            s = torch.einsum("thd,shd->hts", q.float(), kk) * 128 ** -0.5
            s = s.masked_fill(torch.ones_like(s[0]).triu(1).bool(), float("-inf"))
            o = torch.einsum("hts,shd->thd", torch.softmax(s, -1), vv).to(x.dtype)
        x = model.mix(i, x, o)
    lp = torch.log_softmax(model.logits(x), -1)
    total = 0.0
    for j, t in enumerate(tokens):
        total += lp[len(prompt) - 1 + j, t].item()
        if t == eos:
            break
    return total


def test_scores_match_a_run_from_scratch():
    # e4m3 keys and values carry a relative error of 2^-4 at most (2^-5 on average over a value's
    # range), averaged over heads and channels; bf16 activations 2^-9 a layer.  Scores are sums of
    # up to 8 log-probabilities of logits of size about 10: 0.1 a token is allowed.
    import hybrid_beam_decode as ex
    steps = 8
    answers, server = ex.decode(requests=3, beams=4, steps=steps)
    g = torch.Generator().manual_seed(0)
    prompts = [torch.randint(2, 900, (int(n),), generator=g) for n in torch.randint(5, 60, (3,), generator=g)]
    for prompt, beams in zip(prompts, answers):
        assert [s for s, _ in beams] == sorted((s for s, _ in beams), reverse=True)
        assert len({tuple(t) for _, t in beams}) == len(beams)
        for score, tokens in beams:
            assert len(tokens) == steps
            assert abs(score - scratch_scores(server.m, prompt, tokens, 1)) < 0.1 * steps
    # after the release: one state page for each remaining row, at the front
    assert (server.state_refs[:8] == 1).all() and (server.state_refs[8:] == 0).all()
    live = int((server.refs > 0).sum())
    assert (server.refs[:live] > 0).all() and (server.table[:4] == -1).all()


def test_runs_are_the_same():
    import hybrid_beam_decode as ex
    assert ex.decode(requests=2, beams=3, steps=5)[0] == ex.decode(requests=2, beams=3, steps=5)[0]
