"""Beam decoding with a small random model that mixes KDA layers with full attention.

Shows the serving calls together, as a server uses them: the prompts go through the KDA prefill
and into the 8-bit key/value cache; every step then runs the recurrent KDA step on a pool of
states, appends to and attends over the paged cache (what the beams of a request share is gone
through once), selects beams, and reorders both kinds of pages by the selection; finished requests give their pages back and the pools are compacted.

    python examples/hybrid_beam_decode.py [--requests 3] [--beams 4] [--steps 12] [--rotary] [--repetition 1.2]

--rotary turns queries and keys of the attention by their positions as they are appended;
--repetition penalises the logits of tokens that a beam already has.

Needs a GB300 (there is no CPU path).  Weights are random: the tokens mean nothing, but
every run prints the same ones.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_kda_delta_gb300 as K  # noqa: E402

D = 128


class Model:
    """Layers 'kda' (recurrent) and 'full' (attention over a cache), vocabulary and sizes small."""

    def __init__(self, layers=("kda", "full", "kda"), width=256, heads=4, kv_heads=2, vocab=997, device="cuda"):
        g = torch.Generator(device=device).manual_seed(0)
        self.layers, self.heads, self.kv_heads, self.vocab, self.width = layers, heads, kv_heads, vocab, width

        def w(*shape):
            return (torch.randn(*shape, generator=g, device=device) / math.sqrt(shape[0])).to(torch.bfloat16)

        self.embed, self.head = w(vocab, width) * math.sqrt(vocab), w(width, vocab)
        self.weights = []
        for kind in layers:
            kv = heads if kind == "kda" else kv_heads
            self.weights.append(dict(qkv=w(width, (heads + 2 * kv) * D), out=w(heads * D, width), g=w(width, heads * D),
                                     beta=w(width, heads)))

    def logits(self, x):
        return (x @ self.head).float() * 2

    def project(self, i, x):
        """q, k, v of layer i for tokens [T, width]: views of one product."""
        kv = self.heads if self.layers[i] == "kda" else self.kv_heads
        y = torch.nn.functional.rms_norm(x, (self.width,)) @ self.weights[i]["qkv"]
        q, k, v = y.view(x.shape[0], -1, D).split([self.heads, kv, kv], 1)
        if self.layers[i] == "kda":
            unit = torch.nn.functional.normalize
            return unit(q.float(), dim=-1).to(q.dtype), unit(k.float(), dim=-1).to(k.dtype), v.contiguous()
        return q, k, v  # the cache takes strided tokens

    def gates(self, i, x):
        w = self.weights[i]
        g = torch.nn.functional.logsigmoid((x @ w["g"]).float() + 2).view(x.shape[0], self.heads, D)
        return g.contiguous(), torch.sigmoid(x @ w["beta"])

    def mix(self, i, x, o):
        return x + o.reshape(x.shape[0], -1) @ self.weights[i]["out"]


class Server:
    """The model with pools of states and of cache pages for rows = requests x beams."""

    def __init__(self, model, requests, beams, max_tokens, page=16, device="cuda", rotary=False):
        self.m, self.requests, self.beams, self.page = model, requests, beams, page
        angle = torch.arange(max_tokens, device=device)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device=device) / D)
        self.rotary = torch.cat([angle.cos(), angle.sin()], 1) if rotary else None
        self.groups = torch.arange(requests + 1, dtype=torch.int32, device=device) * beams
        rows = requests * beams
        kda, full = (sum(k == kind for k in model.layers) for kind in ("kda", "full"))
        width = -(-max_tokens // page)
        # one private state page a row; cache pages are shared by the beams of a request
        self.states = torch.zeros(kda, rows, model.heads, D, D, device=device)
        cache = (full, rows * width, model.kv_heads)
        self.codes = [torch.zeros(*cache, page, D, dtype=torch.float8_e4m3fn, device=device) for _ in range(2)]
        self.scales = [torch.zeros(*cache, device=device) for _ in range(2)]
        new = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)  # noqa: E731
        self.state_table, self.state_refs = new(rows, 1) - 1, new(rows)
        self.table, self.refs, self.lens = new(rows, width) - 1, new(rows * width), new(rows)

    def cache(self, layer):
        return (self.codes[0][layer], self.codes[1][layer], self.scales[0][layer], self.scales[1][layer])

    def layers(self):
        """(index, kind, index among its kind)"""
        seen = {"kda": 0, "full": 0}
        for i, kind in enumerate(self.m.layers):
            yield i, kind, seen[kind]
            seen[kind] += 1

    def append(self, q, k, v, layer, cu=None):
        """Appends k and v to a layer's cache; returns the queries to attend with."""
        if self.rotary is not None:
            return K.kda_kvcache_append_rotary(q, k, v, self.rotary, *self.cache(layer), self.table, self.lens, cu_tokens=cu)
        K.kda_kvcache_append(k, v, *self.cache(layer), self.table, self.lens, cu_tokens=cu)
        return q

    def prefill(self, prompts):
        """Runs the prompts as the first beam of each request; returns the last tokens' hidden."""
        dev, beams = self.table.device, self.beams
        n = [len(p) for p in prompts]
        first = torch.arange(self.requests, device=dev) * beams  # rows of the first beams
        want = torch.zeros_like(self.lens)
        want[first] = torch.tensor(n, dtype=torch.int32, device=dev)
        self.table, self.refs = K.kda_pages_alloc(self.table, self.refs, -(-want // self.page))
        self.state_table, self.state_refs = K.kda_pages_alloc(self.state_table, self.state_refs, (want > 0).int())
        # new tokens of every row: the first beams have the prompts, the others none
        cu = torch.zeros(self.requests * beams + 1, dtype=torch.int32, device=dev)
        cu[1:] = want.cumsum(0)
        cu_req = torch.zeros(self.requests + 1, dtype=torch.int32, device=dev)
        cu_req[1:] = torch.tensor(n, dtype=torch.int32, device=dev).cumsum(0)
        x = self.m.embed[torch.cat([torch.as_tensor(p, device=dev) for p in prompts])]
        at = self.state_table[first, 0].long()
        for i, kind, j in self.layers():
            q, k, v = self.m.project(i, x)
            if kind == "kda":
                g, beta = self.m.gates(i, x)
                o, final = K.kda_prefill(q, k, v, g, beta, cu_seqlens=cu_req, output_final_state=True)
                self.states[j][at] = final
            else:
                q = self.append(q, k, v, j, cu)
                o = K.kda_kvcache_attention(q, *self.cache(j), self.table, self.lens + want, cu_tokens=cu)
            x = self.m.mix(i, x, o)
        self.lens = self.lens + want
        return x[(cu_req[1:] - 1).long()]

    def step(self, tokens):
        """One token for every row (-1: an empty row); returns the hidden states [rows, width]."""
        active = tokens >= 0
        x = self.m.embed[tokens.clamp(min=0).long()]
        after = self.lens + active.int()
        self.table, self.refs = K.kda_pages_alloc(self.table, self.refs, -(-after // self.page))
        state_pages = torch.where(active, self.state_table[:, 0], -1)
        cu = torch.zeros(tokens.numel() + 1, dtype=torch.int32, device=x.device)
        cu[1:] = active.cumsum(0)
        all_live = bool(active.all())
        live = slice(None) if all_live else active.nonzero()[:, 0]
        for i, kind, j in self.layers():
            q, k, v = self.m.project(i, x)
            if kind == "kda":
                g, beta = self.m.gates(i, x)
                o = K.kda_decode_paged(q, k, v, g, beta, self.states[j], state_pages)
            elif all_live:
                q = self.append(q, k, v, j)
                o = K.kda_kvcache_attention_shared(q, *self.cache(j), self.table, after, self.groups)
            else:  # only the rows that have a token
                o = torch.zeros_like(q)
                o[live] = K.kda_kvcache_attention_shared(self.append(q[live], k[live], v[live], j, cu), *self.cache(j), self.table, after,
                                                         self.groups, cu_tokens=cu)
            x = self.m.mix(i, x, o)
        self.lens = after
        return x

    def reorder(self, parents):
        """Row r continues row parents[r]: states are copied, full cache pages shared."""
        self.state_table, self.state_refs = K.kda_pages_fork(self.state_table, self.state_refs, parents,
                                                             pools=[self.states], layers_first=True)
        self.table, self.refs = K.kda_pages_fork(self.table, self.refs, parents, lens=self.lens, page_tokens=self.page,
                                                 pools=self.codes + self.scales, layers_first=True)
        self.lens = torch.where(parents >= 0, self.lens[parents.clamp(min=0).long()], 0)

    def release(self, drop):
        """Gives the rows' pages back and moves the others to the front of the pools."""
        self.table, self.refs = K.kda_pages_free(self.table, self.refs, drop)
        self.state_table, self.state_refs = K.kda_pages_free(self.state_table, self.state_refs, drop)
        self.lens = torch.where(drop, 0, self.lens)
        self.table, self.refs, _, live = K.kda_pages_compact(self.table, self.refs, pools=self.codes + self.scales, layers_first=True)
        self.state_table, self.state_refs, _, states = K.kda_pages_compact(self.state_table, self.state_refs, pools=[self.states],
                                                                          layers_first=True)
        return live, states


def decode(requests=3, beams=4, steps=12, eos=1, seed=0, rotary=False, repetition=1.0):
    """Beam search over random prompts; returns [(score, tokens)] for each request, best first."""
    g = torch.Generator().manual_seed(seed)
    prompts = [torch.randint(2, 900, (int(n),), generator=g) for n in torch.randint(5, 60, (requests,), generator=g)]
    model = Model()
    server = Server(model, requests, beams, max_tokens=60 + steps + 1, rotary=rotary)
    rows = requests * beams
    hidden = server.prefill(prompts)
    # The first selection: one beam of each request is there, the others score -inf.
    logits = torch.zeros(requests, beams, model.vocab, device="cuda")
    logits[:, 0] = model.logits(hidden)
    scores = torch.full((requests, beams), -math.inf, device="cuda")
    scores[:, 0] = 0
    done = torch.zeros(requests, beams, dtype=torch.bool, device="cuda")
    history = torch.zeros(rows, 0, dtype=torch.int32, device="cuda")
    penalty = torch.full((rows,), repetition, device="cuda")
    for _ in range(steps):
        if repetition != 1.0 and history.shape[1] > 0:
            K.kda_logits_penalize(logits, history=history, repetition=penalty, out=logits)
        scores, tokens, parents, done = K.kda_beam_select(logits, scores, done=done, eos=eos)
        parents, tokens = parents.view(rows), tokens.view(rows)
        server.reorder(parents)
        history = torch.cat([history[parents.clamp(min=0).long()], tokens[:, None]], 1)
        hidden = server.step(torch.where(done.view(rows), -1, tokens))
        logits = model.logits(hidden).view(requests, beams, -1)
    # the first request is answered: its pages go back
    server.release(torch.arange(rows, device="cuda") < beams)
    status = K.kda_get_device_status()
    if status:
        raise RuntimeError(f"device status {K.kda_status_string(status)}")
    history, scores = history.view(requests, beams, -1).tolist(), scores.tolist()
    return [list(zip(scores[r], history[r])) for r in range(requests)], server


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--rotary", action="store_true")
    ap.add_argument("--repetition", type=float, default=1.0)
    a = ap.parse_args()
    answers, server = decode(a.requests, a.beams, a.steps, rotary=a.rotary, repetition=a.repetition)
    for r, beams in enumerate(answers):
        print(f"request {r}")
        for score, tokens in beams:
            print(f"  {score:9.4f}  {tokens}")
    print(f"pages in use after the first request's release: {int((server.refs > 0).sum())} of {server.refs.numel()} (cache), "
          f"{int((server.state_refs > 0).sum())} of {server.state_refs.numel()} (states)")


if __name__ == "__main__":
    main()
