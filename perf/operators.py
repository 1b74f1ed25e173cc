"""Measured cases of the serving operators around the state cache: the 8-bit paged key/value cache
(append, attention), beam selection and the page operations (fork, compact).

``run`` computes a case with elementary torch operations in 32 bits (``own`` false) or with the calls a
user of this package makes (``own`` true); ``exact`` gives the computed numbers in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0


def listed():
    return [
        # one user's next token over a short context: latency
        dict(name="attend_one_row", kind="attend", rows=1, new=1, hq=8, hkv=1, d=128, ctx=1000, page=16, dtype="bf16"),
        # a serving batch's next token: ragged contexts up to the longest
        dict(name="attend_ragged", kind="attend", rows=64, new=1, hq=64, hkv=8, d=128, ctx=8192, page=64, dtype="bf16"),
        # few rows over very long contexts: the work has to be split along the keys
        dict(name="attend_long", kind="attend", rows=4, new=1, hq=32, hkv=4, d=128, ctx=131072, page=128, dtype="bf16"),
        # pieces of prompts that continue cached contexts
        dict(name="attend_block", kind="attend", rows=8, new=512, hq=16, hkv=4, d=64, ctx=4096, page=64, dtype="fp16"),
        # the step's one new token of each row goes into the cache
        dict(name="append_step", kind="append", rows=256, new=1, hkv=8, d=128, ctx=2048, page=64, dtype="bf16"),
        # prompts of odd lengths go into the cache
        dict(name="append_prompt", kind="append", rows=5, new=8191, hkv=8, d=128, ctx=100, page=64, dtype="bf16"),
        # one request's beams over an odd vocabulary: latency
        dict(name="beam_one", kind="beam", batch=1, beams=4, vocab=32001, dtype="fp32"),
        # a batch of requests over a large vocabulary
        dict(name="beam_batch", kind="beam", batch=32, beams=8, vocab=131072, dtype="bf16"),
        # a beam step's reordering of recurrent states: one private page a row, two layers of 64 heads
        dict(name="fork_states", kind="fork", groups=8, beams=8, alive=5, prompt=0, page=0, heads=64, layers=2),
        # a beam step's reordering of cache rows: prompt pages shared, the open page copied
        dict(name="fork_cache", kind="fork", groups=16, beams=8, alive=5, prompt=127, page=64, heads=8, layers=2),
        # a small pool of states shrinks after requests ended
        dict(name="compact_states", kind="compact", pages=96, live=40, width=1, heads=4, page=0, layers=1),
        # a large cache pool shrinks
        dict(name="compact_cache", kind="compact", pages=9001, live=5000, width=64, heads=4, page=64, layers=1),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "append", "beam", "fork", "compact"])
    if kind == "attend":
        d, page, hkv = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        rows, ctx = _log_int(rng, 1, 128), _log_int(rng, 1, 131072)
        new = 1 if rng.random() < 0.6 else _log_int(rng, 2, 512)
        while rows > 1 and rows * (ctx + new) * hkv * d > 128 << 20:
            rows = (rows + 1) // 2
        while new > 1 and rows * new * group * hkv * (ctx + new) > 1 << 28:
            new = (new + 1) // 2
        return dict(kind=kind, rows=rows, new=new, hq=hkv * group, hkv=hkv, d=d, ctx=ctx, page=page, dtype=rng.choice(["bf16", "fp16"]))
    if kind == "append":
        rows = _log_int(rng, 1, 256)
        new = 1 if rng.random() < 0.5 else _log_int(rng, 2, max(2, 30000 // rows))
        return dict(kind=kind, rows=rows, new=new, hkv=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 128]), ctx=_log_int(rng, 1, 2048),
                    page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "fp16"]))
    if kind == "beam":
        beams, vocab = rng.choice([1, 2, 3, 4, 5, 8, 10, 16]), _log_int(rng, 500, 200000)
        batch = min(_log_int(rng, 1, 64), max(1, (32 << 20) // (beams * vocab)))
        return dict(kind=kind, batch=batch, beams=beams, vocab=vocab, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if kind == "fork":
        beams = rng.choice([2, 3, 4, 5, 8])
        c = dict(kind=kind, groups=_log_int(rng, 1, 16), beams=beams, alive=rng.randint(1, beams), layers=rng.randint(1, 2))
        if rng.random() < 0.5:
            return dict(c, groups=min(c["groups"], 64 // beams), prompt=0, page=0, heads=_log_int(rng, 1, 32))
        return dict(c, prompt=_log_int(rng, 1, 120), page=rng.choice([16, 32, 64]), heads=rng.choice([1, 2, 3, 4, 8]))
    pages, state = _log_int(rng, 8, 9000), rng.random() < 0.4
    if state:
        return dict(kind=kind, pages=min(pages, 400), live=rng.randint(1, min(pages, 400)), width=1, heads=_log_int(rng, 1, 16), page=0, layers=1)
    return dict(kind=kind, pages=pages, live=rng.randint(1, pages), width=_log_int(rng, 1, 64), heads=rng.choice([1, 2, 3, 4]),
                page=rng.choice([16, 32, 64]), layers=1)


def _spread(n, low, high):
    """n whole numbers over [low, high], the longest among them: the same set for every seed."""
    if n == 1:
        return [high]
    return [int(round(low + (high - low) * i / (n - 1))) for i in range(n)]


def _old_lengths(case):
    return _spread(case["rows"], max(0, case["ctx"] // 3), case["ctx"])


def _new_lengths(case):
    return [1] * case["rows"] if case["new"] == 1 else _spread(case["rows"], (case["new"] + 1) // 2, case["new"])


class _Draws:
    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(int(seed))

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen, device="cuda")

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.gen, device="cuda")

    def order(self, n):
        return torch.randperm(n, generator=self.gen, device="cuda")

    def bytes(self, *shape):
        return torch.randint(0, 256, shape, generator=self.gen, device="cuda", dtype=torch.uint8)


def _ints(x):
    return torch.as_tensor(x, device="cuda").to(torch.int32)


def _page_tables(rnd, lengths, page):
    """A table of pages for rows of these lengths, from a pool in random order."""
    need = (torch.as_tensor(lengths, device="cuda").to(torch.int64) + page - 1) // page
    width, total = int(need.max()), int(need.sum())
    pool = rnd.order(total + 3)
    at = torch.arange(max(width, 1), device="cuda")
    place = (need.cumsum(0) - need)[:, None] + at
    tables = torch.where(at < need[:, None], pool[place.clamp(max=total + 2)], -1)
    return tables.to(torch.int32), total + 3


def _cache(rnd, pages, hkv, page, d):
    """Codes as an append leaves them (the largest of each block is 448) and their scales."""
    x = rnd.normal(pages, hkv, page, d)
    scale = x.abs().amax((2, 3)) / F8_MAX
    codes = (x / scale[:, :, None, None]).clamp(-F8_MAX, F8_MAX).to(F8)
    return codes, scale * (0.5 + rnd.uniform(pages, hkv))


def prepare(case, seed):
    rnd, kind = _Draws(seed), case["kind"]
    s = dict(case=case)
    if kind in ("attend", "append"):
        order = rnd.order(case["rows"]).tolist()
        old, new = _old_lengths(case), _new_lengths(case)
        old, new = [old[i] for i in order], [new[-1 - i] for i in order]  # the longest contexts get the shortest pieces
        s["tables"], pages = _page_tables(rnd, [a + b for a, b in zip(old, new)], case["page"])
        s["k_codes"], s["k_scale"] = _cache(rnd, pages, case["hkv"], case["page"], case["d"])
        s["v_codes"], s["v_scale"] = _cache(rnd, pages, case["hkv"], case["page"], case["d"])
        ends = [0]
        for n in new:
            ends.append(ends[-1] + n)
        s["cu"], s["new"] = _ints(ends), new
        dt = DTYPES[case["dtype"]]
        if kind == "attend":
            s["lens"] = _ints([a + b for a, b in zip(old, new)])
            s["q"] = (rnd.normal(ends[-1], case["hq"], case["d"]) * 1.5).to(dt)
        else:
            s["lens"] = _ints(old)
            s["k"], s["v"] = (rnd.normal(ends[-1], case["hkv"], case["d"]).to(dt) for _ in range(2))
    elif kind == "beam":
        b, w, v = case["batch"], case["beams"], case["vocab"]
        x = rnd.normal(b, w, v) * 3 + 2 * rnd.uniform(v).log()  # most tokens are rare
        x[:, :, rnd.order(v)[: v // 50]] = -math.inf  # tokens that a rule forbids
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["scores"] = -(rnd.uniform(b, w) * 6).cumsum(1)
        s["done"] = rnd.uniform(b, w) < 0.1
    elif kind == "fork":
        groups, beams, prompt = case["groups"], case["beams"], case["prompt"]
        rows = groups * beams
        pages = rows + groups * prompt + rows  # a row's own page each, the shared prompts, as many free ones
        ids = rnd.order(pages)
        shared = ids[rows: rows + groups * prompt].view(groups, 1, prompt).expand(groups, beams, prompt)
        tables = torch.cat([shared, ids[:rows].view(groups, beams, 1)], 2).reshape(rows, prompt + 1)
        s["tables"] = tables.to(torch.int32).contiguous()
        s["refs"] = torch.bincount(tables.flatten(), minlength=pages).to(torch.int32)
        # `alive` of each group's beams go on, each at least once
        live = torch.argsort(rnd.uniform(groups, beams), 1)[:, : case["alive"]]
        extra = (rnd.uniform(groups, beams - case["alive"]) * case["alive"]).long().clamp(max=case["alive"] - 1)
        parents = torch.cat([live, live.gather(1, extra)], 1)
        parents = parents.gather(1, torch.argsort(rnd.uniform(groups, beams), 1))
        s["parents"] = (parents + beams * torch.arange(groups, device="cuda")[:, None]).flatten().to(torch.int32)
        s["lens"] = torch.full((rows,), prompt * case["page"] + max(1, case["page"] // 2), device="cuda", dtype=torch.int32)
        s["pools"] = _pools(rnd, case, pages)
    else:
        pages, live, width = case["pages"], case["live"], case["width"]
        moved = live * (pages - live) // pages
        low, high = rnd.order(live)[: live - moved], live + rnd.order(pages - live)[:moved]
        ids = torch.cat([low, high])[rnd.order(live)]
        rows = -(-live // width)
        tables = torch.full((rows * width,), -1, device="cuda", dtype=torch.int32)
        tables[:live] = ids.to(torch.int32)
        s["tables"] = tables.view(rows, width)
        s["refs"] = torch.bincount(ids, minlength=pages).to(torch.int32)
        s["pools"] = _pools(rnd, case, pages)
    return s


def _pools(rnd, case, pages):
    """Recurrent states in 32 bits (page 0), or the four tensors of an 8-bit cache."""
    n, h = case["layers"], case["heads"]
    if case["page"] == 0:
        return [rnd.normal(n, pages, h, 128, 128)]
    return [rnd.bytes(n, pages, h, case["page"], 128), rnd.bytes(n, pages, h, case["page"], 128), rnd.uniform(n, pages, h), rnd.uniform(n, pages, h)]


def _page_bytes(case):
    return case["layers"] * case["heads"] * (128 * 128 * 4 if case["page"] == 0 else 2 * (case["page"] * 128 + 4))


def work(case):
    kind = case["kind"]
    if kind == "attend":
        old, new = _old_lengths(case), _new_lengths(case)[::-1]
        total = sum(a + b for a, b in zip(old, new))
        seen = sum(n * a + n * (n + 1) // 2 for a, n in zip(old, new))
        return dict(bytes=2 * total * case["hkv"] * case["d"] + 2 * 2 * sum(new) * case["hq"] * case["d"] + (total // case["page"]) * (8 * case["hkv"] + 4),
                    flops=4 * seen * case["hq"] * case["d"])
    if kind == "append":
        values = 2 * sum(_new_lengths(case)) * case["hkv"] * case["d"]
        return dict(bytes=3 * values, flops=2 * values)
    if kind == "beam":
        n = case["batch"] * case["beams"] * case["vocab"]
        return dict(bytes=n * (4 if case["dtype"] == "fp32" else 2), flops=3 * n)
    if kind == "fork":
        rows = case["groups"] * case["beams"]
        copied = case["groups"] * (case["beams"] - case["alive"])
        return dict(bytes=2 * copied * _page_bytes(case) + 8 * rows * (case["prompt"] + 1) + 8 * (2 * rows + case["groups"] * case["prompt"]), flops=0)
    moved = case["live"] * (case["pages"] - case["live"]) // case["pages"]
    return dict(bytes=2 * moved * _page_bytes(case) + 8 * case["live"] + 12 * case["pages"], flops=0)


# ---- plain forms -------------------------------------------------------------------------------------------


def _rows_of_tokens(cu, tokens):
    return torch.searchsorted(cu[1:].contiguous(), torch.arange(tokens, device=cu.device, dtype=cu.dtype), right=True)


def _plain_attend(s):
    q, tables, lens, cu = s["q"], s["tables"].long(), s["lens"].long(), s["cu"]
    codes_k, codes_v = s["k_codes"], s["v_codes"]
    tokens, hq, d = q.shape
    rows, width = tables.shape
    _, hkv, page, _ = codes_k.shape
    group, most = hq // hkv, max(s["new"])
    row = _rows_of_tokens(cu, tokens)
    place = torch.arange(tokens, device=q.device) - cu.long()[row]
    padded = q.new_zeros(rows, most, hq, d, dtype=torch.float32)
    padded[row, place] = q.float()
    at = tables.clamp(min=0)

    def gathered(codes, scale):
        x = codes.view(torch.uint8)[at].view(F8).float() * scale[at][..., None, None]  # [R, M, Hkv, page, D]
        return x.permute(0, 2, 1, 3, 4).reshape(rows, hkv, width * page, d)

    key = torch.arange(width * page, device=q.device)
    there = (key < lens[:, None]) & (tables >= 0).repeat_interleave(page, 1)
    count = (cu[1:] - cu[:-1]).long()
    sees = key <= (lens - count)[:, None, None] + torch.arange(most, device=q.device)[None, :, None]  # [R, n, L]
    sees = (sees & there[:, None]).repeat_interleave(group, 1)  # [R, n * group, L]
    x = padded.view(rows, most, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(rows, hkv, most * group, d)
    score = x @ gathered(codes_k, s["k_scale"]).transpose(2, 3) * d ** -0.5
    score = score.masked_fill(~sees[:, None], -math.inf)
    top = score.amax(3, keepdim=True)
    p = (score - top.masked_fill(top == -math.inf, 0)).exp()
    v = gathered(codes_v, s["v_scale"]).masked_fill(~there[:, None, :, None], 0)
    out = (p @ v) / p.sum(3, keepdim=True).clamp(min=1e-30)
    return out.view(rows, hkv, most, group, d)[row, :, place].reshape(tokens, hq, d).to(q.dtype)


def _plain_quantise(x, codes, scale, tables, lens, cu):
    pages, _, page, _ = codes.shape
    row = _rows_of_tokens(cu, x.shape[0])
    at = lens.long()[row] + torch.arange(x.shape[0], device=x.device) - cu.long()[row]
    where, inside = tables.long()[row, at // page], at % page
    x = x.float()
    largest = torch.zeros_like(scale).index_reduce_(0, where, x.abs().amax(2), "amax")
    fresh = torch.zeros(pages, device=x.device, dtype=torch.bool)
    fresh[where[inside == 0]] = True
    touched = torch.zeros_like(fresh)
    touched[where] = True
    wanted = largest / torch.full((), F8_MAX, device=x.device)
    grown = torch.where(fresh[:, None], wanted, torch.maximum(scale, wanted))
    grown = torch.where(touched[:, None], grown, scale)
    bits = codes.view(torch.uint8)
    # the open page of each row: its older tokens go by the grown scale
    opened = ((lens % page != 0) & (cu[1:] > cu[:-1])).nonzero()[:, 0]
    which = tables.long()[opened, lens.long()[opened] // page]
    old, was, now = codes.view(torch.uint8)[which].view(F8).float(), scale[which][..., None, None], grown[which][..., None, None]
    again = (old * was / now).clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)
    keep = (was == now) | (torch.arange(page, device=x.device) >= (lens % page)[opened, None])[:, None, :, None]
    bits[which] = torch.where(keep, bits[which], again)
    by = grown[where][..., None]
    bits[where, :, inside] = torch.where(by > 0, x / by, 0).clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)
    scale.copy_(grown)


def _plain_beam(s):
    x, scores, done = s["logits"].float(), s["scores"], s["done"]
    batch, beams, vocab = x.shape
    usable = torch.isfinite(x)
    x = x.masked_fill(~usable, -math.inf)
    top = x.amax(2, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0)
    lse = top + (x - top).exp().sum(2, keepdim=True).log()
    total = (scores[..., None] + (x - lse)).masked_fill(~usable, -math.inf)
    total = total.masked_fill(done[..., None], -math.inf)
    total[..., 1] = torch.where(done, scores, total[..., 1])
    total = (total.masked_fill(torch.isnan(total), -math.inf) + 0.0).view(batch, beams * vocab)
    bits = total.view(torch.int32).long()
    rank = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)  # whole numbers in the order of the totals
    rank = (rank << 32) + (0xFFFFFFFF - torch.arange(beams * vocab, device=x.device))  # the lowest index first
    flat = torch.topk(rank, beams, 1).indices
    best = total.gather(1, flat)
    none = best == -math.inf
    token = (flat % vocab).masked_fill(none, -1)
    parent = (flat // vocab + beams * torch.arange(batch, device=x.device)[:, None]).masked_fill(none, -1)
    ended = none | (token == 1) | done.flatten()[parent.clamp(min=0)]
    return best, token.to(torch.int32), parent.to(torch.int32), ended


def _counts(pages, mask, ids):
    found = torch.zeros(pages + 1, device=ids.device, dtype=torch.int64)
    return found.scatter_add_(0, torch.where(mask, ids, pages).flatten(), torch.ones_like(ids).flatten())[:pages]


def _plain_fork(s):
    tables, refs, parents = s["tables"].long(), s["refs"].long(), s["parents"].long()
    rows, width = tables.shape
    pages, page = refs.numel(), s["case"]["page"]
    source = tables[parents.clamp(min=0)].masked_fill((parents < 0)[:, None], -1)
    full = s["lens"].long()[parents.clamp(min=0)] // page if page else torch.zeros_like(parents)
    shared = (torch.arange(width, device=tables.device) < full[:, None]) & (source >= 0)
    private = ~shared & (source >= 0)
    held = refs - _counts(pages, tables >= 0, tables) + _counts(pages, shared, source)
    order = torch.arange(rows * width, device=tables.device).view(rows, width)
    first = torch.full((pages + 1,), rows * width, device=tables.device)
    first.scatter_reduce_(0, torch.where(private, source, pages).flatten(), order.flatten(), "amin")
    taken = private & (held[source.clamp(min=0)] == 0) & (first[source.clamp(min=0)] == order)
    held = held + _counts(pages, taken, source)
    need = private & ~taken
    free = torch.sort(held != 0, stable=True).indices
    rank = need.flatten().cumsum(0).view(rows, width) - 1
    page_of = torch.where(rank < (held == 0).sum(), free[rank.clamp(0, pages - 1)], -1)
    new = torch.where(need, page_of, torch.where(shared | taken, source, -1))
    copied = need & (page_of >= 0)
    for pool in s["pools"]:
        pool[:, page_of[copied]] = pool[:, source[copied]]
    return new.to(torch.int32), (held + _counts(pages, copied, page_of)).to(torch.int32)


def _plain_compact(s):
    tables, refs = s["tables"].long(), s["refs"]
    pages, live = refs.numel(), refs > 0
    count = live.sum()
    ids = torch.arange(pages, device=refs.device)
    holes = ids[~live & (ids < count)]
    above = ids[live & (ids >= count)]
    moved = torch.where(live, ids, -1)
    moved[above] = holes
    for pool in s["pools"]:
        pool[:, holes] = pool[:, above]
    new_refs = torch.zeros_like(refs)
    new_refs[moved[live]] = refs[live]
    new = torch.where(tables >= 0, moved[tables.clamp(min=0)], -1)
    return new.to(torch.int32), new_refs, moved.to(torch.int32), count.view(1).to(torch.int32)


def run(s):
    kind = s["case"]["kind"]
    if own:
        return _run_own(s, kind)
    if kind == "attend":
        return _plain_attend(s)
    if kind == "append":
        for x in ("k", "v"):
            _plain_quantise(s[x], s[x + "_codes"], s[x + "_scale"], s["tables"], s["lens"], s["cu"])
        return s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"]
    if kind == "beam":
        return _plain_beam(s)
    if kind == "fork":
        return _plain_fork(s), s["pools"]
    return _plain_compact(s), s["pools"]


def _run_own(s, kind):
    import chunked_kda_delta_gb300 as K

    cache = [s.get(x) for x in ("k_codes", "v_codes", "k_scale", "v_scale")]
    one = "cu" in s and s["case"]["new"] == 1
    if kind == "attend":
        return K.kda_kvcache_attention(s["q"], *cache, s["tables"], s["lens"], cu_tokens=None if one else s["cu"])
    if kind == "append":
        K.kda_kvcache_append(s["k"], s["v"], *cache, s["tables"], s["lens"], cu_tokens=None if one else s["cu"])
        return s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"]
    if kind == "beam":
        return K.kda_beam_select(s["logits"], s["scores"], done=s["done"], eos=1)
    if kind == "fork":
        new = K.kda_pages_fork(s["tables"], s["refs"], s["parents"], lens=s["lens"], page_tokens=s["case"]["page"], pools=s["pools"], layers_first=True)
        return new, s["pools"]
    return K.kda_pages_compact(s["tables"], s["refs"], pools=s["pools"], layers_first=True), s["pools"]


# ---- in 64 bits --------------------------------------------------------------------------------------------


def _e4m3_values():
    """The finite non-negative values of the type, in order: the code is the index."""
    v = [m / 8 * 2.0 ** -6 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], device="cuda", dtype=torch.float64)


def _nearest_e4m3(x):
    v = _e4m3_values()
    a = x.abs().clamp(max=F8_MAX)
    up = torch.searchsorted(v, a.contiguous()).clamp(max=126)
    down = (up - 1).clamp(min=0)
    low, high = a - v[down], v[up] - a
    pick = torch.where(low < high, down, torch.where(high < low, up, torch.where(down % 2 == 0, down, up)))
    return v[pick] * x.sign()


def exact(case, seed):
    if case["kind"] in ("fork", "compact"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    if case["kind"] == "attend":
        outs, page, group = [], case["page"], case["hq"] // case["hkv"]
        for r, n in enumerate(s["new"]):
            length, begin = int(s["lens"][r]), int(s["cu"][r])
            ids = s["tables"][r, : -(-length // page)].long()
            sides = []
            for x in ("k", "v"):
                c = s[x + "_codes"].view(torch.uint8)[ids].view(F8).to(torch.float64) * s[x + "_scale"][ids].double()[..., None, None]
                sides.append(c.transpose(0, 1).reshape(case["hkv"], -1, case["d"])[:, :length])
            q = s["q"][begin: begin + n].double()
            hidden = torch.arange(length, device="cuda") > (length - n + torch.arange(n, device="cuda"))[:, None]
            heads = []
            for h in range(case["hq"]):
                z = (q[:, h] @ sides[0][h // group].T / math.sqrt(case["d"])).masked_fill(hidden, -math.inf)
                heads.append(torch.softmax(z, 1) @ sides[1][h // group])
            outs.append(torch.stack(heads, 1))
        return torch.cat(outs)
    if case["kind"] == "append":
        got = []
        for x in ("k", "v"):
            codes, scale = s[x + "_codes"].to(torch.float64), s[x + "_scale"].double()
            for r, n in enumerate(s["new"]):
                begin, old = int(s["cu"][r]), int(s["lens"][r])
                new = s[x][begin: begin + n].double()
                for first in range(old - old % case["page"], old + n, case["page"]):
                    a, b = max(first, old), min(first + case["page"], old + n)
                    p, part = int(s["tables"][r, first // case["page"]]), new[a - old: b - old].transpose(0, 1)
                    now = (part.abs().amax((1, 2)) / F8_MAX).float().double()  # the scale is held in 32 bits
                    if a > first:
                        now = torch.maximum(now, scale[p])
                        by = torch.where(now > scale[p], scale[p] / now, 1.0)
                        codes[p, :, : a - first] = _nearest_e4m3(codes[p, :, : a - first] * by[:, None, None])
                    scale[p] = now
                    codes[p, :, a - first: b - first] = _nearest_e4m3(part / now[:, None, None])
            got += [codes, scale]
        return tuple(got)
    b, w, v = s["logits"].shape
    x = s["logits"].double()
    total = s["scores"].double()[..., None] + torch.log_softmax(x, 2)
    for i, j in s["done"].nonzero().tolist():
        total[i, j] = -math.inf
        total[i, j, 1] = s["scores"][i, j].double()
    return torch.sort(total.view(b, w * v), 1, descending=True).values[:, :w].contiguous(), None, None, None
