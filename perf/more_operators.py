"""Measured cases of a decoding step's operators beside the 8-bit paged key/value cache and beam selection: the
cache append that rotates positions on the way, attention of rows that share a long prefix, and penalties, biases
and grammar masks on logits.

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
        # one user's next token: latency
        dict(name="rotary_one_row", kind="rotary", rows=1, new=1, hq=8, hkv=1, d=128, rot=128, inter=False, ctx=1000, page=16, dtype="bf16"),
        # a serving batch's next token, contexts of all lengths
        dict(name="rotary_step", kind="rotary", rows=256, new=1, hq=64, hkv=8, d=128, rot=128, inter=False, ctx=2048, page=64, dtype="bf16"),
        # prompts of odd lengths that continue short contexts
        dict(name="rotary_prompt", kind="rotary", rows=5, new=8191, hq=32, hkv=8, d=128, rot=128, inter=False, ctx=100, page=64, dtype="bf16"),
        # a model that rotates half of each head in neighbouring pairs, far positions
        dict(name="rotary_pairs", kind="rotary", rows=3, new=2001, hq=12, hkv=4, d=64, rot=32, inter=True, ctx=100000, page=32, dtype="fp16"),
        # one request's beams over its prompt: latency
        dict(name="shared_one_request", kind="shared", groups=1, beams=4, new=1, hq=32, hkv=8, d=128, prompt=2000, mine=40, page=16, dtype="bf16"),
        # beams of a batch of requests over long prompts of different lengths
        dict(name="shared_beams", kind="shared", groups=8, beams=8, new=1, hq=64, hkv=8, d=128, prompt=16384, mine=300, page=64, dtype="bf16"),
        # many users of one long system prompt, each with a conversation of its own
        dict(name="shared_system", kind="shared", groups=1, beams=64, new=1, hq=64, hkv=8, d=128, prompt=32768, mine=1000, page=64, dtype="bf16"),
        # several proposed tokens a row to be looked at together
        dict(name="shared_proposed", kind="shared", groups=5, beams=7, new=6, hq=16, hkv=2, d=64, prompt=10007, mine=129, page=32, dtype="fp16"),
        # one row's penalties and bias: latency
        dict(name="logits_one_row", kind="logits", batch=1, beams=1, vocab=32001, hist=500, bias=30, mask=0.0, penal=True, place=False, dtype="fp32"),
        # a batch of beams: everything at once over a large vocabulary
        dict(name="logits_batch", kind="logits", batch=32, beams=8, vocab=131072, hist=2000, bias=100, mask=0.05, penal=True, place=False, dtype="bf16"),
        # long histories, an odd vocabulary
        dict(name="logits_long", kind="logits", batch=16, beams=1, vocab=50257, hist=32768, bias=0, mask=0.0, penal=True, place=False, dtype="fp32"),
        # a grammar alone, in place: few tokens may follow
        dict(name="logits_grammar", kind="logits", batch=64, beams=1, vocab=151936, hist=0, bias=0, mask=0.02, penal=False, place=True, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rotary", "shared", "logits"])
    d, page, hkv = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "rotary":
        rows = _log_int(rng, 1, 256)
        new = 1 if rng.random() < 0.5 else _log_int(rng, 2, max(2, 30000 // rows))
        while new > 1 and rows * new * (hq + 2 * hkv) * d > 120 << 20:
            new = (new + 1) // 2
        ctx = _log_int(rng, 1, 131072)
        while rows > 1 and ctx > 1 and rows * ctx * hkv * d > 512 << 20:
            ctx = (ctx + 1) // 2
        rot = rng.choice([d, d, d // 2, d // 4 * 3, 16])
        return dict(kind=kind, rows=rows, new=new, hq=hq, hkv=hkv, d=d, rot=rot, inter=rng.random() < 0.4, ctx=ctx, page=page, dtype=dtype)
    if kind == "shared":
        groups, beams = _log_int(rng, 1, 16), _log_int(rng, 2, 64)
        prompt, mine = _log_int(rng, 1, 65536), _log_int(rng, 1, 2000)
        new = 1 if rng.random() < 0.6 else rng.randint(2, 16)
        while groups > 1 and groups * beams > 256:
            groups = (groups + 1) // 2
        while prompt > 1 and groups * beams * new * (prompt + mine) * hq * d > 16 << 30:
            prompt = (prompt + 1) // 2
        while prompt > 1 and groups * beams * (prompt + mine) * hkv * d > 2 << 30:
            prompt = (prompt + 1) // 2
        return dict(kind=kind, groups=groups, beams=beams, new=new, hq=hq, hkv=hkv, d=d, prompt=prompt, mine=max(mine, new), page=page, dtype=dtype)
    beams, vocab = rng.choice([1, 2, 3, 4, 5, 8, 10, 16]), _log_int(rng, 500, 200000)
    batch = min(_log_int(rng, 1, 64), max(1, (32 << 20) // (beams * vocab)))
    mask, dtype = rng.choice([0.0, 0.0, 0.02, 0.5, 0.98]), rng.choice(["bf16", "fp16", "fp32"])
    if mask > 0 and rng.random() < 0.3:
        return dict(kind=kind, batch=batch, beams=beams, vocab=vocab, hist=0, bias=0, mask=mask, penal=False, place=True, dtype=dtype)
    hist = _log_int(rng, 1, max(1, min(32768, (4 << 20) // (batch * beams))))
    return dict(kind=kind, batch=batch, beams=beams, vocab=vocab, hist=hist, bias=rng.choice([0, 1, 7, 64, 300]), mask=mask, penal=True, place=False, dtype=dtype)


def _spread(n, low, high):
    """n whole numbers over [low, high], the longest among them: the same set for every seed."""
    if n == 1:
        return [high]
    return [int(round(low + (high - low) * i / (n - 1))) for i in range(n)]


def _old_lengths(case):
    return _spread(case["rows"], max(0, case["ctx"] // 3), case["ctx"])


def _new_lengths(case):
    return [1] * case["rows"] if case["new"] == 1 else _spread(case["rows"], (case["new"] + 1) // 2, case["new"])


def _prompt_lengths(case):
    return _spread(case["groups"], max(1, case["prompt"] // 2), case["prompt"])


def _own_lengths(case):
    """Tokens of a group's rows behind its prompt, the new ones among them."""
    return _spread(case["beams"], max(case["new"], case["mine"] // 3), case["mine"])


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


def _ints(x):
    return torch.as_tensor(x, device="cuda").to(torch.int32)


def _place_pages(rnd, need, spare=3):
    """Pages from a pool in random order for rows that need so many: (ids [rows, widest], pages in the pool)."""
    need = torch.as_tensor(need, device="cuda").to(torch.int64)
    total = int(need.sum()) + spare
    pool, at = rnd.order(total), torch.arange(max(1, int(need.max())), device="cuda")
    place = (need.cumsum(0) - need)[:, None] + at
    return torch.where(at < need[:, None], pool[place.clamp(max=total - 1)], -1), total


def _cache(rnd, pages, hkv, page, d):
    """Codes as an append leaves them (the largest of each block is 448) and their scales."""
    x = rnd.normal(pages, hkv, page, d)
    scale = x.abs().amax((2, 3)) / F8_MAX
    codes = (x / scale[:, :, None, None]).clamp(-F8_MAX, F8_MAX).to(F8)
    return codes, scale * (0.5 + rnd.uniform(pages, hkv))


def _rotary_table(positions, rot):
    """Cosines, then sines, of every position's angles: worked out in 64 bits, held in 32."""
    turn = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * turn
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    rnd, kind = _Draws(seed), case["kind"]
    s = dict(case=case)
    if kind == "rotary":
        order = rnd.order(case["rows"]).tolist()
        old, new = _old_lengths(case), _new_lengths(case)
        old, new = [old[i] for i in order], [new[-1 - i] for i in order]  # the longest contexts get the shortest pieces
        tables, pages = _place_pages(rnd, [-(-(a + b) // case["page"]) for a, b in zip(old, new)])
        s["tables"], s["lens"], s["new"] = tables.to(torch.int32), _ints(old), new
        s["k_codes"], s["k_scale"] = _cache(rnd, pages, case["hkv"], case["page"], case["d"])
        s["v_codes"], s["v_scale"] = _cache(rnd, pages, case["hkv"], case["page"], case["d"])
        s["cu"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
        # one projection's output: the heads of q, k and v side by side
        x = rnd.normal(sum(new), case["hq"] + 2 * case["hkv"], case["d"]).to(DTYPES[case["dtype"]])
        s["q"], s["k"], s["v"] = x.split([case["hq"], case["hkv"], case["hkv"]], 1)
        s["rotary"] = _rotary_table(case["ctx"] + case["new"] + 1, case["rot"])
    elif kind == "shared":
        groups, beams, page, new = case["groups"], case["beams"], case["page"], case["new"]
        prompts, mine = _prompt_lengths(case), _own_lengths(case)
        own_order = [rnd.order(beams).tolist() for _ in range(groups)]
        lens = [[prompts[g] + mine[i] for i in own_order[g]] for g in range(groups)]
        full = [p // page for p in prompts]  # whole pages of the prompt: the same for all rows of a group
        rest = [[-(-n // page) - full[g] for n in lens[g]] for g in range(groups)]
        ids, pages = _place_pages(rnd, full + [n for x in rest for n in x])
        width = max(full[g] + max(rest[g]) for g in range(groups))
        tables = torch.full((groups, beams, width), -1, device="cuda")
        for g in range(groups):
            most = max(rest[g])
            tables[g, :, : full[g]] = ids[g, : full[g]]
            tables[g, :, full[g]: full[g] + most] = ids[groups + g * beams: groups + (g + 1) * beams, :most]
        s["tables"] = tables.view(groups * beams, width).to(torch.int32)
        s["lens"] = _ints(lens).flatten()
        s["cu_rows"] = _ints(list(range(0, groups * beams + 1, beams)))
        s["cu"] = _ints(list(range(0, groups * beams * new + 1, new)))
        s["k_codes"], s["k_scale"] = _cache(rnd, pages, case["hkv"], page, case["d"])
        s["v_codes"], s["v_scale"] = _cache(rnd, pages, case["hkv"], page, case["d"])
        s["q"] = (rnd.normal(groups * beams * new, case["hq"], case["d"]) * 1.5).to(DTYPES[case["dtype"]])
    else:
        b, w, v, n, m = case["batch"], case["beams"], case["vocab"], case["hist"], case["bias"]
        rows = b * w
        x = rnd.normal(b, w, v) * 3 + 2 * rnd.uniform(v).log()  # most tokens are rare
        s["logits"] = x.to(DTYPES[case["dtype"]])
        if case["penal"]:
            often = rnd.order(v)
            # tokens of a text: a few are frequent
            s["history"] = often[(v * rnd.uniform(rows, n) ** 4).long().clamp(max=v - 1)].to(torch.int32)
            lens = _spread(rows, max(1, n // 3), n)
            s["lens"] = _ints(lens)[rnd.order(rows)]
            s["prompt"] = (s["lens"] * rnd.uniform(rows) * 0.7).to(torch.int32)
            s["repetition"], s["presence"], s["frequency"] = 1 + 0.3 * rnd.uniform(rows), rnd.uniform(rows) * 0.8, rnd.uniform(rows) * 0.4
        if m:
            s["bias_tokens"] = torch.stack([rnd.order(v)[:m] for _ in range(rows)]).to(torch.int32)
            s["bias"] = rnd.normal(rows, min(m, v)) * 4
        if case["mask"] > 0:
            words = -(-v // 32)
            s["mask"] = torch.zeros(rows, words, device="cuda", dtype=torch.int32)
            for i in range(32):
                s["mask"] |= (rnd.uniform(rows, words) < case["mask"]).to(torch.int32) << i
    return s


def work(case):
    kind = case["kind"]
    if kind == "rotary":
        old, new = _old_lengths(case), _new_lengths(case)[::-1]
        tokens, seen = sum(new), set()
        for a, n in zip(old, new):
            seen.update(range(a, a + n))
        return dict(bytes=tokens * case["d"] * (6 * case["hkv"] + 4 * case["hq"]) + 4 * len(seen) * case["rot"],
                    flops=tokens * (3 * (case["hq"] + case["hkv"]) * case["rot"] + 4 * case["hkv"] * case["d"]))
    if kind == "shared":
        prompts, mine, new = _prompt_lengths(case), _own_lengths(case), case["new"]
        tokens = case["groups"] * case["beams"] * new
        held = sum(prompts) + case["groups"] * sum(mine)
        seen = sum(new * (p + m) - new * (new - 1) // 2 for p in prompts for m in mine)
        return dict(bytes=2 * held * case["hkv"] * case["d"] + 4 * tokens * case["hq"] * case["d"] + held // case["page"] * (8 * case["hkv"] + 4),
                    flops=4 * seen * case["hq"] * case["d"])
    rows, v, size = case["batch"] * case["beams"], case["vocab"], 4 if case["dtype"] == "fp32" else 2
    mask = 4 * rows * -(-v // 32) if case["mask"] > 0 else 0
    if case["place"]:
        return dict(bytes=mask + int(rows * v * (1 - case["mask"])) * size, flops=rows * v)
    held = sum(_spread(rows, max(1, case["hist"] // 3), case["hist"]))
    return dict(bytes=2 * rows * v * size + mask + 4 * held + 8 * rows * case["bias"], flops=4 * rows * v)


# ---- plain forms -------------------------------------------------------------------------------------------


def _rows_of_tokens(cu, tokens):
    return torch.searchsorted(cu[1:].contiguous(), torch.arange(tokens, device=cu.device, dtype=cu.dtype), right=True)


def _plain_rotate(x, table, inter):
    """x [tokens, heads, d] by each token's row of the table; in 64 bits, as codes beside a border depend on it."""
    half = table.shape[1] // 2
    x, cos, sin = x.double(), table[:, None, :half].double(), table[:, None, half:].double()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else (slice(0, half), slice(half, 2 * half))
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y.float()


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
    old, was, now = bits[which].view(F8).float(), scale[which][..., None, None], grown[which][..., None, None]
    again = (old * was / now).clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)
    keep = (was == now) | (torch.arange(page, device=x.device) >= (lens % page)[opened, None])[:, None, :, None]
    bits[which] = torch.where(keep, bits[which], again)
    by = grown[where][..., None]
    bits[where, :, inside] = torch.where(by > 0, x / by, 0).clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)
    scale.copy_(grown)


def _plain_rotary(s):
    row = _rows_of_tokens(s["cu"], s["q"].shape[0])
    at = s["lens"].long()[row] + torch.arange(len(row), device=row.device) - s["cu"].long()[row]
    table, inter = s["rotary"][at], s["case"]["inter"]
    k = _plain_rotate(s["k"], table, inter)
    _plain_quantise(k, s["k_codes"], s["k_scale"], s["tables"], s["lens"], s["cu"])
    _plain_quantise(s["v"], s["v_codes"], s["v_scale"], s["tables"], s["lens"], s["cu"])
    return _plain_rotate(s["q"], table, inter).to(s["q"].dtype), s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"]


def _plain_shared(s):
    q, tables, lens = s["q"], s["tables"].long(), s["lens"].long()
    rows, width = tables.shape
    tokens, hq, d = q.shape
    _, hkv, page, _ = s["k_codes"].shape
    new, group = tokens // rows, hq // hkv
    at = tables.clamp(min=0)

    def gathered(codes, scale):
        x = codes.view(torch.uint8)[at].view(F8).float() * scale[at][..., None, None]  # [R, M, Hkv, page, D]
        return x.permute(0, 2, 1, 3, 4).reshape(rows, hkv, width * page, d)

    key = torch.arange(width * page, device=q.device)
    there = (key < lens[:, None]) & (tables >= 0).repeat_interleave(page, 1)
    sees = key <= (lens - new)[:, None, None] + torch.arange(new, device=q.device)[None, :, None]  # [R, n, L]
    sees = (sees & there[:, None]).repeat_interleave(group, 1)
    x = q.float().view(rows, new, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(rows, hkv, new * group, d)
    score = x @ gathered(s["k_codes"], s["k_scale"]).transpose(2, 3) * d ** -0.5
    score = score.masked_fill(~sees[:, None], -math.inf)
    top = score.amax(3, keepdim=True)
    p = (score - top.masked_fill(top == -math.inf, 0)).exp()
    v = gathered(s["v_codes"], s["v_scale"]).masked_fill(~there[:, None, :, None], 0)
    out = (p @ v) / p.sum(3, keepdim=True).clamp(min=1e-30)
    return out.view(rows, hkv, new, group, d).permute(0, 2, 1, 3, 4).reshape(tokens, hq, d).to(q.dtype)


def _plain_logits(s):
    shape = s["logits"].shape
    x = s["logits"].float().view(-1, shape[-1])
    if "history" in s:
        history, at = s["history"].long(), torch.arange(s["history"].shape[1], device=x.device)
        told, said = at < s["lens"][:, None], (at < s["lens"][:, None]) & (at >= s["prompt"][:, None])
        seen = torch.zeros_like(x).scatter_add_(1, history, told.float())
        count = torch.zeros_like(x).scatter_add_(1, history, said.float())
        by = s["repetition"][:, None]
        x = torch.where(seen > 0, torch.where(x > 0, x / by, x * by), x)
        x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if "bias" in s:
        x = x.scatter_add(1, s["bias_tokens"].long(), s["bias"])
    if "mask" in s:
        bits = s["mask"][:, :, None] >> torch.arange(32, device=x.device, dtype=torch.int32) & 1
        x = x.masked_fill(bits.view(x.shape[0], -1)[:, : shape[-1]] == 0, -math.inf)
    x = x.view(shape).to(s["logits"].dtype)
    return s["logits"].copy_(x) if s["case"]["place"] else x


def run(s):
    kind = s["case"]["kind"]
    if own:
        return _run_own(s, kind)
    if kind == "rotary":
        return _plain_rotary(s)
    return _plain_shared(s) if kind == "shared" else _plain_logits(s)


def _run_own(s, kind):
    import chunked_kda_delta_gb300 as K

    one = s["case"].get("new") == 1
    cu = None if one else s.get("cu")
    cache = [s.get(x) for x in ("k_codes", "v_codes", "k_scale", "v_scale", "tables", "lens")]
    if kind == "rotary":
        q = K.kda_kvcache_append_rotary(s["q"], s["k"], s["v"], s["rotary"], *cache, cu_tokens=cu, interleaved=s["case"]["inter"])
        return q, s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"]
    if kind == "shared":
        return K.kda_kvcache_attention_shared(s["q"], *cache, s["cu_rows"], cu_tokens=cu)
    return K.kda_logits_penalize(s["logits"], history=s.get("history"), lens=s.get("lens"), prompt_lens=s.get("prompt"),
                                 repetition=s.get("repetition"), presence=s.get("presence"), frequency=s.get("frequency"),
                                 bias_tokens=s.get("bias_tokens"), bias=s.get("bias"), mask=s.get("mask"),
                                 out=s["logits"] if s["case"]["place"] else None)


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


def _exact_rotary(case, s):
    parts = {"q": [], "k": []}
    rot, inter = case["rot"], case["inter"]
    for r, n in enumerate(s["new"]):
        begin, old = int(s["cu"][r]), int(s["lens"][r])
        turn = torch.view_as_complex(s["rotary"][old: old + n].double().view(n, 2, rot // 2).transpose(1, 2).contiguous())
        for name in parts:
            x = s[name][begin: begin + n].double()
            z = x[..., :rot].unflatten(-1, (rot // 2, 2)) if inter else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, None])
            y = y.flatten(-2) if inter else y.transpose(-1, -2).flatten(-2)
            parts[name].append(torch.cat([y, x[..., rot:]], -1))
    got = [torch.cat(parts["q"])]
    for x, values in (("k", parts["k"]), ("v", [s["v"][int(s["cu"][r]): int(s["cu"][r]) + n].double() for r, n in enumerate(s["new"])])):
        codes, scale = s[x + "_codes"].to(torch.float64), s[x + "_scale"].double()
        for r, n in enumerate(s["new"]):
            old = int(s["lens"][r])
            for first in range(old - old % case["page"], old + n, case["page"]):
                a, b = max(first, old), min(first + case["page"], old + n)
                p, part = int(s["tables"][r, first // case["page"]]), values[r][a - old: b - old].transpose(0, 1)
                now = (part.abs().amax((1, 2)) / F8_MAX).float().double()  # the scale is held in 32 bits
                if a > first:
                    now = torch.maximum(now, scale[p])
                    by = torch.where(now > scale[p], scale[p] / now, 1.0)
                    codes[p, :, : a - first] = _nearest_e4m3(codes[p, :, : a - first] * by[:, None, None])
                scale[p] = now
                codes[p, :, a - first: b - first] = _nearest_e4m3(part / now[:, None, None])
        got += [codes, scale]
    return tuple(got)


def _exact_shared(case, s):
    outs, page, new, hkv = [], case["page"], case["new"], case["hkv"]
    for r in range(s["lens"].numel()):
        length = int(s["lens"][r])
        ids = s["tables"][r, : -(-length // page)].long()
        sides = []
        for x in ("k", "v"):
            c = s[x + "_codes"].view(torch.uint8)[ids].view(F8).to(torch.float64) * s[x + "_scale"][ids].double()[..., None, None]
            sides.append(c.transpose(0, 1).reshape(hkv, -1, case["d"])[:, :length])
        q = s["q"][r * new: (r + 1) * new].double().view(new, hkv, -1, case["d"])
        hidden = torch.arange(length, device="cuda") > (length - new + torch.arange(new, device="cuda"))[:, None]
        z = torch.einsum("nhgd,hld->hgnl", q, sides[0]) / math.sqrt(case["d"])
        w = torch.softmax(z.masked_fill(hidden, -math.inf), 3)
        outs.append(torch.einsum("hgnl,hld->nhgd", w, sides[1]).flatten(1, 2))
    return torch.cat(outs)


def _exact_logits(s):
    v = s["logits"].shape[-1]
    got = s["logits"].double().view(-1, v).clone()
    for r in range(got.shape[0]):
        if "history" in s:
            n, p = int(s["lens"][r]), int(s["prompt"][r])
            every = torch.bincount(s["history"][r, :n].long(), minlength=v) > 0
            count = torch.bincount(s["history"][r, p:n].long(), minlength=v).double()
            by = s["repetition"][r].double()
            got[r] = torch.where(every, torch.minimum(got[r] / by, got[r] * by), got[r])  # (by >= 1 here)
            got[r] -= s["frequency"][r].double() * count + s["presence"][r].double() * count.clamp(max=1)
        if "bias" in s:
            got[r, s["bias_tokens"][r].long()] += s["bias"][r].double()
        if "mask" in s:
            t = torch.arange(v, device="cuda")
            got[r, (s["mask"][r].long()[t // 32] >> (t % 32)) % 2 == 0] = -math.inf
    return got.view(s["logits"].shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "rotary":
        return _exact_rotary(case, s)
    return _exact_shared(case, s) if case["kind"] == "shared" else _exact_logits(s)
