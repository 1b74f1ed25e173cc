"""References of the serving operators in 64 bits (numpy), from their definitions."""
import math

import numpy as np

F8_MAX = 448.0


def e4m3_table():
    """Value of every e4m3 code (NaN at 0x7f and 0xff)."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if (c & 0x7F) == 0x7F:
            x = math.nan
        v[c] = -x if c & 0x80 else x
    return v


E4M3 = e4m3_table()


def to_e4m3(x):
    """Codes of finite values in [-448, 448], round to nearest even (x exact in 64 bits)."""
    x = np.asarray(x, dtype=np.float64)
    pos = E4M3[:127]
    a = np.abs(x)
    up = np.clip(np.searchsorted(pos, a), 0, 126)
    down = np.maximum(up - 1, 0)
    lo, hi = a - pos[down], pos[up] - a
    pick = np.where(lo < hi, down, np.where(hi < lo, up, np.where(down % 2 == 0, down, up)))
    return (pick | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def quotient(x, s):
    """fp32 quotient of the append's definition."""
    x, s = np.float32(x), np.float32(s)
    with np.errstate(all="ignore"):
        q = x / s if s > 0 else np.zeros_like(x)
    q = np.where(np.isnan(x), np.float32(0), q)
    q = np.where(np.isinf(x), np.copysign(np.float32(F8_MAX), x), q)
    return np.clip(q, -F8_MAX, F8_MAX)


def append(x, codes, scale, tables, lens, counts, page):
    """Appends x [T, H, D] to codes [P, H, page, D] and scale [P, H], in place."""
    at = 0
    for r, n in enumerate(counts):
        new, pos = x[at: at + n], int(lens[r])
        at += n
        done = 0
        while done < n:
            slot, off = divmod(pos + done, page)
            m = min(page - off, n - done)
            p = int(tables[r, slot]) if slot < tables.shape[1] else -1
            part = new[done: done + m].transpose(1, 0, 2)
            done += m
            if not 0 <= p < codes.shape[0]:
                continue
            for h in range(codes.shape[1]):
                v = np.float32(part[h])
                finite = np.abs(v[np.isfinite(v)])
                s = np.float32(finite.max() if finite.size else 0) / np.float32(F8_MAX)
                if off > 0:
                    was = np.float32(scale[p, h])
                    if s > was:
                        old = np.float32(E4M3[codes[p, h, :off]]) * was
                        codes[p, h, :off] = to_e4m3(quotient(old, s))
                    else:
                        s = was
                scale[p, h] = s
                codes[p, h, off: off + m] = to_e4m3(quotient(v, s))


def attention(q, kc, vc, ks, vs, tables, lens, counts, page, scale):
    """(out, bound) in 64 bits: bound = sum_j p_j |v_j|, what rounding errors of weights scale with."""
    hq, hkv, d = q.shape[1], kc.shape[1], q.shape[2]
    g = hq // hkv
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    at = 0
    for r, n in enumerate(counts):
        length = int(lens[r])
        ids = tables[r, : -(-length // page)]
        ok = np.repeat((ids >= 0) & (ids < kc.shape[0]), page)[:length]
        ids = np.where((ids >= 0) & (ids < kc.shape[0]), ids, 0)
        side = []
        for c, s in ((kc, ks), (vc, vs)):
            x = E4M3[c[ids]] * s[ids].astype(np.float64)[..., None, None]
            side.append(x.transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :length])
        for i in range(n):
            p = length - n + i
            if p < 0:
                continue
            sees = ok[: p + 1]
            for h in range(hq):
                if not sees.any():
                    continue
                k, v = side[0][h // g][: p + 1][sees], side[1][h // g][: p + 1][sees]
                z = scale * (k @ q[at + i, h].astype(np.float64))
                w = np.exp(z - z.max())
                w /= w.sum()
                out[at + i, h], bound[at + i, h] = w @ v, w @ np.abs(v)
        at += n
    return out, bound


def free_pages(held):
    return iter(np.nonzero(held == 0)[0].tolist())


def alloc(tables, refs, want):
    new, held = tables.copy(), refs.copy()
    free = free_pages(held)
    for r in range(tables.shape[0]):
        for j in range(min(tables.shape[1], int(want[r]))):
            if new[r, j] < 0:
                p = next(free, -1)
                new[r, j] = p
                if p >= 0:
                    held[p] = 1
    return new, held


def fork(tables, refs, parents, lens, page):
    """(new tables, new refs, copies [(src, dst)])."""
    rows, width = tables.shape
    pages = len(refs)
    held = refs.copy()
    new = np.full_like(tables, -1)
    private = []
    for r in range(rows):
        for j in range(width):
            if 0 <= tables[r, j] < pages:
                held[tables[r, j]] -= 1
    for r in range(rows):
        a = int(parents[r])
        if not 0 <= a < rows:
            continue
        full = int(lens[a]) // page if page else 0
        for j in range(width):
            x = int(tables[a, j])
            if not 0 <= x < pages:
                continue
            if j < full:
                new[r, j] = x
                held[x] += 1
            else:
                private.append((r, j, x))
    need = []
    taken = {x: True for x in range(pages) if held[x] > 0}
    for r, j, x in private:
        if x not in taken:
            taken[x] = True
            new[r, j] = x
            held[x] = 1
        else:
            need.append((r, j, x))
    free = free_pages(held)
    copies = []
    for r, j, x in need:
        p = next(free, -1)
        new[r, j] = p
        if p >= 0:
            held[p] = 1
            copies.append((x, p))
    return new, held, copies


def compact(tables, refs):
    live = np.nonzero(refs > 0)[0]
    n = len(live)
    page_map = np.full(len(refs), -1)
    holes = iter([x for x in range(n) if refs[x] <= 0])
    copies = []
    for x in live:
        page_map[x] = x if x < n else next(holes)
        if x >= n:
            copies.append((x, page_map[x]))
    new_refs = np.zeros_like(refs)
    new_refs[page_map[live]] = refs[live]
    ok = (tables >= 0) & (tables < len(refs))
    new = np.where(ok, page_map[np.where(ok, tables, 0)], -1)
    return new, new_refs, page_map, n, copies


def beam(logits, scores, k, done=None, eos=-1):
    """New scores (fp32 rounding of the definition's two steps), tokens, parents, done."""
    b, w, v = logits.shape
    x = logits.astype(np.float64)
    x = np.where(np.isfinite(x), x, -np.inf)
    outs = []
    for i in range(b):
        keys = []
        for j in range(w):
            if done is not None and done[i, j]:
                if scores[i, j] > -np.inf:
                    keys.append((-float(scores[i, j]), j * v + eos))
                continue
            if not np.isfinite(x[i, j]).any():
                continue
            top = x[i, j].max()
            lse = np.float32(top + np.log(np.exp(x[i, j] - top).sum()))
            with np.errstate(all="ignore"):
                total = np.float32(scores[i, j]) + (np.float32(x[i, j]) - lse)
            total = np.where(np.isfinite(x[i, j]) & (total > -np.inf), total, -np.inf)
            at = np.lexsort((np.arange(v), -total))[:k]
            keys += [(-float(total[t]), j * v + int(t)) for t in at if total[t] > -np.inf]
        keys = sorted(keys)[:k]
        s = [-a for a, _ in keys] + [-math.inf] * (k - len(keys))
        t = [f % v for _, f in keys] + [-1] * (k - len(keys))
        p = [i * w + f // v for _, f in keys] + [-1] * (k - len(keys))
        e = [int(p_ < 0 or t_ == eos or (done is not None and done[i, p_ - i * w])) for t_, p_ in zip(t, p)]
        outs.append((s, t, p, e))
    return tuple(np.array([o[n] for o in outs]) for n in range(4))
