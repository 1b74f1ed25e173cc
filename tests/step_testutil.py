"""References in 64 bits of the rotating append, and helpers of the tests of a decoding step's operators."""
import numpy as np
import torch

import serving_testutil as ref

F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def ints(x):
    return torch.as_tensor(np.asarray(x)).to(torch.int32).cuda()


def cu_of(counts):
    return ints([0] + list(np.cumsum(counts)))


def rotary_table(n, rot, far=0):
    """Cosines and sines of positions far .. far + n - 1, in fp32."""
    turn = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    angle = (far + np.arange(n))[:, None] * turn
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def rotate(x, rows, inter):
    """x [T, H, D] by rows [T, rot] (None: as it is), in 64 bits."""
    y = np.asarray(x, dtype=np.float64).copy()
    half = rows.shape[1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        c, s = rows[:, i, None].astype(np.float64), rows[:, half + i, None].astype(np.float64)
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, b] * c + x[:, :, a] * s
    return y


def check_quantised(y, before, after, scale_before, scale_after, tables, lens, counts, page):
    """The cache side `after` against values y [T, H, D] in 64 bits, appended to `before`.

    A value off by 2^-22 of itself (two units in the last place of fp32) moves a page's scale by as much
    and one rounding more; a code is the nearest one to a quotient that is off by 2^-21 at most."""
    want_scale, touched = scale_before.astype(np.float64), np.zeros(before.shape[:1] + (before.shape[2],), bool)
    again = {}
    at = 0
    for r, n in enumerate(counts):
        pos, done = int(lens[r]), 0
        while done < n:
            slot, off = divmod(pos + done, page)
            m = min(page - off, n - done)
            p = int(tables[r, slot]) if slot < tables.shape[1] else -1
            part = y[at + done: at + done + m]
            done += m
            if not 0 <= p < before.shape[0]:
                continue
            top = np.abs(part).max((0, 2)) / 448.0
            if off > 0:
                top = np.maximum(top, want_scale[p])
                again[p] = off
            want_scale[p] = top
            touched[p, off: off + m] = True
            s = scale_after[p].astype(np.float64)
            assert (np.abs(s - top) <= 2.0 ** -21 * top).all()
            codes = ref.E4M3[after[p, :, off: off + m]].transpose(1, 0, 2)
            with np.errstate(all="ignore"):
                x = np.where(s[None, :, None] > 0, part / s[None, :, None], 0)
            step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -20))), -6) / 8
            assert (np.abs(codes - x) <= step / 2 + 2.0 ** -21 * np.abs(x)).all()
        at += n
    for p in range(before.shape[0]):
        off = again.get(p, 0)
        same = np.ones(before.shape[2], bool)
        same[touched[p]] = False
        for h in range(before.shape[1]):
            old = before[p, h]
            if off:
                was, now = scale_before[p, h], scale_after[p, h]
                if now > was:
                    old = old.copy()
                    old[:off] = ref.to_e4m3(ref.quotient(np.float32(ref.E4M3[old[:off]]) * np.float32(was), now))
                    # what rounds to zero keeps no sign here
                    a, b = old[:off], after[p, h][:off]
                    assert ((a == b) | ((a | b) & 0x7F == 0)).all()
                    same[:off] = False
                else:
                    assert now == was
            elif not touched[p].any():
                assert scale_after[p, h] == scale_before[p, h]
            assert (after[p, h][same] == old[same]).all()
