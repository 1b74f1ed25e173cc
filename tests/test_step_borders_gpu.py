"""Calls of a decoding step's operators at the borders of what they document: offsets, lengths and tokens out of range,
values that are not finite, scales any distance apart, scratch, threads; and what rows are found to share."""
import ctypes
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
import serving_testutil as ref
import test_logits_gpu as logits
import test_rotary_gpu as rotary
from chunked_kda_delta_gb300.kda import KdaKvCache, KdaLogitsRules, KdaScratchAllocator
from step_testutil import DT, check_quantised, cu_of, ints, rotary_table, rotate
from test_shared_attention_gpu import gpu_cache, make_cache

pytestmark = pytest.mark.gpu
P = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr() if isinstance(t, torch.Tensor) else t)  # noqa: E731


def test_penalties_from_several_threads():
    # the C calls run at the same time and need different amounts of shared memory for the same kernel
    lib = K.load_library()
    rng = np.random.default_rng(1)
    rows, vocab, jobs = 300, 25003, []
    x = torch.as_tensor(rng.standard_normal((rows, vocab)).astype(np.float32)).cuda().bfloat16()
    for width, biases in ((100, 20), (2000, 100), (100, 20), (5000, 300)):
        made = logits.make(rng, rows, vocab, width=width, biases=biases, lens=False)
        t = {k: ints(v) if v.dtype == np.int64 else torch.as_tensor(v).cuda() for k, v in made.items()}
        rules = KdaLogitsRules(history_width=width, num_bias=biases, **{k: v.data_ptr() for k, v in t.items()})
        jobs.append((t, rules, torch.zeros_like(x), K.kda_logits_penalize(x, **t), torch.cuda.Stream().cuda_stream))
    torch.cuda.synchronize()

    def work(job):
        _, rules, out, _, stream = job
        return {lib.kda_logits_penalize(ctypes.byref(rules), rows, vocab, P(x), 1, vocab, P(out), vocab, P(stream)) for _ in range(1500)}

    with ThreadPoolExecutor(len(jobs)) as pool:
        codes = list(pool.map(work, jobs))
    torch.cuda.synchronize()
    assert codes == [{0}] * len(jobs)
    for _, _, out, want, _ in jobs:
        assert torch.equal(out, want)


def rotated(x, rows, inter):
    """x [T, H, D] turned by rows in 64 bits, products that leave fp32 infinite."""
    y = x.astype(np.float64)
    half = rows.shape[1] // 2
    with np.errstate(all="ignore"):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
            c, s = (rows[:, j, None].astype(np.float64) for j in (i, half + i))
            over = lambda z: np.where(np.abs(z) > np.finfo(np.float32).max, np.copysign(np.inf, z), z)  # noqa: E731
            y[:, :, a], y[:, :, b] = over(x[:, :, a] * c) - over(x[:, :, b] * s), over(x[:, :, b] * c) + over(x[:, :, a] * s)
    return y


@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_infinite_values_are_rotated_to_infinities(n, inter, dtype):
    # at angles that are not 0, either member of a pair or both; and products past fp32 under a scaled table
    rng = np.random.default_rng(n)
    lens, counts, d, rot = [7, 30], [n, n], 64, 64
    codes, scales, tab, x = rotary.make(rng, lens, counts, 3, 2, d, 16, dtype)
    i, j = (0, 1) if inter else (0, 32)  # channels of a pair
    inf = float("inf")
    x[0, 0, i], x[0, 1, j], x[0, 2, j] = inf, inf, -inf   # queries
    x[0, 3, j], x[0, 4, i] = inf, -inf                    # keys
    x[n, 0, i], x[n, 0, j] = inf, inf
    x[n, 3, i], x[n, 3, j] = inf, -inf
    rows = rotary_table(64, rot)
    rows[30:] *= 1.5
    if dtype == "bf16":
        x[n, 1, j], x[n, 2, i] = 3e38, -3e38
        x[n, 4, j] = 3e38
        rows[30:, [0, rot // 2]] = -1.25, 1.5  # of the first pair: cosine and sine
    at = rotary.places(lens, counts)
    dev = rotary.device(codes, scales, tab)
    q, k, v = x.cuda().split([3, 2, 2], 1)
    K.kda_get_device_status()
    out = K.kda_kvcache_append_rotary(q, k, v, torch.as_tensor(rows).cuda(), *dev, ints(lens), cu_tokens=cu_of(counts) if n > 1 else None, interleaved=inter)
    assert K.kda_get_device_status() == 9
    want = rotated(x[:, :3].double().numpy(), rows[at], inter)
    got = out.double().cpu().numpy()
    assert np.isinf(want).any() and np.isnan(want).any()
    assert (np.isnan(got) == np.isnan(want)).all()
    top = float(torch.finfo(DT[dtype]).max)
    big = np.abs(want) > top * (1 + 2.0 ** -12)
    assert (got[big] == np.copysign(np.inf, want[big])).all()
    ok = np.isfinite(want) & (np.abs(want) <= top)
    eps = torch.finfo(DT[dtype]).eps / 2
    assert (np.abs(got[ok] - want[ok]) <= (eps + 2.0 ** -21) * np.abs(want[ok]) + 2.0 ** -25).all()
    # keys: infinities are the largest code, NaN is 0, and neither enters a page's scale
    want = rotated(x[:, 3:5].double().numpy(), rows[at], inter)
    got = dev[0].double().cpu().numpy()
    for token in (0, n):
        r, pos = token // n, lens[token // n]
        c = got[tab[r, pos // 16], :, pos % 16]
        assert (c[np.isposinf(want[token])] == 448).all() and (c[np.isneginf(want[token])] == -448).all() and (c[np.isnan(want[token])] == 0).all()
    assert np.isinf(want[0]).sum() >= 4
    fine = np.where(np.isfinite(want), want, 0)
    for page in np.unique([tab[r, p // 16] for r in range(2) for p in range(lens[r], lens[r] + n)]):
        mine = [fine[t] for t in range(2 * n) if tab[t // n, at[t] // 16] == page]
        top = np.maximum(np.abs(mine).max((0, 2)) / 448, 0 if any(at[t] % 16 == 0 for t in range(2 * n) if tab[t // n, at[t] // 16] == page) else scales[0][page])
        assert (np.abs(dev[2][page].double().cpu().numpy() - top) <= 2.0 ** -21 * top).all()


@pytest.mark.parametrize("order", [1, -1, 0])
@pytest.mark.parametrize("small,large", [(0, 2.0 ** 110), (2.0 ** -70, 2.0 ** 60), (2.0 ** -20, 2.0 ** 110)])
@pytest.mark.parametrize("n,hq,d,shared", [(1, 4, 64, 256), (1, 16, 128, 256), (1, 24, 64, 256), (100, 8, 64, 256), (60, 16, 128, 128), (1, 8, 64, 5120)])
def test_scales_of_values_any_distance_apart(n, hq, d, shared, small, large, order):
    # equal scores; scales of v are large in the prefix and small behind it, or the other way, or either by
    # chance.  Keys of small scales keep their share of the weights.  The bound is the one of rows that share nothing.
    rng = np.random.default_rng(shared + d)
    behind = 200 if shared < 5120 else 3000
    kc, vc, ks, vs, tables, lens = make_cache(rng, [[(0, shared + behind)] + [(shared, shared + behind - i) for i in range(1, 4)]], 16, 2, d)
    first = np.zeros(len(vs), bool)
    first[tables[0, : shared // 16]] = True
    vs[:] = np.where(rng.random(len(vs)) < 0.5 if order == 0 else first == (order > 0), large, small)[:, None]
    q = torch.zeros(4 * n, hq, d, dtype=torch.bfloat16)
    want, weight = ref.attention(q.double().numpy(), kc, vc, ks, vs, tables, lens, [n] * 4, 16, 0.125)
    got = K.kda_kvcache_attention_shared(q.cuda(), *gpu_cache(kc, vc, ks, vs, tables), ints(lens), ints([0, 4]), cu_tokens=cu_of([n] * 4),
                                         scale=0.125).double().cpu().numpy()
    assert np.isfinite(got).all()
    allowed = 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * weight + 1e-6
    assert (np.abs(got - want) <= allowed).all(), np.max(np.abs(got - want) / allowed)


class Scratch:
    """Scratch of this thread's calls: their sizes, and whatever `give` returns (nothing: the calls end there)."""

    def __init__(self, give=lambda size: None):
        def allocate(context, size, stream):
            self.sizes.append(size)
            return give(size)
        self.sizes = []
        fields = KdaScratchAllocator._fields_
        self.a = KdaScratchAllocator(fields[0][1](allocate), fields[1][1](lambda context, p, size, stream: None), 0)

    def __enter__(self):
        assert K.load_library().kda_set_scratch_allocator(ctypes.byref(self.a), None) == 0
        return self

    def __exit__(self, *error):
        assert K.load_library().kda_set_scratch_allocator(None, None) == 0


def scratch_sizes(rows, groups, hq, hkv, d, width=1024):
    """Bytes of scratch that the calls with and without shared prefixes ask for."""
    lib, at, sizes = K.load_library(), iter(range(1 << 40, 1 << 47, 1 << 40)), []
    # (addresses far apart: no work is put on the stream without scratch)
    c = KdaKvCache(*(next(at) for _ in range(4)), 1 << 10, 64, hkv, d, next(at), rows, width)
    q, lens, cu_rows, out = (next(at) for _ in range(4))
    with Scratch() as s:
        tail = (ctypes.c_float(0.1), P(out), hq * d, None)
        assert lib.kda_kvcache_attention_shared(ctypes.byref(c), P(q), hq, 0, hq * d, rows, P(lens), None, P(cu_rows), groups, *tail) == 4
        assert lib.kda_kvcache_attention(ctypes.byref(c), P(q), hq, 0, hq * d, rows, P(lens), None, *tail) == 4
    return s.sizes


@pytest.mark.parametrize("rows,groups,hq,hkv,d", [(16384, 4096, 64, 8, 128), (2048, 512, 64, 64, 128), (16384, 16383, 64, 64, 128), (2048, 1024, 64, 64, 128),
                                                  (4096, 2048, 64, 8, 128), (1024, 512, 32, 32, 128), (32768, 9000, 64, 32, 64)])
def test_scratch_of_shared_prefixes_is_bounded(rows, groups, hq, hkv, d):
    shared, _ = scratch_sizes(rows, groups, hq, hkv, d)
    assert shared <= 2 ** 31


def test_scratch_where_prefixes_are_shared_and_where_not():
    state = 1024 * 64 * 128 * 4
    shared, alone = scratch_sizes(1024, 256, 64, 8, 128)
    assert state < shared <= 2 ** 31 and alone < state
    shared, alone = scratch_sizes(2, 1, 8, 1, 128, width=1 << 16)  # (of rows with so few query rows three share, not two)
    assert shared == alone
    shared, alone = scratch_sizes(3, 1, 8, 1, 128, width=1 << 16)
    assert shared > alone
    shared, alone = scratch_sizes(16384, 4096, 64, 64, 128)  # (of too many groups' and heads' prefixes the parts would take 35 GB)
    assert shared == alone


def found_in_scratch(groups, lens, tables, page, hq, hkv, counts=None, cu=None, cu_rows=None, compare=True):
    """Runs attention of rows with shared prefixes on the caller's scratch and returns that as bytes."""
    lib, held = K.load_library(), []

    def give(size):
        held.append(torch.full((size,), 0xEE, dtype=torch.uint8, device="cuda"))
        return held[-1].data_ptr()

    rows, d, pages = len(lens), 64, int(tables.max()) + 1
    gen = torch.Generator("cuda").manual_seed(1)
    codes = [(torch.randn(pages, hkv, page, d, device="cuda", generator=gen) * 50).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.rand(pages, hkv, device="cuda", generator=gen) / 50 + 0.01 for _ in range(2)]
    tab = torch.full((rows, 4_000_000 // page), -1, dtype=torch.int32, device="cuda")
    tab[:, : tables.shape[1]] = ints(tables)
    tokens = rows if cu is None else counts
    q = torch.randn(tokens, hq, d, device="cuda", generator=gen).bfloat16()
    ln, gr, out = ints(lens), ints(cu_rows if cu_rows is not None else np.cumsum([0] + groups)), torch.zeros_like(q)
    c = KdaKvCache(*(t.data_ptr() for t in codes + scales), pages, page, hkv, d, tab.data_ptr(), rows, tab.shape[1])
    with Scratch(give) as s:
        assert lib.kda_kvcache_attention_shared(ctypes.byref(c), P(q), hq, 0, hq * d, tokens, P(ln), P(cu), P(gr), gr.numel() - 1, ctypes.c_float(0.1), P(out),
                                                hq * d, P(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert len(s.sizes) == 1
    if compare:
        want = K.kda_kvcache_attention(q, *codes, *scales, tab, ln, cu_tokens=cu, scale=0.1)
        assert (out.double() - want.double()).abs().max() <= 2.0 ** -7 * want.abs().max()
    return held[0].cpu().numpy().tobytes()


def records(begin, tokens, shared, row):
    """A group: first token, its rows' tokens, tokens of the prefix, the row whose table is read."""
    return np.array([(b, t, s, r, 0) if s else (b, 0, 0, 0, 0) for b, t, s, r in zip(begin, tokens, shared, row)],
                    dtype=[("begin", "<i8"), ("tokens", "<i4"), ("shared", "<i4"), ("row", "<i4"), ("unused", "<i4")]).tobytes()


def private(rows, pages):
    return np.arange(rows * pages).reshape(rows, pages)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_what_rows_share_is_found(page):
    # groups of four rows: what they have in common ends where a table differs, where a row's first new token is, in units of 128
    n = 1024 // page
    tables = private(24, n)
    lens = np.full(24, 1000)
    for g, common in enumerate([128, 1024, 640, 640, 0, 512]):
        tables[4 * g: 4 * g + 4, : common // page] = tables[4 * g, : common // page]
    lens[4:8] = [513, 1000, 600, 514]           # 512 keys before the least row's token
    lens[8:12] = [512, 1000, 600, 514]          # 511 keys: 384
    tables[14, 300 // page] = tables[23, n - 1]  # a page of its own among the common ones
    lens[20:24] = [1, 1000, 1000, 1000]
    shared = [128, 512, 384, 256, 0, 0]
    got = found_in_scratch([4] * 6, lens, tables, page, 8, 1)
    assert records(range(0, 24, 4), [4] * 6, shared, range(0, 24, 4)) in got
    assert np.repeat(shared, 4).astype("<i4").tobytes() in got


@pytest.mark.parametrize("length,shared", [(127, 0), (128, 0), (129, 128), (130, 128), (256, 128), (257, 256)])
def test_units_of_128_tokens(length, shared):
    tables = np.tile(private(1, 32), (3, 1))
    lens = np.array([400, length, 300])
    got = found_in_scratch([3], lens, tables, 16, 4, 1)
    assert records([0], [3], [shared], [0]) in got
    assert np.full(3, shared, "<i4").tobytes() in got


def test_rows_that_share():
    # with up to eight query rows a key/value head three rows share, of more two do
    tables = np.repeat(private(3, 32), [2, 3, 1], 0)
    lens = np.full(6, 500)
    got = found_in_scratch([2, 3, 1], lens, tables, 16, 8, 1)
    assert records([0, 2, 5], [2, 3, 1], [0, 384, 0], [0, 2, 0]) in got
    assert np.array([0, 0, 384, 384, 384, 0], "<i4").tobytes() in got
    got = found_in_scratch([2, 3, 1], lens, tables, 16, 16, 1)
    assert records([0, 2, 5], [2, 3, 1], [384, 384, 0], [0, 2, 0]) in got


def test_rows_without_tokens():
    tables = np.tile(private(1, 32), (5, 1))
    tables[1] = -1  # an ended beam
    lens = np.array([500, 0, 400, 300, 500])
    got = found_in_scratch([5], lens, tables, 16, 16, 1, counts=6, cu=ints([0, 2, 2, 4, 5, 6]))
    assert records([0], [6], [256], [0]) in got
    assert np.full(5, 256, "<i4").tobytes() in got
    # a first row without tokens; two groups
    order = [1, 0, 2, 3, 4]
    got = found_in_scratch([3, 2], lens[order], tables[order], 16, 16, 1, counts=6, cu=ints([0, 0, 2, 4, 5, 6]))
    assert records([0, 4], [4, 2], [384, 256], [1, 3]) in got


@pytest.mark.parametrize("cu_rows", [[0, 3, 5], [1, 3, 6], [0, 7, 6], [0, -1, 6]])
def test_malformed_groups_share_nothing(cu_rows):
    tables, lens = np.repeat(private(2, 32), 3, 0), np.full(6, 500)
    K.kda_get_device_status()
    got = found_in_scratch([3, 3], lens, tables, 16, 16, 1, cu_rows=cu_rows)
    assert K.kda_get_device_status() != 0
    assert records([0, 0], [0, 0], [0, 0], [0, 0]) in got and np.zeros(6, "<i4").tobytes() in got


# Offsets that go back, leave the tokens or do not begin or end with them, also where a group's rows add up to what its
# first and last offset say, and where groups come again.
@pytest.mark.parametrize("cu", [[0, 3, 2, 4, 5, 7, 8], [-3, 2, 5, 9, 4, 6, 8], [0, 2, 6, 3, 8, 11, 8], [0, 4, 8, 0, 4, 8, 8], [1, 2, 3, 4, 5, 6, 8], [0, 2, 3, 4, 5, 6, 7],
                                [0, 4, 2, 6, 20, 8, 8], [0, 8, 8, 0, 8, 0, 8]])
@pytest.mark.parametrize("groups", [[6], [1, 5], [3, 3], [2, 1, 2, 1]])
def test_nothing_is_shared_with_malformed_offsets(cu, groups):
    tables, lens = np.tile(private(1, 32), (6, 1)), np.full(6, 500)
    K.kda_get_device_status()
    got = found_in_scratch(groups, lens, tables, 16, 16, 1, counts=8, cu=ints(cu), compare=False)
    assert K.kda_get_device_status() != 0
    begin = np.cumsum([0] + groups)[:-1]
    assert records([cu[r] for r in begin], groups, [0] * len(groups), begin) in got
    assert np.zeros(6, "<i4").tobytes() in got


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n", [1, 3])
def test_rows_of_negative_length(n, inter):
    # their tokens have no pages; queries of places before 0 are outside of the table, those from 0 on are turned
    rng = np.random.default_rng(n)
    lens, counts = [20, -2, 5], [n] * 3
    codes, scales, tab, x = rotary.make(rng, [20, 0, 5], counts, 3, 2, 64, 16, "bf16")
    rows = rotary_table(40, 64)
    at = rotary.places(lens, counts)
    plain = np.concatenate([np.ones((1, 32)), np.zeros((1, 32))], 1).astype(np.float32)
    for positions in (None, at[::-1].copy() + 2):
        dev = rotary.device(codes, scales, tab)
        q, k, v = x.cuda().split([3, 2, 2], 1)
        K.kda_get_device_status()
        out = K.kda_kvcache_append_rotary(q, k, v, torch.as_tensor(rows).cuda(), *dev, ints(lens), cu_tokens=cu_of(counts) if n > 1 else None,
                                          positions=None if positions is None else ints(positions), interleaved=inter)
        assert K.kda_get_device_status() == 1
        by = at if positions is None else positions
        turned = np.where((by < 0)[:, None], plain, rows[np.maximum(by, 0)])
        y = [rotate(t.double().numpy(), turned, inter) for t in x.split([3, 2, 2], 1)[:2]]
        rotary.check_q(out, y[0], "bf16")
        there = [0, 2]
        keep = np.concatenate([np.arange(r * n, r * n + n) for r in there])
        check_quantised(y[1][keep], codes[0], dev[0].view(torch.uint8).cpu().numpy(), scales[0], dev[2].cpu().numpy(), tab[there],
                        [lens[r] for r in there], [n] * 2, 16)


@pytest.mark.parametrize("n", [1, 45])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", [False, True])
def test_angles_of_zero_give_the_appends_values(n, dtype, inter):
    # with zeros of both signs beside partners of both signs: equal but for the sign of zero
    rng = np.random.default_rng(n)
    lens, counts = [0, 7, 30], [n] * 3
    codes, scales, tab, x = rotary.make(rng, lens, counts, 3, 2, 128, 32, dtype)
    x[torch.as_tensor(rng.random(x.shape) < 0.3)] = 0.0
    x[torch.as_tensor(rng.random(x.shape) < 0.3)] = -0.0
    one = torch.cat([torch.ones(128, 32), torch.zeros(128, 32)], 1).cuda()
    a, b = rotary.device(codes, scales, tab), rotary.device(codes, scales, tab)
    q, k, v = x.cuda().split([3, 2, 2], 1)
    cu = cu_of(counts) if n > 1 else None
    out = K.kda_kvcache_append_rotary(q, k, v, one, *a, ints(lens), cu_tokens=cu, interleaved=inter)
    K.kda_kvcache_append(k, v, *b, ints(lens), cu_tokens=cu)
    assert (out == q).all()
    for s, t in zip(a[:4], b[:4]):
        assert (s.float() == t.float()).all()
    assert torch.equal(a[1].view(torch.uint8), b[1].view(torch.uint8))  # values are not turned


def test_histories_without_penalties_are_not_read():
    x = torch.randn(3, 100, device="cuda")
    history = torch.full((3, 7), 10 ** 6, dtype=torch.int32, device="cuda")
    bias_tokens, bias = ints([[5], [6], [7]]), torch.full((3, 1), 2.0, device="cuda")
    want = x.clone()
    want[[0, 1, 2], [5, 6, 7]] += 2
    K.kda_get_device_status()
    assert torch.equal(K.kda_logits_penalize(x, history=history, lens=ints([8, -1, 7]), bias_tokens=bias_tokens, bias=bias), want)
    assert K.kda_get_device_status() == 0
    K.kda_logits_penalize(x, history=history, presence=torch.zeros(3, device="cuda"))
    assert K.kda_get_device_status() == 1


def check_logits(got, x, rules, dtype, adds=0):
    """As in tests/test_logits_gpu.py, with NaN as wrong as any other value."""
    want, size, touched = logits.reference(x.double().numpy().reshape(-1, x.shape[-1]), rules)
    assert got.shape == x.shape
    wrong_logits(got.cpu().reshape(want.shape), x.reshape(want.shape), want, size, touched, dtype, adds)


def wrong_logits(got, x, want, size, touched, dtype, adds):
    g, masked = got.double().numpy(), np.isneginf(want)
    assert np.isneginf(g[masked]).all()
    same = torch.as_tensor(~touched & ~masked)
    assert torch.equal(got[same], x[same])
    ok = touched & ~masked
    allowed = torch.finfo(DT[dtype]).eps / 2 * np.abs(want) + (4 + adds) * 2.0 ** -23 * size + (2.0 ** -24 if dtype == "fp16" else 0)
    with np.errstate(invalid="ignore"):
        assert (np.abs(g - want) <= allowed)[ok].all()


@pytest.mark.parametrize("vocab", [1, 33, 500, 32001, 70000])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("place", [False, True])
@pytest.mark.parametrize("rules", [dict(width=100, biases=33, mask=0.6), dict(width=5000, lens=False), dict(biases=700), dict(width=6000, biases=10, mask=0.9)])
def test_penalised_logits_are_numbers(vocab, dtype, place, rules):
    rng = np.random.default_rng(vocab)
    made = logits.make(rng, 6, vocab, **rules)
    x = torch.as_tensor(rng.standard_normal((2, 3, vocab)) * 5).to(DT[dtype])
    y = x.cuda()
    check_logits(logits.call(y, made, out=y if place else None), x, made, dtype, adds=rules.get("biases", 0))


def test_large_vocabularies_are_numbers():
    rng = np.random.default_rng(4)
    rows, vocab = 300, 600_001
    made = logits.make(rng, rows, vocab, width=50, biases=3, mask=0.9)
    x = torch.randn(rows, vocab, device="cuda").to(torch.bfloat16)
    got, some = logits.call(x, made), [0, 1, 150, 298, 299]
    check_logits(got[some], x[some].cpu(), {k: v[some] for k, v in made.items()}, "bf16", adds=3)


def test_calls_repeat_themselves():
    # the same bits in every call: no order of sums is left to chance
    rng = np.random.default_rng(9)
    groups = [[(0, 3000), (2900, 2950), (2900, 2999)], [(0, 700), (640, 690), (640, 720)]]
    cache = make_cache(rng, groups, 16, 2, 128)
    lens = ints(cache[5])
    dev = gpu_cache(*cache[:5])
    for n, hq in ((1, 8), (1, 32), (40, 16)):
        q = torch.randn(6 * n, hq, 128, device="cuda").bfloat16()
        call = lambda: K.kda_kvcache_attention_shared(q, *dev, lens, ints([0, 3, 6]), cu_tokens=cu_of([n] * 6))  # noqa: E731
        want = call()
        assert all(torch.equal(call(), want) for _ in range(50))
    made = logits.make(rng, 20, 50257, width=3000, biases=600, mask=0.9)
    made["bias_tokens"] %= 50
    x = torch.randn(20, 50257, device="cuda")
    want = logits.call(x, made)
    assert all(torch.equal(logits.call(x, made), want) for _ in range(20))
