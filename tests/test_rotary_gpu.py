"""The cache append that rotates positions on the way, against 64 bits."""
import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
from step_testutil import DT, F8, check_quantised, cu_of, ints, rotary_table, rotate

pytestmark = pytest.mark.gpu


def make(rng, lens, counts, hq, hkv, d, page, dtype, spare=2):
    need = [-(-(int(a) + int(n)) // page) for a, n in zip(lens, counts)]
    pages = sum(need) + spare
    order, at = rng.permutation(pages), 0
    tables = np.full((len(lens), max(1, max(need))), -1)
    for r, n in enumerate(need):
        tables[r, :n] = order[at: at + n]
        at += n
    codes = [rng.integers(0, 256, (pages, hkv, page, d), dtype=np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 0x7F) == 0x7F] = 0x11
    scales = [rng.uniform(0.2, 2.0, (pages, hkv)).astype(np.float32) / 448 for _ in range(2)]
    x = torch.as_tensor(rng.standard_normal((sum(counts), hq + 2 * hkv, d))).to(DT[dtype])
    return codes, scales, tables, x


def device(codes, scales, tables):
    return [torch.as_tensor(c).cuda().view(F8) for c in codes] + [torch.as_tensor(s).cuda() for s in scales] + [ints(tables)]


def places(lens, counts):
    return np.concatenate([np.arange(a, a + n) for a, n in zip(lens, counts)]).astype(np.int64)


def check_q(got, want, dtype):
    # rounded once from a value off by 2^-22 of itself; fp16 has steps of 2^-24 below 2^-14
    eps = torch.finfo(DT[dtype]).eps / 2
    assert (np.abs(got.double().cpu().numpy() - want) <= (eps + 2.0 ** -21) * np.abs(want) + 2.0 ** -25).all()


def check(lens, counts, hq, hkv, d, page, rot, inter, dtype, cu=True, positions=None, far=0, in_place=False, seed=0, tables=None):
    rng = np.random.default_rng(seed)
    codes, scales, tab, x = make(rng, lens, counts, hq, hkv, d, page, dtype)
    if tables is not None:
        tab = tables(tab)
    at = places(lens, counts) if positions is None else np.asarray(positions)
    rows = rotary_table(int(at.max(initial=0)) + 1 if not far else 64, rot, far)
    dev = device(codes, scales, tab)
    fused = x.cuda()
    q, k, v = fused.split([hq, hkv, hkv], 1)  # strided views of one projection
    out = K.kda_kvcache_append_rotary(q, k, v, torch.as_tensor(rows).cuda(), *dev, ints(lens), cu_tokens=cu_of(counts) if cu else None,
                                      positions=None if positions is None else ints(positions), interleaved=inter, out=q if in_place else None)
    assert out.dtype == q.dtype and (out.data_ptr() == q.data_ptr()) == (in_place or q.numel() == 0)
    y = [rotate(t.double().numpy(), rows[at], inter) for t in x.split([hq, hkv, hkv], 1)[:2]] + [x[:, hq + hkv:].double().numpy()]
    check_q(out, y[0], dtype)
    assert torch.equal(fused[:, hq:].cpu(), x[:, hq:])
    for i in range(2):
        check_quantised(y[1 + i], codes[i], dev[i].view(torch.uint8).cpu().numpy(), scales[i], dev[2 + i].cpu().numpy(), tab, lens, counts, page)


@pytest.mark.parametrize("hq,hkv,d,page,rot", [(1, 1, 128, 16, 128), (8, 1, 64, 32, 64), (12, 3, 128, 64, 64), (7, 7, 64, 128, 16), (33, 2, 128, 16, 96)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_token(hq, hkv, d, page, rot, inter, dtype):
    lens = [0, 1, 15, 16, 17, 127, 128, 129, 300]
    check(lens, [1] * len(lens), hq, hkv, d, page, rot, inter, dtype, cu=False, seed=hq, in_place=inter)


@pytest.mark.parametrize("hq,hkv,d,page,rot,inter", [(4, 4, 128, 16, 128, False), (6, 2, 64, 64, 48, True), (17, 1, 128, 128, 32, False), (5, 1, 64, 128, 64, True),
                                                     (9, 3, 128, 32, 128, True), (40, 2, 64, 16, 64, False), (16, 2, 128, 64, 128, False), (3, 1, 64, 32, 32, False)])
@pytest.mark.parametrize("in_place", [False, True])
def test_several_tokens(hq, hkv, d, page, rot, inter, in_place):
    lens, counts = [9, 0, 500, 40, 333, 0, 64, 128], [0, 3, 1, 140, 70, 300, 64, 0]
    check(lens, counts, hq, hkv, d, page, rot, inter, "bf16" if page > 32 else "fp16", in_place=in_place, seed=page + d)


def test_given_and_far_positions():
    check([3, 5], [7, 1], 2, 1, 64, 16, 64, False, "bf16", positions=[5, 0, 0, 40, 9, 9, 63, 1])
    check([3, 5, 0], [1, 1, 1], 2, 1, 128, 16, 128, True, "fp16", cu=False, positions=[63, 7, 0], far=10 ** 6)
    check([1000], [60], 2, 1, 128, 64, 128, False, "bf16", positions=list(range(60)), far=2 ** 24 - 30)


def test_many_rows():
    rng = np.random.default_rng(1)
    counts = [int(n) for n in rng.integers(0, 4, 700)]
    check([int(n) for n in rng.integers(0, 40, 700)], counts, 2, 1, 64, 16, 64, False, "bf16")


@pytest.mark.parametrize("n", [1, 45])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_angles_of_zero_give_the_append(n, dtype):
    rng = np.random.default_rng(n)
    lens, counts = [0, 7, 30], [n] * 3
    codes, scales, tab, x = make(rng, lens, counts, 3, 2, 128, 32, dtype)
    one = torch.cat([torch.ones(128, 32), torch.zeros(128, 32)], 1).cuda()
    a, b = device(codes, scales, tab), device(codes, scales, tab)
    q, k, v = x.cuda().split([3, 2, 2], 1)
    cu = cu_of(counts) if n > 1 else None
    out = K.kda_kvcache_append_rotary(q, k, v, one, *a, ints(lens), cu_tokens=cu)
    K.kda_kvcache_append(k, v, *b, ints(lens), cu_tokens=cu)
    assert torch.equal(out, q)
    for s, t in zip(a, b):
        assert torch.equal(s.view(torch.uint8) if s.dtype == F8 else s, t.view(torch.uint8) if t.dtype == F8 else t)


@pytest.mark.parametrize("n", [1, 20])
def test_positions_outside_of_the_table_and_missing_pages(n):
    rng = np.random.default_rng(5)
    lens, counts = [10, 30, 3], [n] * 3
    codes, scales, tab, x = make(rng, lens, counts, 2, 1, 64, 16, "bf16")
    where = places(lens, counts).reshape(3, n)
    where[0, 0], where[1, -1] = -1, 64
    rows = rotary_table(64, 64)
    dev = device(codes, scales, tab)
    q, k, v = x.cuda().split([2, 1, 1], 1)
    K.kda_get_device_status()
    cu = cu_of(counts) if n > 1 else None
    out = K.kda_kvcache_append_rotary(q, k, v, torch.as_tensor(rows).cuda(), *dev, ints(lens), cu_tokens=cu, positions=ints(where.reshape(-1)))
    assert K.kda_get_device_status() == 1
    turned = np.concatenate([rows, np.concatenate([np.ones((1, 32)), np.zeros((1, 32))], 1).astype(np.float32)])
    at = np.where((where < 0) | (where >= 64), 64, where).reshape(-1)
    y = [rotate(t.double().numpy(), turned[at], False) for t in x.split([2, 1, 1], 1)[:2]]
    check_q(out, y[0], "bf16")
    check_quantised(y[1], codes[0], dev[0].view(torch.uint8).cpu().numpy(), scales[0], dev[2].cpu().numpy(), tab, lens, counts, 16)
    # a page that is not there: its tokens are dropped, their queries turned all the same
    tab[1] = -1
    tab[2, 0] = codes[0].shape[0]
    dev = device(codes, scales, tab)
    out = K.kda_kvcache_append_rotary(q, k, v, torch.as_tensor(rows).cuda(), *dev, ints(lens), cu_tokens=cu)
    assert K.kda_get_device_status() == 1
    at = places(lens, counts)
    y = [rotate(t.double().numpy(), rows[at], False) for t in x.split([2, 1, 1], 1)[:2]]
    check_q(out, y[0], "bf16")
    check_quantised(y[1], codes[0], dev[0].view(torch.uint8).cpu().numpy(), scales[0], dev[2].cpu().numpy(), tab, lens, counts, 16)


@pytest.mark.parametrize("n", [1, 20])
def test_values_that_are_not_finite(n):
    rng = np.random.default_rng(6)
    lens, counts = [0, 5], [n] * 2
    codes, scales, tab, x = make(rng, lens, counts, 1, 2, 64, 16, "fp16")
    x[0, 1, 3], x[n, 2, 63], x[1, 4, 0] = float("inf"), float("nan"), float("-inf")
    rows = rotary_table(40, 64)
    dev = device(codes, scales, tab)
    q, k, v = x.cuda().split([1, 2, 2], 1)
    K.kda_get_device_status()
    K.kda_kvcache_append_rotary(q, k, v, torch.as_tensor(rows).cuda(), *dev, ints(lens), cu_tokens=cu_of(counts) if n > 1 else None)
    assert K.kda_get_device_status() == 9
    p = tab[0, 0]
    got = dev[0][p, 0, 0].float()  # token 0, head 0 of k: inf * 0 is NaN, stored as 0; inf cos 0 = inf as 448
    assert got[3] == 448 and got[35] == 0
    assert torch.isfinite(dev[0][p].float()).all() and torch.isfinite(dev[2][p]).all()
    keep = [i for i in range(64) if i not in (3, 35)]
    y = rotate(np.nan_to_num(x[:1, 1:3].double().numpy(), posinf=0), rows[:1], False)
    assert np.abs(got.cpu().numpy()[keep] * float(dev[2][p, 0]) - y[0, 0, keep]).max() <= 2.0 ** -4 * np.abs(y[0, 0]).max()


def test_no_tokens_streams_and_graphs():
    rng = np.random.default_rng(7)
    lens, counts = [3, 20, 0], [4, 1, 30]
    codes, scales, tab, x = make(rng, lens, counts, 4, 2, 128, 16, "bf16")
    rows = torch.as_tensor(rotary_table(64, 128)).cuda()
    args = lambda dev, t: (*t.split([4, 2, 2], 1), rows, *dev, ints(lens), cu_of(counts))  # noqa: E731
    want_dev, fused = device(codes, scales, tab), x.cuda()
    want = K.kda_kvcache_append_rotary(*args(want_dev, fused))
    empty = fused[:0]
    assert K.kda_kvcache_append_rotary(*empty.split([4, 2, 2], 1), rows, *device(codes, scales, tab), ints(lens), cu_of([0, 0, 0])).shape == (0, 4, 128)
    # a stream of its own
    dev, side = device(codes, scales, tab), torch.cuda.Stream()
    a = args(dev, fused)
    side.wait_stream(torch.cuda.current_stream())
    got = K.kda_kvcache_append_rotary(*a, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    # captured, replayed on other inputs
    dev, moved = device(codes, scales, tab), torch.zeros_like(fused)
    a = args(dev, moved)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = K.kda_kvcache_append_rotary(*a)
    for s, t in zip(dev, device(codes, scales, tab)):
        s.copy_(t)
    moved.copy_(fused)
    graph.replay()
    assert torch.equal(got, want)
    for s, t in zip(dev, want_dev):
        assert torch.equal(s.view(torch.uint8) if s.dtype == F8 else s, t.view(torch.uint8) if t.dtype == F8 else t)


def test_refusals():
    rng = np.random.default_rng(8)
    codes, scales, tab, x = make(rng, [0, 5], [1, 1], 2, 1, 64, 16, "bf16")
    dev, lens = device(codes, scales, tab), ints([0, 5])
    q, k, v = (t.contiguous() for t in x.cuda().split([2, 1, 1], 1))
    rows = torch.as_tensor(rotary_table(16, 64)).cuda()

    def refused(error, **over):
        a = dict(q=q, k=k, v=v, rotary=rows, out=None, positions=None)
        a.update(over)
        with pytest.raises(error):
            K.kda_kvcache_append_rotary(a["q"], a["k"], a["v"], a["rotary"], *dev, lens, positions=a["positions"], out=a["out"])

    refused(ValueError, q=q.half())
    refused(ValueError, q=q[:1])
    refused(ValueError, q=q[:, :, :32])
    refused(ValueError, k=k.float(), v=v.float())
    refused(ValueError, rotary=rows.double())
    refused(ValueError, rotary=rows[:, ::2])
    refused(ValueError, positions=torch.zeros(2, device="cuda"))
    refused(ValueError, positions=ints([0]))
    refused(ValueError, out=q.float())
    refused(K.KdaError, rotary=rows[:, :24].contiguous())
    refused(K.KdaError, rotary=torch.zeros(16, 80, device="cuda"))
    both = torch.zeros(2, 3, 64, device="cuda", dtype=torch.bfloat16)
    refused(K.KdaError, q=both[:, :2], out=both[:, 1:])          # overlaps q by a head
    refused(K.KdaError, k=both[:, :1], out=both[:, :2])          # overlaps k
    K.kda_kvcache_append_rotary(both[:, :2], both[:, 2:], v, rows, *dev, lens, out=both[:, :2])  # beside k: fine
