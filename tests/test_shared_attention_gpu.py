"""Attention over shared prefixes against 64 bits, and against the attention that shares nothing.

The bound is the one of tests/test_kvcache_gpu.py: twice the output's rounding plus 2^-10 sum_j p_j |v_j| for
weights that are rounded to fp16, plus 1e-6."""
import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
import serving_testutil as ref
from step_testutil import DT, F8, cu_of, ints

pytestmark = pytest.mark.gpu


def make_cache(rng, groups, page, hkv, d, spare=3, full=True):
    """groups: lists of (tokens in common with the group's first row, tokens in all), one for each row.  Pages of
    whole common tokens are shared, the others the row's own; what a page holds past a row's tokens is NaN where
    nobody else holds it.  full: tables of a width with which sharing can pay."""
    tables, lens = [], []
    pages = sum(-(-n // page) for g in groups for _, n in g) + spare
    order, at = rng.permutation(pages), 0
    kc, vc = (rng.integers(0, 256, (pages, hkv, page, d), dtype=np.uint8) for _ in range(2))
    for c in (kc, vc):
        c[(c & 0x7F) == 0x7F] = 0x11
    rows = sum(len(g) for g in groups)
    width = max([1] + [-(-n // page) for g in groups for _, n in g]) + (4_000_000 // page // max(1, rows - len(groups)) if full else 0)
    for g in groups:
        first = None
        for common, n in g:
            need, same = -(-n // page), min(common, n) // page if first is not None else 0
            t = np.full(width, -1)
            t[:same] = first[:same] if first is not None else 0
            t[same:need] = order[at: at + need - same]
            at += need - same
            if n % page and need > same:
                for c in (kc, vc):
                    c[t[need - 1], :, n % page:] |= 0x7F
            first = t if first is None else first
            tables.append(t)
            lens.append(n)
    ks, vs = (rng.uniform(0.2, 2.0, (pages, hkv)).astype(np.float32) / 448 for _ in range(2))
    return kc, vc, ks, vs, np.array(tables).reshape(-1, width), lens


def gpu_cache(kc, vc, ks, vs, tables):
    return (torch.as_tensor(kc).cuda().view(F8), torch.as_tensor(vc).cuda().view(F8), torch.as_tensor(ks).cuda(), torch.as_tensor(vs).cuda(), ints(tables))


def check(rng, groups, counts, hq, hkv, d, page, dtype, cu=True, q_scale=1.0, change=None, cu_rows=None, status=0, exact=True, full=True):
    kc, vc, ks, vs, tables, lens = make_cache(rng, groups, page, hkv, d, full=full)
    if change:
        change(kc, vc, ks, vs, tables)
    q = torch.as_tensor(rng.standard_normal((sum(counts), hq, d)) * q_scale).to(DT[dtype])
    scale = d ** -0.5
    rows = cu_of([len(g) for g in groups]) if cu_rows is None else ints(cu_rows)
    K.kda_get_device_status()
    got = K.kda_kvcache_attention_shared(q.cuda(), *gpu_cache(kc, vc, ks, vs, tables), ints(lens), rows, cu_tokens=cu_of(counts) if cu else None, scale=scale)
    assert K.kda_get_device_status() == status
    assert got.dtype == q.dtype and torch.isfinite(got).all()
    got = got.double().cpu().numpy()
    eps = torch.finfo(DT[dtype]).eps
    if exact:
        want, weight = ref.attention(q.double().numpy(), kc, vc, ks, vs, tables, lens, counts, page, scale)
        allowed = eps * np.abs(want) + 2.0 ** -10 * weight + 1e-6
        assert (np.abs(got - want) <= allowed).all(), np.max(np.abs(got - want) / allowed)
    else:  # the other entry, within both roundings of either
        other = K.kda_kvcache_attention(q.cuda(), *gpu_cache(kc, vc, ks, vs, tables), ints(lens), cu_tokens=cu_of(counts) if cu else None, scale=scale)
        other = other.double().cpu().numpy()
        allowed = 2 * eps * np.abs(other) + 2.0 ** -9
        assert (np.abs(got - other) <= allowed).all(), np.max(np.abs(got - other) / allowed)


BEAMS = [[(0, 700), (600, 650), (600, 640), (600, 777)], [(0, 130), (128, 129)], [(0, 40)], [(0, 300), (200, 260), (299, 300)], [], [(0, 257), (256, 257)]]


@pytest.mark.parametrize("hq,hkv,d,page", [(1, 1, 128, 16), (8, 1, 64, 32), (12, 3, 128, 64), (7, 1, 128, 128), (32, 2, 64, 16), (40, 1, 128, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_token(hq, hkv, d, page, dtype):
    check(np.random.default_rng(hq * 1000 + d + page), BEAMS, [1] * 12, hq, hkv, d, page, dtype, cu=False)


@pytest.mark.parametrize("hq,hkv,d,page", [(4, 4, 128, 16), (6, 2, 64, 64), (16, 1, 128, 32), (5, 1, 64, 128)])
def test_several_tokens(hq, hkv, d, page):
    counts = [3, 1, 7, 40, 1, 1, 40, 2, 0, 6, 1, 1]
    check(np.random.default_rng(hq + d + page), BEAMS, counts, hq, hkv, d, page, "bf16")


@pytest.mark.parametrize("d,page,group,dtype", [(128, 16, 8, "bf16"), (128, 128, 5, "fp16"), (64, 32, 8, "bf16"), (64, 64, 7, "fp16")])
def test_pieces_of_prompts_behind_a_prefix(d, page, group, dtype):
    # rows of more query rows than the kernel for few of them takes
    groups = [[(0, 900), (512, 700), (512, 613)] + [(512, 600)] * 9, [(0, 300), (128, 333)]]
    check(np.random.default_rng(d + page), groups, [9, 7, 50, 1, 3, 60, 1, 0, 1, 1, 1, 2, 9, 12], 2 * group, 2, d, page, dtype)


@pytest.mark.parametrize("rows,hq,hkv,d,shared,page", [(2, 20, 1, 128, 128, 128), (3, 2, 1, 128, 128, 128), (33, 8, 1, 64, 640, 16), (70, 16, 2, 128, 384, 64), (300, 4, 1, 64, 256, 32)])
def test_large_groups(rows, hq, hkv, d, shared, page):
    rng = np.random.default_rng(rows)
    group = [(0, shared + 20)] + [(shared, shared + int(n)) for n in rng.integers(1, 60, rows - 1)]
    check(rng, [group], [1] * rows, hq, hkv, d, page, "bf16", cu=False)


@pytest.mark.parametrize("d", [64, 128])
def test_long_prefixes_and_many_groups(d):
    rng = np.random.default_rng(d)
    check(rng, [[(0, 20011)] + [(20000, 20000 + i) for i in range(1, 6)]], [1] * 6, 16, 2, d, 64, "bf16", cu=False, exact=False)
    groups = [[(0, int(n))] + [(int(n) - 5, int(n) + i) for i in range(int(k))] for n, k in zip(rng.integers(6, 1500, 200), rng.integers(0, 5, 200))]
    check(rng, groups, [1] * sum(len(g) for g in groups), 8, 2, d, 32, "fp16", cu=False, exact=False)
    counts = [int(n) for n in rng.integers(0, 6, sum(len(g) for g in groups))]
    groups = [[(a, n + 6) for a, n in g] for g in groups]
    check(rng, groups, counts, 8, 2, d, 32, "fp16", exact=False)


def test_group_sizes_past_the_kernels_lists():
    rng = np.random.default_rng(1)
    groups = [[(0, 140), (128, 131), (128, 129)] for _ in range(1200)]
    check(rng, groups, [1] * 3600, 2, 1, 64, 16, "bf16", cu=False, exact=False)


def test_rows_without_tokens_do_not_limit_the_prefix():
    # an ended beam: no tokens, no pages
    groups = [[(0, 400), (0, 0), (390, 395), (390, 399)], [(0, 0), (0, 300), (0, 10)]]
    check(np.random.default_rng(2), groups, [1, 0, 1, 2, 0, 1, 0], 8, 2, 128, 16, "bf16")


def test_pages_that_differ_or_are_missing():
    def differ(kc, vc, ks, vs, tables):
        tables[2, 9] = tables[0, 20]        # a row's own page among the shared ones
    check(np.random.default_rng(3), BEAMS, [1] * 12, 8, 2, 64, 16, "bf16", cu=False, change=differ)

    def missing(kc, vc, ks, vs, tables):
        tables[:4, 3] = -1                  # of the prefix, in all rows
        tables[:4, 8] = kc.shape[0]
        tables[3, 45] = -1
    check(np.random.default_rng(4), BEAMS, [1] * 12, 8, 2, 64, 16, "bf16", cu=False, change=missing, status=1)

    def all_missing(kc, vc, ks, vs, tables):
        tables[:4, : 512 // 16] = -1
    check(np.random.default_rng(5), BEAMS, [1] * 12, 8, 2, 128, 16, "fp16", cu=False, change=all_missing, status=1)


@pytest.mark.parametrize("counts", [[1] * 4, [60] * 4])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_and_scores_far_apart(d, counts):
    # weights times v scales that leave fp16's normal range are off by up to 2^-25 of the row's largest one: scales over
    # twelve orders of magnitude, in the prefix and behind it
    rng = np.random.default_rng(d)
    groups = [[(0, 700), (640, 690), (640, 720), (640, 710)]]
    kc, vc, ks, vs, tables, lens = make_cache(rng, groups, 16, 2, d)
    ks *= rng.uniform(0, 3, ks.shape).astype(np.float32)
    vs *= (10.0 ** rng.integers(-6, 6, vs.shape)).astype(np.float32)
    vs[tables[0, 0]] = vs[tables[1, 42]] = 0
    ks[tables[1, 3]] = 0
    n, hq = counts[0], 16
    q = torch.as_tensor(rng.standard_normal((sum(counts), hq, d)) * 3).to(torch.bfloat16)
    want, weight = ref.attention(q.double().numpy(), kc, vc, ks, vs, tables, lens, counts, 16, 0.125)
    got = K.kda_kvcache_attention_shared(q.cuda(), *gpu_cache(kc, vc, ks, vs, tables), ints(lens), ints([0, 4]), cu_tokens=cu_of(counts),
                                         scale=0.125).double().cpu().numpy()
    below = np.zeros_like(want)
    for r in range(4):
        ids = tables[r, : -(-lens[r] // 16)]
        k, v = (np.nan_to_num(ref.E4M3[c[ids]]).transpose(1, 0, 2, 3).reshape(2, -1, d)[:, : lens[r]] for c in (kc, vc))
        sk, sv = (np.repeat(x[ids].T.astype(np.float64), 16, 1)[:, : lens[r]] for x in (ks, vs))
        for i in range(n):
            p = lens[r] - n + i + 1
            for h in range(hq):
                g = h * 2 // hq
                z = 0.125 * (k[g, :p] @ q[r * n + i, h].double().numpy()) * sk[g, :p]
                w = np.exp(z - z.max())
                below[r * n + i, h] = 2.0 ** -25 * (w * sv[g, :p]).max() / w.sum() * np.abs(v[g, :p]).sum(0)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * weight + below + 1e-6).all()


def test_queries_of_all_sizes():
    rng = np.random.default_rng(6)
    kc, vc, ks, vs, tables, lens = make_cache(rng, [[(0, 300), (256, 280), (256, 299)]], 64, 1, 64)
    q = torch.as_tensor(rng.standard_normal((3, 4, 64)))
    q[0] *= 1e30
    q[1] *= 1e-30
    q[2, 1] = 0
    q = q.to(torch.bfloat16)
    for s in (1e-30, 0.0, 1.0, -1.0):
        some = slice(0, 3) if abs(s) < 1 else slice(1, 3)
        want, weight = ref.attention(q.double().numpy()[some], kc, vc, ks, vs, tables[some], lens[some], [1] * len(lens[some]), 64, s)
        got = K.kda_kvcache_attention_shared(q.cuda(), *gpu_cache(kc, vc, ks, vs, tables), ints(lens), ints([0, 3]), scale=s).double().cpu().numpy()[some]
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * weight + 1e-6).all()


@pytest.mark.parametrize("cu_rows", [[1, 12], [0, 11], [0, 5, 4, 12], [0, -3, 12], [0, 13, 12], [0, 4, 40]])
def test_malformed_groups_share_nothing(cu_rows):
    check(np.random.default_rng(7), BEAMS, [1] * 12, 8, 2, 64, 32, "bf16", cu=False, cu_rows=cu_rows, status=1)
    check(np.random.default_rng(7), BEAMS, [1] * 12, 8, 2, 64, 32, "bf16", cu=False, cu_rows=cu_rows, full=False)  # not read


@pytest.mark.parametrize("counts", [[1] * 12, [3, 1, 7, 4, 1, 1, 9, 2, 0, 6, 1, 1]])
def test_small_tables(counts):
    check(np.random.default_rng(11), BEAMS, counts, 16, 2, 64, 16, "bf16", full=False)


def test_any_groups_give_the_same():
    for cu_rows in ([0, 12], [0, 0, 2, 2, 12, 12], list(range(13)), [0, 3, 6, 9, 12]):
        check(np.random.default_rng(8), BEAMS, [1] * 12, 8, 2, 64, 32, "bf16", cu=False, cu_rows=cu_rows)


def test_strided_tensors_streams_and_graphs():
    rng = np.random.default_rng(9)
    kc, vc, ks, vs, tables, lens = make_cache(rng, BEAMS, 16, 2, 128)
    cache, ln, rows = gpu_cache(kc, vc, ks, vs, tables), ints(lens), cu_of([len(g) for g in BEAMS])
    fused = torch.randn(12, 12, 128, device="cuda").to(torch.bfloat16)
    q = fused[:, :8]
    want = K.kda_kvcache_attention_shared(q.contiguous(), *cache, ln, rows)
    wide = torch.zeros(12, 10, 128, device="cuda", dtype=torch.bfloat16)
    got = K.kda_kvcache_attention_shared(q, *cache, ln, rows, out=wide[:, 1:9])
    assert torch.equal(got, want) and (wide[:, 0] == 0).all() and (wide[:, 9] == 0).all()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = K.kda_kvcache_attention_shared(q, *cache, ln, rows, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    # two graphs that run at the same time on other inputs
    inputs, graphs, outs = [torch.zeros_like(want) for _ in range(2)], [], []
    for x in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(K.kda_kvcache_attention_shared(x, *cache, ln, rows))
        graphs.append(graph)
    inputs[0].copy_(q)
    inputs[1].copy_(-q)
    torch.cuda.synchronize()
    for _ in range(5):
        for graph in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    assert torch.equal(outs[1], K.kda_kvcache_attention_shared(-q, *cache, ln, rows))
    empty = K.kda_kvcache_attention_shared(q[:0].contiguous(), *cache, ln, rows, cu_tokens=ints([0] * 13))
    assert empty.shape == (0, 8, 128)


def test_refusals():
    rng = np.random.default_rng(10)
    kc, vc, ks, vs, tables, lens = make_cache(rng, [[(0, 40), (30, 35)]], 16, 1, 64)
    cache, ln, rows = gpu_cache(kc, vc, ks, vs, tables), ints(lens), ints([0, 2])
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    for bad in (dict(cu_rows=rows.long()), dict(cu_rows=rows.cpu()), dict(cu_rows=rows.view(1, 2)), dict(cu_rows=rows[:0]), dict(q=q.float()), dict(q=q[:, :, :32])):
        a = dict(q=q, cu_rows=rows)
        a.update(bad)
        with pytest.raises(ValueError):
            K.kda_kvcache_attention_shared(a["q"], *cache, ln, a["cu_rows"])
    for bad in (dict(cu_rows=rows[:1]), dict(q=q[:1])):
        a = dict(q=q, cu_rows=rows)
        a.update(bad)
        with pytest.raises(K.KdaError):
            K.kda_kvcache_attention_shared(a["q"], *cache, ln, a["cu_rows"])
