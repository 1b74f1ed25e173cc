"""The 8-bit paged cache: append bit for bit, attention against 64 bits.

Attention's bound, from its roundings: the softmax weights are fp16 (relative 2^-11, and
2^-25 of the largest weight where they leave fp16's normal range) on the weighted sum of |v|,
scores carry fp32 errors of a few 2^-23 of their size (below 64 here: 2^-15 of the weights),
the output is rounded once (2^-9 for bf16, 2^-12 for fp16, of its own size).  Allowed: twice
the output's rounding plus 2^-10 sum_j p_j |v_j| plus 1e-6."""
import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
import serving_testutil as ref

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def make_cache(rng, rows, hkv, page, d, lens, spare=2):
    """Random codes everywhere (NaN codes included past the rows' tokens), tables in random order."""
    need = [-(-int(n) // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    tables = np.full((rows, max(1, max(need, default=1))), -1)
    at = 0
    kc, vc = (rng.integers(0, 256, (pages, hkv, page, d), dtype=np.uint8) for _ in range(2))
    for r in range(rows):
        tables[r, : need[r]] = order[at: at + need[r]]
        at += need[r]
        for i in range(need[r]):
            m = min(page, int(lens[r]) - i * page)
            for c in (kc, vc):
                x = c[tables[r, i], :, :m]
                x[(x & 0x7F) == 0x7F] = 0x11
                c[tables[r, i], :, m:] |= 0x7F  # NaN where no token is
    ks, vs = (rng.uniform(0.2, 2.0, (pages, hkv)).astype(np.float32) / 448 for _ in range(2))
    return kc, vc, ks, vs, tables


def gpu_cache(kc, vc, ks, vs, tables):
    return (torch.as_tensor(kc).cuda().view(F8), torch.as_tensor(vc).cuda().view(F8), torch.as_tensor(ks).cuda(),
            torch.as_tensor(vs).cuda(), torch.as_tensor(tables).to(torch.int32).cuda())


def cu_of(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def check_attention(rng, rows, hq, hkv, d, page, lens, counts, dtype, cu=True, q_scale=1.0, scale=None, q=None, tables=None):
    kc, vc, ks, vs, tab = make_cache(rng, rows, hkv, page, d, lens)
    if tables is not None:
        tab = tables(tab)
    if q is None:
        q = torch.as_tensor(rng.standard_normal((sum(counts), hq, d)) * q_scale).to(DT[dtype])
    scale = d ** -0.5 if scale is None else scale
    want, weight = ref.attention(q.double().numpy(), kc, vc, ks, vs, tab, lens, counts, page, scale)
    got = K.kda_kvcache_attention(q.cuda(), *gpu_cache(kc, vc, ks, vs, tab), torch.as_tensor(lens).to(torch.int32).cuda(),
                                  cu_tokens=cu_of(counts) if cu else None, scale=scale)
    assert got.dtype == q.dtype
    got = got.double().cpu().numpy()
    eps = 2.0 ** (-8 if dtype == "bf16" else -11)
    allowed = eps * np.abs(want) + 2.0 ** -10 * weight + 1e-6
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= allowed).all(), np.max(np.abs(got - want) / allowed)


@pytest.mark.parametrize("hq,hkv,d,page", [(1, 1, 128, 16), (8, 1, 64, 32), (12, 3, 128, 64), (7, 1, 128, 128), (32, 2, 64, 16), (40, 1, 128, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_token(hq, hkv, d, page, dtype):
    rng = np.random.default_rng(hq * 1000 + d + page)
    lens = [0, 1, 15, 16, 17, 127, 128, 129, 300, 1000]
    check_attention(rng, len(lens), hq, hkv, d, page, lens, [1] * len(lens), dtype, cu=False)


@pytest.mark.parametrize("hq,hkv,d,page", [(4, 4, 128, 16), (6, 2, 64, 64), (16, 1, 128, 32), (5, 1, 64, 128)])
def test_several_tokens(hq, hkv, d, page):
    rng = np.random.default_rng(hq + d + page)
    counts = [0, 3, 1, 40, 70, 5, 0]
    lens = [9, 3, 500, 40, 333, 2, 0]  # all new, mostly old, more new tokens than cached ones
    check_attention(rng, len(lens), hq, hkv, d, page, lens, counts, "bf16")


@pytest.mark.parametrize("d,page", [(128, 64), (64, 16)])
def test_many_tokens_equal_single_tokens(d, page):
    # the kernel for many tokens against the one for single tokens, which the tests above hold to
    # 64 bits: several items and hundreds of tiles for every block
    rng = np.random.default_rng(d)
    rows, n, hq, hkv = 16, 24, 32, 4
    lens = rng.integers(n, 3000, rows)
    cache = gpu_cache(*make_cache(rng, rows, hkv, page, d, lens))
    ln = torch.as_tensor(lens).to(torch.int32).cuda()
    g = torch.Generator(device="cuda").manual_seed(d)
    K.kda_get_device_status()
    for _ in range(5):
        q = torch.randn(rows, n, hq, d, generator=g, device="cuda").to(torch.bfloat16)
        many = K.kda_kvcache_attention(q.view(rows * n, hq, d), *cache, ln, cu_tokens=cu_of([n] * rows)).view(rows, n, hq, d)
        for i in range(n):
            one = K.kda_kvcache_attention(q[:, i], *cache, ln - n + i + 1)
            # both round to bf16 once (2^-8 between neighbours) and their weights to fp16
            assert ((many[:, i].float() - one.float()).abs() <= 2.0 ** -7 * one.float().abs() + 2.0 ** -9).all()
    assert K.kda_get_device_status() == 0


@pytest.mark.parametrize("d,page,group,dtype", [(128, 16, 8, "bf16"), (128, 128, 5, "fp16"), (64, 32, 8, "bf16"), (64, 64, 7, "fp16")])
@pytest.mark.parametrize("missing", [False, True])
def test_pieces_of_prompts(d, page, group, dtype, missing):
    # large enough for the kernel of 128 query rows an item
    rng = np.random.default_rng(d + page)
    counts, lens = [200, 0, 301, 1, 77], [200, 40, 700, 900, 78]

    def drop(tab):
        tab = tab.copy()
        tab[2, 1] = tab[2, 300 // page] = tab[0, 0] = tab[3, 800 // page] = -1
        return tab

    K.kda_get_device_status()
    check_attention(rng, 5, 4 * group, 4, d, page, lens, counts, dtype, tables=drop if missing else None)
    assert K.kda_get_device_status() == (1 if missing else 0)


@pytest.mark.parametrize("d,hq", [(64, 16), (128, 24)])
@pytest.mark.parametrize("n", [1, 300])
def test_scales_and_scores_far_apart(d, hq, n):
    # references of the weights that grow along the keys: rows' maxima by far more than 2^8, v's scales
    # by orders of magnitude, scales of zero; for single tokens and for pieces of prompts.  A weight p vs
    # that leaves fp16's normal range is off by up to 2^-25 of the row's largest one.
    rng = np.random.default_rng(1000 * n + d)
    counts, lens = [n, n], [640, 999]
    kc, vc, ks, vs, tab = make_cache(rng, 2, 4, 16, d, lens)
    ks *= rng.uniform(0, 3, ks.shape).astype(np.float32)
    vs *= (10.0 ** rng.integers(-6, 6, vs.shape)).astype(np.float32)
    vs[tab[0, 0]] = vs[tab[1, 50]] = 0
    ks[tab[1, 3]] = 0
    q = torch.as_tensor(rng.standard_normal((2 * n, hq, d)) * 3).to(torch.bfloat16)
    want, weight = ref.attention(q.double().numpy(), kc, vc, ks, vs, tab, lens, counts, 16, 0.125)
    got = K.kda_kvcache_attention(q.cuda(), *gpu_cache(kc, vc, ks, vs, tab), torch.tensor(lens, dtype=torch.int32).cuda(),
                                  cu_tokens=cu_of(counts), scale=0.125).double().cpu().numpy()
    below = np.zeros_like(want)
    for r in range(2):
        ids = tab[r, : -(-lens[r] // 16)]
        k, v = (ref.E4M3[c[ids]].transpose(1, 0, 2, 3).reshape(4, -1, d)[:, : lens[r]] for c in (kc, vc))
        sk, sv = (np.repeat(x[ids].T.astype(np.float64), 16, 1)[:, : lens[r]] for x in (ks, vs))
        for i in range(n):
            p = lens[r] - n + i + 1
            for h in range(hq):
                g = h * 4 // hq
                z = 0.125 * (k[g, :p] @ q[r * n + i, h].double().numpy()) * sk[g, :p]
                w = np.exp(z - z.max())
                below[r * n + i, h] = 2.0 ** -25 * (w * sv[g, :p]).max() / w.sum() * np.abs(v[g, :p]).sum(0)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * weight + below + 1e-6).all()


def test_one_long_row_is_split():
    rng = np.random.default_rng(3)
    check_attention(rng, 2, 8, 1, 128, 64, [20000, 1], [1, 1], "fp16", cu=False)


@pytest.mark.parametrize("rows,hkv,group,d,n,length", [
    (1, 1, 3, 128, 34, 5670),  # one item of many parts, and more of fewer
    (2, 2, 7, 64, 7, 9000), (6, 3, 5, 128, 8, 3001), (12, 4, 4, 64, 20, 1945), (3, 8, 16, 64, 9, 700),
    (1, 1, 5, 64, 1, 40001), (1, 1, 12, 128, 1, 20001), (5, 8, 2, 128, 2, 3333), (9, 8, 1, 64, 1, 2500)])
def test_few_items_of_many_parts(rows, hkv, group, d, n, length):
    rng = np.random.default_rng(length)
    lens = [length - 7 * i for i in range(rows)]
    check_attention(rng, rows, hkv * group, hkv, d, 32, lens, [n] * rows, "fp16", cu=n > 1)


@pytest.mark.parametrize("counts", [[20] * 700, [1] * 1500, [600] + [3] * 20 + [0, 150, 900], [2, 1100, 0, 70]])
def test_many_rows_and_rows_of_many_blocks(counts):
    rng = np.random.default_rng(len(counts))
    lens = [n + int(rng.integers(0, 40)) for n in counts]
    check_attention(rng, len(lens), 2, 1, 64, 16, lens, counts, "bf16")


def test_large_scores_and_extreme_queries():
    rng = np.random.default_rng(4)
    q = torch.as_tensor(rng.standard_normal((3, 4, 64)))
    q[0] *= 1e30  # beyond fp16
    q[1] *= 1e-30
    q[2] = 0
    q = q.to(torch.bfloat16)
    kc, vc, ks, vs, tab = make_cache(rng, 3, 2, 16, 64, [40, 40, 40])
    for r, s in ((0, 1e-30), (1, 1e30), (2, 1.0)):
        one = slice(r, r + 1)
        want, weight = ref.attention(q[one].double().numpy(), kc, vc, ks, vs, tab[one], [40], [1], 16, s)
        got = K.kda_kvcache_attention(q[one].cuda(), *gpu_cache(kc, vc, ks, vs, tab[one]), torch.tensor([40], dtype=torch.int32).cuda(), scale=s)
        got = got.double().cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * weight + 1e-6).all()


def test_scales_that_differ_by_orders_of_magnitude():
    rng = np.random.default_rng(6)
    lens = [200]
    kc, vc, ks, vs, tab = make_cache(rng, 1, 1, 16, 64, lens)
    vs *= (10.0 ** rng.integers(-6, 6, vs.shape)).astype(np.float32)
    vs[tab[0, 0]] = 0
    q = torch.as_tensor(rng.standard_normal((1, 4, 64))).to(torch.bfloat16)
    want, weight = ref.attention(q.double().numpy(), kc, vc, ks, vs, tab, lens, [1], 16, 0.125)
    got = K.kda_kvcache_attention(q.cuda(), *gpu_cache(kc, vc, ks, vs, tab), torch.tensor(lens, dtype=torch.int32).cuda()).double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * weight + 1e-6).all()


def test_missing_pages_are_skipped_and_recorded():
    rng = np.random.default_rng(7)
    K.kda_get_device_status()

    def broken(t):
        t = t.copy()
        t[0, 1], t[1, 0] = -1, 10 ** 6
        return t

    check_attention(rng, 2, 4, 2, 128, 16, [100, 16], [1, 1], "bf16", cu=False, tables=broken)
    assert K.kda_get_device_status() == 1


def test_lengths_past_the_table_are_recorded():
    rng = np.random.default_rng(8)
    kc, vc, ks, vs, tab = make_cache(rng, 2, 1, 16, 64, [32, 32])
    q = torch.randn(2, 1, 64, device="cuda", dtype=torch.bfloat16)
    cache = gpu_cache(kc, vc, ks, vs, tab)
    K.kda_get_device_status()
    a = K.kda_kvcache_attention(q, *cache, torch.tensor([33, -5], dtype=torch.int32, device="cuda"))
    assert K.kda_get_device_status() == 1
    b = K.kda_kvcache_attention(q, *cache, torch.tensor([32, 0], dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b) and (b[1] == 0).all() and K.kda_get_device_status() == 0


def test_strided_queries_and_outputs_and_reruns():
    rng = np.random.default_rng(9)
    lens = [77, 3000, 12]
    cache = gpu_cache(*make_cache(rng, 3, 2, 32, 128, lens))
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    wide = torch.randn(3, 3, 8, 128, device="cuda", dtype=torch.bfloat16)  # [tokens, qkv, heads, dim]
    q = wide[:, 1]
    plain = K.kda_kvcache_attention(q.contiguous(), *cache, ln)
    out = torch.zeros(3, 2, 8, 128, device="cuda", dtype=torch.bfloat16)
    K.kda_kvcache_attention(q, *cache, ln, out=out[:, 0])
    assert torch.equal(out[:, 0], plain) and (out[:, 1] == 0).all()
    for _ in range(3):
        assert torch.equal(K.kda_kvcache_attention(q, *cache, ln), plain)


def test_malformed_offsets_are_recorded():
    rng = np.random.default_rng(10)
    cache = gpu_cache(*make_cache(rng, 2, 1, 16, 64, [40, 40]))
    ln = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    q = torch.randn(4, 1, 64, device="cuda", dtype=torch.bfloat16)
    K.kda_get_device_status()
    for bad in ([0, 5, 4], [1, 2, 4], [0, 2, 3], [0, -3, 4]):
        K.kda_kvcache_attention(q, *cache, ln, cu_tokens=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert K.kda_get_device_status() == 1, bad
        K.kda_kvcache_append(q, q, *cache, ln - 8, cu_tokens=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert K.kda_get_device_status() == 1, bad


def test_offsets_past_32_bits():
    # 2^25 key blocks of 128 bytes and more: the last pages lie past 2^32 bytes of codes
    pages, d, page = 40000, 128, 128
    codes = torch.zeros(pages, 8, page, d, dtype=torch.uint8, device="cuda")  # 5.2 GB
    scale = torch.ones(pages, 8, device="cuda")
    rng = np.random.default_rng(11)
    kc, vc, ks, vs, _ = make_cache(rng, 1, 8, page, d, [page], spare=0)
    codes[-1] = torch.as_tensor(vc[0]).cuda()
    q = torch.as_tensor(rng.standard_normal((1, 8, d))).to(torch.bfloat16)
    tab = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    ln = torch.tensor([page], dtype=torch.int32, device="cuda")
    got = K.kda_kvcache_attention(q.cuda(), codes.view(F8), codes.view(F8), scale, scale, tab, ln)
    one = codes[-1:].contiguous()
    near = K.kda_kvcache_attention(q.cuda(), one.view(F8), one.view(F8), scale[:1].contiguous(), scale[:1].contiguous(), torch.zeros_like(tab), ln)
    assert torch.equal(got, near) and got.abs().max() > 0
    k = torch.randn(1, 8, d, device="cuda").to(torch.bfloat16)
    K.kda_kvcache_append(k, k, codes.view(F8), codes.view(F8).clone(), scale, scale.clone(), tab, ln - 1)
    K.kda_kvcache_append(k, k, one.view(F8), one.view(F8).clone(), torch.ones_like(scale[:1]), torch.ones_like(scale[:1]), torch.zeros_like(tab), ln - 1)
    assert torch.equal(codes[-1], one[0])


def check_append(rng, hkv, d, page, lens, counts, dtype, cu=True, spoil=None, strided=False):
    total = [a + b for a, b in zip(lens, counts)]
    kc, vc, ks, vs, tab = make_cache(rng, len(lens), hkv, page, d, total)
    for c in (kc, vc):
        c[(c & 0x7F) == 0x7F] = 0x11  # older tokens are finite
    xs = [torch.as_tensor(rng.standard_normal((sum(counts), hkv, d)) * s).to(DT[dtype]) for s in (1.0, 3.0)]
    if spoil:
        spoil(xs)
    dc = gpu_cache(kc, vc, ks, vs, tab)
    cu_t = cu_of(counts) if cu else None
    ln = torch.as_tensor(lens).to(torch.int32).cuda()
    if strided:
        wide = torch.zeros(sum(counts), 3, hkv, d, dtype=DT[dtype], device="cuda")
        wide[:, 0], wide[:, 2] = xs[0].cuda(), xs[1].cuda()
        K.kda_kvcache_append(wide[:, 0], wide[:, 2], *dc, ln, cu_tokens=cu_t)
    else:
        K.kda_kvcache_append(xs[0].cuda(), xs[1].cuda(), *dc, ln, cu_tokens=cu_t)
    for x, c, s, gc, gs in ((xs[0], kc, ks, dc[0], dc[2]), (xs[1], vc, vs, dc[1], dc[3])):
        ref.append(x.float().numpy(), c, s, tab, lens, counts, page)
        assert np.array_equal(gs.cpu().numpy(), s)
        assert np.array_equal(gc.view(torch.uint8).cpu().numpy(), c)


@pytest.mark.parametrize("hkv,d,page,dtype", [(1, 128, 16, "bf16"), (3, 64, 32, "fp16"), (8, 128, 64, "bf16"), (2, 64, 128, "bf16"), (5, 128, 128, "fp16")])
def test_append(hkv, d, page, dtype):
    rng = np.random.default_rng(hkv * page)
    K.kda_get_device_status()
    check_append(rng, hkv, d, page, [0, 1, page - 1, page, 5 * page + 3, 40, 7], [1] * 7, dtype, cu=False)
    check_append(rng, hkv, d, page, [0, 1, page - 1, page, 5 * page + 3, 40, 7], [0, 1, 2, page, 3 * page + 1, 2 * page - 1, 0], dtype)
    check_append(rng, hkv, d, page, [3, 0], [300, 1], dtype, strided=True)
    assert K.kda_get_device_status() == 0


def test_append_many_rows():
    rng = np.random.default_rng(12)
    rows = 300
    check_append(rng, 1, 64, 16, rng.integers(0, 40, rows).tolist(), rng.integers(0, 40, rows).tolist(), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_of_blocks_of_every_size(dtype):
    # largest magnitudes from the type's least to its greatest values, quotients at and around
    # the codes' rounding boundaries, divisors whose fraction is all ones
    g = torch.Generator().manual_seed(1)
    blocks, hkv, page, d = 400, 2, 16, 64
    least, most = (-133, 127) if dtype == "bf16" else (-24, 15)
    size = torch.exp2(torch.linspace(least, most, blocks, dtype=torch.float64)).repeat_interleave(page)[:, None, None]
    x = torch.rand(blocks * page, hkv, d, generator=g, dtype=torch.float64) * 2 - 1
    x[::3] = torch.round(x[::3] * 240) / 240  # multiples of the largest value's simple fractions
    x[::page, :, 0] = 1
    x = (x * size).to(DT[dtype])
    tab = np.arange(blocks)[:, None]
    kc = np.zeros((blocks, hkv, page, d), np.uint8)
    ks = np.zeros((blocks, hkv), np.float32)
    cache = gpu_cache(kc, kc.copy(), ks, ks.copy(), tab)
    lens = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    K.kda_get_device_status()
    K.kda_kvcache_append(x.cuda(), x.cuda(), *cache, lens, cu_tokens=cu_of([page] * blocks))
    assert K.kda_get_device_status() == 0
    ref.append(x.float().numpy(), kc, ks, tab, [0] * blocks, [page] * blocks, page)
    assert np.array_equal(cache[2].cpu().numpy(), ks)
    assert np.array_equal(cache[0].view(torch.uint8).cpu().numpy(), kc)
    assert torch.equal(cache[0].view(torch.uint8), cache[1].view(torch.uint8))


@pytest.mark.parametrize("cu", [False, True])
def test_append_of_values_that_are_not_finite(cu):
    def spoil(xs):
        xs[0][0, 0, 3], xs[0][1, 1, 5], xs[1][2, 0, 0] = float("nan"), float("inf"), float("-inf")
        xs[1][1] = float("nan")
        xs[0][3] = 0

    rng = np.random.default_rng(13)
    K.kda_get_device_status()
    check_append(rng, 2, 64, 16, [4, 0, 16, 0], [1] * 4, "bf16", cu=cu, spoil=spoil)
    assert K.kda_get_device_status() == 9


def test_append_without_a_page_is_recorded():
    rng = np.random.default_rng(14)
    kc, vc, ks, vs, tab = make_cache(rng, 2, 1, 16, 64, [16, 16], spare=0)
    tab[0, 0] = -1
    cache = gpu_cache(kc, vc, ks, vs, tab)
    before = cache[0].view(torch.uint8).clone()
    x = torch.randn(2, 1, 64, device="cuda", dtype=torch.bfloat16)
    K.kda_get_device_status()
    for lens in ([3, 16], [3, -1]):  # no page; past the table; a negative length
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        K.kda_kvcache_append(x, x, *cache, ln)
        assert K.kda_get_device_status() == 1
        K.kda_kvcache_append(x, x, *cache, ln, cu_tokens=cu_of([1, 1]))
        assert K.kda_get_device_status() == 1
    assert torch.equal(cache[0].view(torch.uint8), before)


def test_append_then_attend_in_a_graph():
    rng = np.random.default_rng(15)
    lens = [30, 63, 0]
    kc, vc, ks, vs, tab = make_cache(rng, 3, 2, 32, 64, [n + 2 for n in lens])
    cache = gpu_cache(kc, vc, ks, vs, tab)
    k, v, q = (torch.randn(3, h, 64, device="cuda", dtype=torch.bfloat16) for h in (2, 2, 4))
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)

    def step():
        K.kda_kvcache_append(k, v, *cache, ln)
        K.kda_kvcache_attention(q, *cache, ln + 1, out=out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    for x in (k, v, q):
        x.copy_(torch.randn_like(x))
    g.replay()
    torch.cuda.synchronize()
    first = out.clone()
    step()
    assert torch.equal(out, first)


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("small,large", [(0, 2.0 ** 30), (0, 2.0 ** 110), (2.0 ** -70, 2.0 ** 60), (2.0 ** -20, 2.0 ** 110)])
@pytest.mark.parametrize("hq,d,n,length", [(4, 64, 1, 64), (16, 128, 1, 5000), (16, 64, 100, 128), (32, 128, 100, 3000)])
def test_scales_of_values_any_distance_apart(hq, d, n, length, small, large, order):
    # equal scores, half of the pages with a small or zero scale of v: those keep their half of the
    # weights.  Weights are fp16 and their pages' contributions no closer than 2^-90 of the largest
    # scale's (2^-80 here, of 448: far below the bound of the large ones).  Outputs of 448 * 2^110 are finite in bf16.
    rng = np.random.default_rng(length + d)
    kc, vc, ks, vs, tab = make_cache(rng, 1, 4, 16, d, [length])
    first = np.arange(tab.shape[1]) < tab.shape[1] // 2
    vs[tab[0]] = np.where(first == (order > 0), small, large).astype(np.float32)[:, None]
    q = torch.zeros(n, hq, d, dtype=torch.bfloat16)
    want, weight = ref.attention(q.double().numpy(), kc, vc, ks, vs, tab, [length], [n], 16, 0.125)
    got = K.kda_kvcache_attention(q.cuda(), *gpu_cache(kc, vc, ks, vs, tab), torch.tensor([length], dtype=torch.int32).cuda(),
                                  cu_tokens=cu_of([n]), scale=0.125).double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * weight + 1e-6).all()


@pytest.mark.parametrize("hq,n", [(4, 1), (8, 100)])
def test_codes_of_a_scale_of_zero_are_zero(hq, n):
    # what infinities in an otherwise empty page leave behind
    rng = np.random.default_rng(17)
    kc, vc, ks, vs, tab = make_cache(rng, 1, 1, 16, 64, [200])
    vs[:] = 0
    q = torch.as_tensor(rng.standard_normal((n, hq, 64))).to(torch.bfloat16)
    got = K.kda_kvcache_attention(q.cuda(), *gpu_cache(kc, vc, ks, vs, tab), torch.tensor([200], dtype=torch.int32).cuda(), cu_tokens=cu_of([n]))
    assert (got == 0).all()


@pytest.mark.parametrize("away", [13.0, 16.0, 18.0])
@pytest.mark.parametrize("hq,n,rows", [(1, 1, 1), (4, 1, 1200), (12, 1, 1200), (4, 64, 300)])
def test_many_small_weights_beside_a_large_one(hq, n, rows, away):
    # A first key whose score lies `away` above all others and whose value is zero; 2^17 keys of equal
    # scores and values v.  With M of them seen, o = v M e^-away / (1 + M e^-away).  Bound: fp16 weights
    # (2^-11, of a weight below fp16's normal range up to 2^-32 of the largest), scores in fp32 (2^-18
    # of the weights), one rounding to bf16 (2^-9).  Enough rows that a part is most of one.
    d, page, length = 64, 128, 2 ** 17
    pages = length // page
    code = {1.0: 0x38, 2.0: 0x40}
    kc, vc = np.zeros((2, 1, page, d), np.uint8), np.full((2, 1, page, d), code[1.0], np.uint8)
    vc[..., 1::2] = code[2.0] | 0x80
    kc[0, 0, 0, 0], vc[0, 0, 0] = code[1.0], 0
    ks, vs = np.full((2, 1), away, np.float32), np.full((2, 1), 0.5, np.float32)
    tab = np.array([[0] + [1] * (pages - 1)] * rows)
    q = torch.zeros(rows * n, hq, d)
    q[..., 0] = 1
    got = K.kda_kvcache_attention(q.bfloat16().cuda(), *gpu_cache(kc, vc, ks, vs, tab), torch.full((rows,), length, dtype=torch.int32).cuda(),
                                  cu_tokens=cu_of([n] * rows), scale=1.0).double().cpu().numpy()
    m = (length - n + np.tile(np.arange(n), rows))[:, None, None].astype(np.float64)  # others that a token sees
    v = np.where(np.arange(d) % 2, -1.0, 0.5)
    w = np.exp(-away)
    want = v * m * w / (1 + m * w)
    allowed = (2.0 ** -8 + 2.0 ** -10) * np.abs(want) + 2.0 ** -32 * m * np.abs(v) / (1 + m * w)
    assert (np.abs(got - want) <= allowed).all(), np.max(np.abs(got - want) / allowed)


@pytest.mark.parametrize("hq,n,parts", [(1, 1, 1824), (16, 1, 1216), (4, 40, 304)])
def test_rows_of_almost_two_to_the_31_tokens(hq, n, parts):
    # one page throughout, so every key of it is seen equally often but for the last few.  A length past
    # the limit is recorded and taken as it.  Sums and outputs are fp32, a part's in steps of 16 keys: 2^-24
    # of a sum for each step.
    rng = np.random.default_rng(18)
    kc, vc, ks, vs, _ = make_cache(rng, 1, 1, 128, 64, [128], spare=0)
    cache = gpu_cache(kc, vc, ks, vs, np.zeros((1, 1)))
    table = torch.zeros(1, 1 << 24, dtype=torch.int32, device="cuda")
    q = torch.as_tensor(rng.standard_normal((n, hq, 64))).to(torch.bfloat16)
    want, weight = ref.attention(q.double().numpy().reshape(1, n * hq, 64), kc, vc, ks, vs, np.zeros((1, 1), int), [128], [1], 128, 0.125)
    want, weight = want.reshape(n, hq, 64), weight.reshape(n, hq, 64)
    sums = 2 * 2.0 ** -24 * 2 ** 31 / 16 / parts
    K.kda_get_device_status()
    for length, status in ((2 ** 31 - 4096, 0), (2 ** 31 - 1, 1)):
        ln = torch.tensor([length], dtype=torch.int32, device="cuda")
        got = K.kda_kvcache_attention(q.cuda(), *cache[:4], table, ln, cu_tokens=cu_of([n]), scale=0.125).double().cpu().numpy()
        assert K.kda_get_device_status() == status
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + sums) * weight + 1e-6).all()
