"""Page operations against plain loops: tables, references, contents; whole numbers, so every
comparison is exact."""
import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
import serving_testutil as ref

pytestmark = pytest.mark.gpu

NO_FREE, INVALID = 8, 1


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def make_rows(rng, rows, width, spare, share=0.5, holes=0.1):
    """Tables whose rows share some pages and miss some entries, their references, and one page
    that someone else holds as well."""
    total = rows * width
    pool = rng.permutation(total + spare)
    tables = pool[:total].reshape(rows, width).copy()
    for r in range(1, rows):
        for j in range(width):
            if rng.random() < share:
                tables[r, j] = tables[rng.integers(0, r), j]
    tables[rng.random((rows, width)) < holes] = -1
    refs = np.bincount(tables[tables >= 0].ravel(), minlength=total + spare)
    held = np.nonzero(refs)[0]
    if held.size:
        refs[held[0]] += 1
    return tables, refs


def make_pools(rng, pages):
    """Pools of several types, page sizes (16-, 4- and 1-byte units) and layouts."""
    g = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 30)))
    wide = torch.randn(pages, 3, 40, generator=g, device="cuda")
    return [torch.randn(pages, 2, 16, 16, generator=g, device="cuda"),
            torch.randint(0, 256, (pages, 5, 7), generator=g, device="cuda", dtype=torch.uint8),
            torch.randn(pages, 3, generator=g, device="cuda"),
            wide[:, 1, :36],  # a slice: pages apart, contiguous inside
            torch.randn(pages, 9000, generator=g, device="cuda").to(torch.bfloat16)]


def copied(pools, copies):
    out = [p.clone() for p in pools]
    for p, o in zip(pools, out):
        for a, b in copies:
            o[b] = p[a]
    return out


@pytest.mark.parametrize("rows,width,spare,page", [
    (1, 1, 0, 0), (6, 1, 6, 0), (7, 5, 40, 16), (33, 3, 99, 64), (16, 9, 3, 16), (5, 4, 20, 0)])
@pytest.mark.parametrize("seed", [0, 1])
def test_fork(rows, width, spare, page, seed):
    rng = np.random.default_rng(100 * seed + rows)
    tables, refs = make_rows(rng, rows, width, spare)
    parents = rng.integers(-1, rows, rows)
    lens = rng.integers(0, max(1, width * max(page, 1)) + 1, rows)
    pools = make_pools(rng, len(refs))
    want_t, want_r, copies = ref.fork(tables, refs, parents, lens, page)
    want_pools = copied(pools, copies)
    t, r = dev(tables), dev(refs)
    K.kda_get_device_status()
    nt, nr = K.kda_pages_fork(t, r, dev(parents), lens=dev(lens), page_tokens=page, pools=pools)
    assert torch.equal(nt.cpu().long(), torch.as_tensor(want_t).long())
    assert torch.equal(nr.cpu().long(), torch.as_tensor(want_r).long())
    for p, w in zip(pools, want_pools):
        assert torch.equal(p, w)
    assert torch.equal(t, dev(tables)) and torch.equal(r, dev(refs))  # inputs stay
    short = ((want_t < 0) & (np.where(parents[:, None] >= 0, tables[parents], -1) >= 0)).any()
    assert K.kda_get_device_status() == (NO_FREE if short else 0)


def test_fork_of_states_needs_no_spare_pages():
    # beams: every page is in use, half the rows end, the others are continued twice
    rows = 64
    parents = np.repeat(np.arange(0, rows, 2), 2)[np.random.default_rng(1).permutation(rows)]
    pool = torch.randn(2, rows, 4, 8, device="cuda")
    tables = np.random.default_rng(2).permutation(rows)[:, None]
    before = pool.clone()
    nt, nr = K.kda_pages_fork(dev(tables), dev(np.ones(rows)), dev(parents), pools=[pool], layers_first=True)
    assert K.kda_get_device_status() == 0
    new = nt.cpu().numpy()[:, 0]
    assert sorted(new.tolist()) == list(range(rows)) and (nr == 1).all()
    for r in range(rows):
        assert torch.equal(pool[:, new[r]], before[:, tables[parents[r], 0]])


def test_fork_large_plan_matches_loops():
    # above the one-CTA limit: eight CTAs scan entries and pages
    rng = np.random.default_rng(5)
    rows, width, page = 96, 70, 16
    tables, refs = make_rows(rng, rows, width, 7001, share=0.7)
    parents = rng.integers(-1, rows, rows)
    lens = rng.integers(0, width * page + 1, rows)
    want_t, want_r, copies = ref.fork(tables, refs, parents, lens, page)
    pool = torch.arange(len(refs), device="cuda", dtype=torch.int32).view(-1, 1).repeat(1, 4)
    nt, nr = K.kda_pages_fork(dev(tables), dev(refs), dev(parents), lens=dev(lens), page_tokens=page, pools=[pool])
    assert np.array_equal(nt.cpu().numpy(), want_t) and np.array_equal(nr.cpu().numpy(), want_r)
    want = np.arange(len(refs))
    for a, b in copies:
        want[b] = a
    assert np.array_equal(pool[:, 3].cpu().numpy(), want)
    K.kda_get_device_status()


def test_more_pages_than_shared_memory_holds():
    rng = np.random.default_rng(6)
    rows, width, pages = 50, 40, 140001
    order = rng.permutation(pages)
    tables = order[: rows * width].reshape(rows, width).copy()
    tables[1:, :9] = tables[0, :9]
    refs = np.bincount(tables.ravel(), minlength=pages)
    parents = rng.integers(0, rows, rows)
    lens = np.full(rows, 9 * 16 + 3)
    want_t, want_r, copies = ref.fork(tables, refs, parents, lens, 16)
    pool = torch.arange(pages, device="cuda", dtype=torch.int32).view(-1, 1)
    nt, nr = K.kda_pages_fork(dev(tables), dev(refs), dev(parents), lens=dev(lens), page_tokens=16, pools=[pool])
    assert np.array_equal(nt.cpu().numpy(), want_t) and np.array_equal(nr.cpu().numpy(), want_r)
    want = np.arange(pages)
    for a, b in copies:
        want[b] = a
    assert np.array_equal(pool[:, 0].cpu().numpy(), want)
    want_t, want_r, want_m, n, _ = ref.compact(tables, refs)
    ct, cr, pm, live = K.kda_pages_compact(dev(tables), dev(refs))
    assert np.array_equal(ct.cpu().numpy(), want_t) and np.array_equal(cr.cpu().numpy(), want_r)
    assert np.array_equal(pm.cpu().numpy(), want_m) and live.item() == n
    want_t, want_r = ref.alloc(tables[:, :20], refs, np.full(rows, 20))
    at, ar = K.kda_pages_alloc(dev(np.ascontiguousarray(tables[:, :20])), dev(refs), dev(np.full(rows, 20)))
    assert np.array_equal(at.cpu().numpy(), want_t) and np.array_equal(ar.cpu().numpy(), want_r)


@pytest.mark.parametrize("rows,width,pages", [(3, 4, 20), (1, 1, 1), (40, 130, 9000), (5, 3, 4), (9, 30, 16385), (9, 30, 32768), (9, 30, 65537)])
def test_alloc_and_free(rows, width, pages):
    rng = np.random.default_rng(rows)
    tables = np.full((rows, width), -1)
    have = rng.permutation(pages)[: min(pages // 3, rows * width // 2)]
    at = rng.permutation(rows * width)[: len(have)]
    tables.ravel()[at] = have
    refs = np.bincount(have, minlength=pages)
    want = rng.integers(0, width + 1, rows)
    want_t, want_r = ref.alloc(tables, refs, want)
    K.kda_get_device_status()
    nt, nr = K.kda_pages_alloc(dev(tables), dev(refs), dev(want))
    assert np.array_equal(nt.cpu().numpy(), want_t) and np.array_equal(nr.cpu().numpy(), want_r)
    short = any((want_t[r, : want[r]] < 0).any() for r in range(rows))
    assert K.kda_get_device_status() == (NO_FREE if short else 0)
    drop = rng.random(rows) < 0.5
    ft, fr = K.kda_pages_free(nt, nr, dev(drop, torch.bool))
    gone = want_t[drop]
    left = want_r - np.bincount(gone[gone >= 0].ravel(), minlength=pages)
    assert np.array_equal(ft.cpu().numpy(), np.where(drop[:, None], -1, want_t))
    assert np.array_equal(fr.cpu().numpy(), left)


@pytest.mark.parametrize("rows,width,spare,seed", [(4, 3, 10, 0), (1, 1, 0, 1), (9, 7, 64, 2), (90, 64, 5000, 3)])
def test_compact(rows, width, spare, seed):
    rng = np.random.default_rng(seed)
    tables, refs = make_rows(rng, rows, width, spare, holes=0.4)
    pools = make_pools(rng, len(refs))[: 5 if rows < 20 else 1]
    want_t, want_r, want_m, n, copies = ref.compact(tables, refs)
    want_pools = copied(pools, copies)
    nt, nr, pm, live = K.kda_pages_compact(dev(tables), dev(refs), pools=pools)
    assert np.array_equal(nt.cpu().numpy(), want_t) and np.array_equal(nr.cpu().numpy(), want_r)
    assert np.array_equal(pm.cpu().numpy(), want_m) and live.item() == n
    for p, w in zip(pools, want_pools):
        assert torch.equal(p, w)


def test_copy_skips_and_records():
    pool = torch.randn(6, 5000, device="cuda")
    want = pool.clone()
    want[1], want[5] = pool[0], pool[3]
    K.kda_get_device_status()
    K.kda_pages_copy(dev([0, -1, 3, 2]), dev([1, 2, 5, -1]), [pool])
    assert torch.equal(pool, want) and K.kda_get_device_status() == 0
    K.kda_pages_copy(dev([0, 6]), dev([2, 4]), [pool])  # page 6 is not there
    want[2] = want[0]
    assert torch.equal(pool, want) and K.kda_get_device_status() == INVALID


def test_numbers_out_of_range_are_absent_and_recorded():
    tables, refs = dev([[0, 7], [1, 2]]), dev([1, 1, 1, 0])
    nt, nr = K.kda_pages_fork(tables, refs, dev([0, 1]), page_tokens=0)
    assert nt.tolist() == [[0, -1], [1, 2]] and nr.tolist() == [1, 1, 1, 0]
    assert K.kda_get_device_status() == INVALID
    nt, nr = K.kda_pages_fork(dev([[0], [1]]), dev([1, 1]), dev([5, 1]))
    assert nt.tolist() == [[-1], [1]] and nr.tolist() == [0, 1]
    assert K.kda_get_device_status() == INVALID
    nt, *_ = K.kda_pages_compact(tables, refs)
    assert nt.tolist() == [[0, -1], [1, 2]] and K.kda_get_device_status() == INVALID


def test_no_rows_and_no_pages():
    nt, nr = K.kda_pages_fork(dev(np.zeros((0, 3))), dev([0, 2]), dev([]))
    assert nt.shape == (0, 3) and nr.tolist() == [0, 2]
    nt, nr, pm, n = K.kda_pages_compact(dev([[-1, -1]]), dev([]))
    assert nt.tolist() == [[-1, -1]] and n.item() == 0


def test_offsets_past_32_bits():
    # a pool of 5 GiB: page 4 starts past 2^32 bytes
    pool = torch.empty(5, 1 << 30, dtype=torch.uint8, device="cuda")
    pool[0, -5000:] = torch.arange(5000, device="cuda").to(torch.uint8)
    K.kda_pages_copy(dev([0]), dev([4]), [pool])
    assert torch.equal(pool[4, -5000:], pool[0, -5000:])


def test_graph_and_side_stream():
    rows = 8
    pool = torch.randn(rows, 64, device="cuda")
    tables, refs, parents = dev(np.arange(rows)[:, None]), dev(np.ones(rows)), dev(np.zeros(rows))
    nt, nr = torch.empty_like(tables), torch.empty_like(refs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call = lambda: K.kda_pages_fork(tables, refs, parents, pools=[pool], new_tables=nt, new_refs=nr)  # noqa: E731
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    torch.cuda.current_stream().wait_stream(s)
    assert (pool == pool[0]).all()
    pool.copy_(torch.randn(rows, 64, device="cuda"))
    parents.fill_(3)
    g.replay()
    torch.cuda.synchronize()
    assert (pool == pool[3]).all() and nt[0, 0].item() == 3
