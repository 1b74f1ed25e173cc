"""Beam selection against 64 bits: tokens and parents exactly, scores to fp32 rounding.

Logits lie on a coarse grid (multiples of 1/8), so totals of one beam are equal or at least
1/8 apart and rounding cannot change their order; scores of different beams are random.
Score bound: lse, the difference and the sum are rounded once each (3 x 2^-24 of values below
64, lse's sum of exponentials adds 2^-20): 2^-16."""
import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
import serving_testutil as ref

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def draw(rng, b, w, v, spread=3.0, tail=0.0):
    x = np.round(rng.standard_normal((b, w, v)) * spread * 8) / 8
    x[rng.random(x.shape) < tail] = -np.inf
    return np.clip(x, -15.875, 15.875) if not tail else x


def check(x, scores, k=None, done=None, eos=-1, dtype="fp32", strided=False):
    b, w, v = x.shape
    k = w if k is None else k
    logits = torch.as_tensor(x).to(DT[dtype]).cuda()
    if strided:
        wide = torch.full((b, w, v + 5), float("nan"), dtype=DT[dtype], device="cuda")
        wide[..., 2: v + 2] = logits
        logits = wide[..., 2: v + 2]
    want = ref.beam(logits.double().cpu().numpy(), scores, k, done, eos)
    got = K.kda_beam_select(logits, torch.as_tensor(scores).float().cuda(), num_out=k,
                            done=None if done is None else torch.as_tensor(done).cuda(), eos=eos)
    assert np.array_equal(got[1].cpu().numpy(), want[1]), (got[1].cpu().numpy(), want[1])
    assert np.array_equal(got[2].cpu().numpy(), want[2])
    s = got[0].double().cpu().numpy()
    assert np.array_equal(np.isinf(s), np.isinf(want[0]))
    ok = np.isfinite(want[0])
    assert (np.abs(s[ok] - want[0][ok]) <= 2.0 ** -16 * np.maximum(1, np.abs(want[0][ok]) / 64)).all()
    if done is not None:
        assert np.array_equal(got[3].cpu().numpy().astype(int), want[3])


def scores_of(rng, b, w):
    return -np.cumsum(rng.uniform(0, 4, (b, w)), 1).astype(np.float32)


@pytest.mark.parametrize("b,w,v", [(1, 1, 1), (1, 4, 3), (2, 3, 17), (3, 5, 1000), (2, 8, 8192), (1, 4, 8193), (2, 2, 32001), (40, 16, 2500)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_select(b, w, v, dtype):
    rng = np.random.default_rng(b + 10 * w + v)
    check(draw(rng, b, w, v), scores_of(rng, b, w), dtype=dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_many_outputs_and_padded_rows(dtype):
    rng = np.random.default_rng(1)
    check(draw(rng, 2, 6, 700), scores_of(rng, 2, 6), k=64, dtype=dtype, strided=True)
    check(draw(rng, 1, 64, 3001), scores_of(rng, 1, 64), k=64, dtype=dtype, strided=True)
    check(draw(rng, 3, 1, 40000), scores_of(rng, 3, 1), k=2, dtype=dtype)


@pytest.mark.parametrize("v", [520, 777, 1030, 2049, 9077])
@pytest.mark.parametrize("k", [16, 31, 32, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_short_segments(v, k, dtype):
    # rows, and ends of rows, of a few of the scan's steps; also with a block of tokens allowed only
    rng = np.random.default_rng(v + k)
    x = draw(rng, 2, 16, v)
    check(x, scores_of(rng, 2, 16), k=k, dtype=dtype)
    x[:, :, : v // 3] = -np.inf
    x[:, :, v // 3 + v // 2:] = -np.inf
    check(x, scores_of(rng, 2, 16), k=k, dtype=dtype)


def test_finished_beams():
    rng = np.random.default_rng(2)
    done = rng.random((6, 4)) < 0.5
    done[0] = True
    check(draw(rng, 6, 4, 900), scores_of(rng, 6, 4), done=done, eos=7)
    check(draw(rng, 6, 4, 900), scores_of(rng, 6, 4), k=9, done=done.astype(np.uint8), eos=0)


def test_equal_logits_go_to_the_lowest_index():
    check(np.zeros((2, 3, 20000)), np.zeros((2, 3), np.float32))
    check(np.full((1, 2, 700), -2.5), np.array([[-1.0, -1.0]], np.float32), k=40, dtype="bf16")


def test_first_step_with_beams_that_are_not_there():
    rng = np.random.default_rng(3)
    s = np.full((2, 4), -np.inf, np.float32)
    s[:, 0] = 0
    check(draw(rng, 2, 4, 5000), s)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_totals_that_rounding_makes_equal(dtype):
    # scores of -1e9 have a spacing of 64: all totals of such a beam are equal, so the lowest
    # tokens win whatever their logits are, beyond what any segment's largest logits hold
    rng = np.random.default_rng(4)
    x = draw(rng, 2, 2, 30000)
    x[0, 0, 5:] = -np.inf  # one beam has five candidates, the rest come from the other
    check(x, np.array([[0.0, -1e9], [-1e9, -1e9]], np.float32), k=12, dtype=dtype)


def test_masks():
    rng = np.random.default_rng(5)
    x = draw(rng, 4, 3, 4000, tail=0.9)
    x[0, 1] = -np.inf                     # a row that leaves nothing
    x[1] = -np.inf                        # a request that leaves nothing
    x[2, :, 2:] = -np.inf                 # fewer candidates than places
    check(x, scores_of(rng, 4, 3))
    x = draw(rng, 1, 2, 3000)
    x[0, 0, 10:] = np.finfo(np.float32).min   # the type's lowest value as a mask
    x[0, 1, 20:] = np.finfo(np.float32).min
    check(x, np.zeros((1, 2), np.float32), k=40)


def test_logits_that_are_not_finite_are_no_candidates():
    rng = np.random.default_rng(6)
    x = draw(rng, 2, 3, 9000)
    x[0, 0, 100], x[0, 1, 5000], x[1, 2, 8999] = np.nan, np.inf, np.nan
    x[1, 0] = np.nan
    check(x, scores_of(rng, 2, 3))


def test_large_vocabulary_and_reruns():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(4, 8, 131072, generator=g, device="cuda") * 3
    s = -torch.rand(4, 8, generator=g, device="cuda") * 8
    got = K.kda_beam_select(x, s)
    total = (s.double()[..., None] + torch.log_softmax(x.double(), 2)).view(4, -1)
    best = torch.topk(total, 8).values
    assert (got[0].double() - best).abs().max() <= 2.0 ** -16
    flat = (got[2].long() - 8 * torch.arange(4, device="cuda")[:, None]) * 131072 + got[1].long()
    assert (total.gather(1, flat) - best).abs().max() <= 2.0 ** -16
    for _ in range(3):
        again = K.kda_beam_select(x, s)
        assert all(torch.equal(a, b) for a, b in zip(again, got))


def test_selection_feeds_the_fork():
    rng = np.random.default_rng(8)
    b, w, v = 3, 4, 500
    x, s = draw(rng, b, w, v), scores_of(rng, b, w)
    pool = torch.randn(b * w, 33, device="cuda")
    before = pool.clone()
    _, _, parents = K.kda_beam_select(torch.as_tensor(x).float().cuda(), torch.as_tensor(s).cuda())
    tables = torch.arange(b * w, device="cuda", dtype=torch.int32).view(-1, 1)
    nt, nr = K.kda_pages_fork(tables, torch.ones(b * w, dtype=torch.int32, device="cuda"), parents.view(-1), pools=[pool])
    assert torch.equal(pool[nt[:, 0].long()], before[parents.view(-1).long()]) and (nr == 1).all()


LARGE = [1e9, 1e10, 1e12, 1e20, 1e29]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", LARGE)
def test_masks_of_large_numbers(size, dtype):
    # as additive masks have them: over whole loads of most lanes, in the last row over all of it (its
    # totals are then its score: fp32 does not hold the logarithm of the count beside such numbers)
    rng = np.random.default_rng(9)
    x = draw(rng, 2, 3, 9000)
    x[:, :, 40:8000] = -size
    x[1, 2] = -size
    check(x, scores_of(rng, 2, 3), k=7, dtype=dtype)
    x[:, :, 9:] = -size  # fewer others than places
    check(x, scores_of(rng, 2, 3), k=40, dtype=dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("size", LARGE)
def test_large_logits(size, dtype):
    rng = np.random.default_rng(10)
    x = draw(rng, 2, 2, 9000)
    x[0, 0, [70, 4000]] = size, size * 1.5
    x[0, 1, 8999] = size
    x[1, 0, 500:] = size
    x[1, 1, 3:] = -size
    x[1, 1, 3000] = -size * 0.5
    check(x, scores_of(rng, 2, 2), k=9, dtype=dtype)


@pytest.mark.parametrize("dtype,score", [("bf16", -1e6), ("fp16", -1e5)])
def test_equal_totals_of_logits_a_step_apart(dtype, score):
    # two tokens a step of the type above two of lower index, all four totals equal in fp32 and the
    # next smaller logit's below them: the two of lower index win, the second of which a segment that
    # keeps three candidates left out.  (Values are searched whose totals are no closer than a tenth of
    # the scores' spacing to where fp32 rounds the other way.)
    gap = float(np.spacing(np.float32(-score)))
    step = {"bf16": 2.0 ** -5, "fp16": 2.0 ** -8}[dtype]  # of the type in [4, 8)
    rng = np.random.default_rng(11)
    found = 0
    for low in np.arange(4 + step, 8 - 2 * step, step):
        x = draw(rng, 1, 1, 4000) / 4
        x[0, 0, [500, 600]], x[0, 0, [800, 900]] = low, low + step
        lse = np.log(np.exp(x[0, 0]).sum())
        t = (score + np.array([low + step, low, low - step]) - lse) / gap
        if np.abs(t - np.round(t)).max() > 0.4 or len(set(np.round(t[:2]))) > 1 or round(t[2]) == round(t[1]):
            continue
        found += 1
        want = ref.beam(x, np.array([[score]], np.float32), 2)
        assert want[1].tolist() == [[500, 600]]
        check(x, np.array([[score]], np.float32), k=2, dtype=dtype)
    assert found > 5
