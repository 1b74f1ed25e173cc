"""kda_decode on a pool of states: bit for bit what kda_decode gives on the gathered states."""
import numpy as np
import pytest
import torch

import chunked_kda_delta_gb300 as K
from chunked_kda_delta_gb300.inputs import custom, make_inputs

pytestmark = pytest.mark.gpu


def tokens(B, T, H, Hq, seed):
    inp = make_inputs(custom([T] * B, H, False, seed, dense=True, num_q_heads=Hq), "cuda")
    return [inp[n].view(B, T, *inp[n].shape[1:]) for n in ("q", "k", "v", "g", "beta")]


@pytest.mark.parametrize("B,T,H,Hq", [(1, 1, 1, 1), (5, 1, 4, 4), (7, 3, 6, 2), (33, 1, 12, 12)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_matches_decode(B, T, H, Hq, dtype):
    x = tokens(B, T, H, Hq, 3)
    pages = 2 * B + 1
    pool = (torch.randn(pages, H + 1, 128, 128, device="cuda") * 0.1).to(dtype)[:, :H]  # pages apart
    at = torch.as_tensor(np.random.default_rng(B).permutation(pages)[:B]).to(torch.int32).cuda()
    want_pool = pool.clone()
    s = pool[at.long()].contiguous()
    want, fin = K.kda_decode(*x, initial_state=s, final_state=s)
    want_pool[at.long()] = fin
    got = K.kda_decode_paged(*x, pool, at)
    assert torch.equal(got, want) and torch.equal(pool, want_pool)


def test_idle_sequences_and_pages_out_of_range():
    x = tokens(4, 1, 2, 2, 5)
    pool = torch.randn(3, 2, 128, 128, device="cuda") * 0.1
    before = pool.clone()
    K.kda_get_device_status()
    out = K.kda_decode_paged(*x, pool, torch.tensor([-1, 2, -7, 0], dtype=torch.int32, device="cuda"))
    assert K.kda_get_device_status() == 0
    assert (out[0] == 0).all() and (out[2] == 0).all() and (out[1] != 0).any()
    assert torch.equal(pool[1], before[1]) and not torch.equal(pool[0], before[0])
    before = pool.clone()
    out = K.kda_decode_paged(*x, pool, torch.tensor([3, -1, -1, -1], dtype=torch.int32, device="cuda"))
    assert K.kda_get_device_status() == 1 and (out == 0).all() and torch.equal(pool, before)


def test_refusals():
    x = tokens(2, 1, 2, 2, 6)
    pool = torch.zeros(2, 2, 128, 128, device="cuda")
    at = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        K.kda_decode_paged(*x, pool, at.long())
    with pytest.raises(ValueError):
        K.kda_decode_paged(*x, pool[:, :1], at)
    with pytest.raises(ValueError):
        K.kda_decode_paged(*x, pool.transpose(2, 3), at)
    with pytest.raises(K.KdaError):  # grouped query heads would race on the state
        K.kda_decode_paged(*tokens(2, 1, 2, 4, 6), pool, at)


@pytest.mark.parametrize("handle", [0, 1])
def test_handles_of_the_default_stream(handle):
    # the call comes after work that is pending there
    x = tokens(3, 1, 2, 2, 8)
    state = torch.randn(3, 2, 128, 128, device="cuda") * 0.1
    at = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    want_pool = state.clone()
    want = K.kda_decode_paged(*x, want_pool, at)
    pool = torch.zeros_like(state)
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.default_stream()):
        for _ in range(8):
            busy = busy @ busy * 1e-3
        pool.copy_(state)
    got = K.kda_decode_paged(*x, pool, at, stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(pool, want_pool)
