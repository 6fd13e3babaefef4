"""8-bit append: a block's tokens anywhere in the slot list, in any order, are
written together, bit for bit as the oracle does it."""
import numpy as np
import pytest
import torch

import paged_kv_cache_400_b200 as pk
from oracle import quantized as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODE = pytest.mark.parametrize("code", ["int8", "e4m3"])


def make_pool(num_blocks, heads, dim, code, seed=0):
    r = np.random.RandomState(seed)
    p = pk.Q8Pool(num_blocks, heads, dim, code)
    c = r.randint(0, 100, p.codes.shape).astype(np.uint8)
    p.codes.view(torch.uint8).copy_(torch.from_numpy(c))
    p.scales.copy_(torch.from_numpy((np.exp(r.randn(num_blocks, 2, heads)) / 100).astype(np.float32)))
    return p


def rows(n, heads, dim, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, dim, generator=g) * torch.exp(torch.randn(n, 1, 1, generator=g))).to(dtype)


def check(p, k, v, slots, want_error=0):
    codes, scales = p.codes.view(torch.uint8).cpu().numpy().copy(), p.scales.cpu().numpy().copy()
    good = np.where(np.asarray(slots) < p.num_blocks * 16, slots, -1)
    oq.append(codes, scales, k.float().numpy(), v.float().numpy(), good, p.code)
    pk.pa_reshape_and_cache_q8(k.to(DEV), v.to(DEV), p, torch.as_tensor(np.asarray(slots, np.int64), device=DEV))
    assert pk.pa_get_device_error() == want_error
    assert np.array_equal(p.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(p.codes.view(torch.uint8).cpu().numpy(), codes)


@CODE
@pytest.mark.parametrize("requests,steps,start", [(33, 2, 0), (64, 4, 0), (64, 4, 5), (300, 3, 14), (1000, 7, 0)])
def test_time_major_list(requests, steps, start, code):
    """The tokens of one time after those of the one before, for more requests than a warp has lanes."""
    perm = np.random.RandomState(requests).permutation(2 * requests)
    pos = start + np.arange(steps)
    slots = np.stack([perm[2 * r + pos // 16] * 16 + pos % 16 for r in range(requests)], 1).ravel()
    n = len(slots)
    p = make_pool(2 * requests, 2, 64, code, 1)
    check(p, rows(n, 2, 64, 2), rows(n, 2, 64, 3), slots)


@CODE
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,dim,tokens", [(1, 128, 700), (3, 64, 5000), (8, 128, 3000), (20, 64, 100)])
def test_shuffled_list(heads, dim, tokens, dtype, code):
    """Any order, some of the rows of each block, padding in between, blocks that start afresh and others."""
    r = np.random.RandomState(tokens)
    blocks = tokens // 10 + 2
    slots = r.permutation(blocks * 16)[:tokens]
    slots[r.rand(tokens) < 0.1] = -1
    p = make_pool(blocks, heads, dim, code, 4)
    check(p, rows(tokens, heads, dim, 5, dtype), rows(tokens, heads, dim, 6, dtype), slots)


@CODE
def test_rows_named_again_far_away(code):
    """The later of two tokens counts, whatever lies between them; a fresh row 0 at the list's very end."""
    r = np.random.RandomState(3)
    slots = np.concatenate([np.arange(3, 16), 64 + np.arange(40), r.randint(0, 20, 3000) * 16 + r.randint(1, 16, 3000),
                            [7, 5, 5], [-1] * 100, [0]])
    p = make_pool(20, 2, 128, code, 7)
    check(p, rows(len(slots), 2, 128, 8), rows(len(slots), 2, 128, 9), slots)
    slots = np.concatenate([[18], [-1] * 9000, [16], [-1] * 2047, [18, 400]])
    check(p, rows(len(slots), 2, 128, 10), rows(len(slots), 2, 128, 11), slots, pk.PA_DEVERR_SLOT)


@CODE
@pytest.mark.parametrize("tokens", [2047, 2048, 2049, 30000, 120000])
def test_long_lists(tokens, code):
    """One KV head: up to 256 entries of a CTA."""
    r = np.random.RandomState(tokens)
    blocks = tokens // 16 + 1
    perm = r.permutation(blocks)
    at = np.arange(tokens)
    slots = perm[at // 16] * 16 + at % 16
    swap = r.permutation(tokens)[:tokens // 8]
    slots[swap] = slots[np.sort(swap)]
    p = make_pool(blocks, 1, 64, code, 12)
    check(p, rows(tokens, 1, 64, 13, torch.bfloat16), rows(tokens, 1, 64, 14, torch.bfloat16), slots)
