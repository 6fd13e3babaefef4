"""Attention over 8-bit pools with V tiles of exact zeros beside small ones: a zero
tile takes its share of the softmax's sum and nothing of the others' precision,
whatever it scores."""
import numpy as np
import pytest
import torch

import paged_kv_cache_400_b200 as pk
import test_gpu_q8 as q8

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODE = pytest.mark.parametrize("code", ["int8", "e4m3"])
AMP = pytest.mark.parametrize("amp", [1.0, 1e-3, 1e-5, 1e-6, 1e-8])


def pool_with(code, dim, blocks, amp, zero, seed, heads=2):
    """V scales of about amp / 100, zero in the blocks of `zero`."""
    p = q8.make_pool(blocks, heads, dim, code, seed)
    p.scales[:, 1] *= amp
    p.scales[torch.as_tensor(sorted(zero), device=DEV, dtype=torch.long), 1] = 0
    return p


def check(p, q, lens, news, tables, codes, scales, out, start, scale, io, chain, biased):
    q8.check_rows(out, q, lens, news, start, codes, scales, tables, p, io, scale,
                  2.0 ** -11 if io == "bf16" else 2.0 ** -22, chain, biased=biased)


def zero_blocks(tables, lens, which):
    """Of every sequence: its first block, its last one, every third, or all but the fourth."""
    out = set()
    for t, n in zip(tables, lens):
        blk = t[:(n + 15) // 16]
        out |= set({"first": blk[:1], "last": blk[-1:], "third": blk[::3],
                    "most": np.delete(blk, min(3, len(blk) - 1))}[which].tolist())
    return out


WHICH = pytest.mark.parametrize("which", ["first", "last", "third", "most"])


@CODE
@AMP
@WHICH
@pytest.mark.parametrize("io,dim,group", [("bf16", 128, 4), ("f32", 128, 1), ("bf16", 64, 9), ("f32", 64, 12)])
def test_decode(io, dim, group, which, amp, code):
    """One pass, partitions with a merge, and a warp for each sequence."""
    for lens, max_len in (([64, 50, 200, 1, 17], 256), ([3000, 64, 130, 2049], 3008), ([64, 40, 33, 80] * 60, 100)):
        blocks = sum((n + 15) // 16 for n in lens) + 3
        tables = q8.tables_for(lens, blocks, (max_len + 15) // 16, 5)
        p = pool_with(code, dim, blocks, amp, zero_blocks(tables, lens, which), 6)
        codes, scales = q8.host(p)
        q = q8.rows(len(lens), 2 * group, dim, io, 7, 0.3)
        out = q8.decode(p, q, tables, lens, max_len, dim ** -0.5)
        assert pk.pa_get_device_error() == 0
        check(p, q, lens, [1] * len(lens), tables, codes, scales, out, range(len(lens)), dim ** -0.5, io,
              32 * 16 + 4 + (max_len + 127) // 128, q8.biased(code, io))


@CODE
@AMP
@WHICH
def test_prefill(which, amp, code):
    lens, news = [64, 200, 1, 17, 500, 130], [64, 200, 1, 5, 40, 130]
    blocks = sum((n + 15) // 16 for n in lens) + 3
    tables = q8.tables_for(lens, blocks, None, 5)
    p = pool_with(code, 128, blocks, amp, zero_blocks(tables, lens, which), 6)
    codes, scales = q8.host(p)
    start = np.concatenate([[0], np.cumsum(news)]).tolist()
    q = q8.rows(start[-1], 8, 128, "bf16", 7, 0.3)
    out = q8.prefill(p, q, tables, lens, start, 128 ** -0.5, max(news))
    assert pk.pa_get_device_error() == 0
    check(p, q, lens, news, tables, codes, scales, out, start, 128 ** -0.5, "bf16", max(lens), False)


@CODE
@pytest.mark.parametrize("amp", [1.0, 1e-4])
@pytest.mark.parametrize("lead", [20, 60, 90, 400])
@pytest.mark.parametrize("where", [0, 2, 7])
def test_zero_tile_that_scores_highest(where, lead, amp, code):
    """Keys along the query in one block: its scores lie `lead` (log2) above the
    others', which are small; the output is the others' V, that much smaller."""
    dim, lens = 128, [128, 128]
    tables = q8.tables_for(lens, 20, 8, 5)
    p = pool_with(code, dim, 20, amp, tables[:, where].tolist(), 6)
    k = p.codes.view(torch.uint8).clone()
    k[:, 0] = 0
    one = 64 if code == "int8" else 0x58  # 16 as e4m3
    for t in tables:
        k[int(t[where]), 0] = one
        for i in range(8):
            if i != where:
                k[int(t[i]), 0, :, :, :2] = 1 + i  # small scores that differ
    p.codes.view(torch.uint8).copy_(k)
    value = 64.0 if code == "int8" else 16.0
    p.scales[:, 0] = lead / (value * dim * 1.4427)
    codes, scales = q8.host(p)
    for io in ("bf16", "f32"):
        q = torch.ones(2, 8, dim).to(q8.IO[io])
        out = q8.decode(p, q, tables, lens, 128, 1.0)
        assert pk.pa_get_device_error() == 0
        check(p, q, lens, [1, 1], tables, codes, scales, out, range(2), 1.0, io, 128, q8.biased(code, io))
    q = torch.ones(2 * 40, 8, dim).to(torch.bfloat16)
    out = q8.prefill(p, q, tables, lens, [0, 40, 80], 1.0, 40)
    assert pk.pa_get_device_error() == 0
    check(p, q, lens, [40, 40], tables, codes, scales, out, [0, 40], 1.0, "bf16", 128, False)


@CODE
@pytest.mark.parametrize("amp", [1.0, 1e-6])
def test_bad_block_counts_as_zero_vectors(amp, code):
    """A table entry outside the pool: zero K and V, which take no precision either."""
    lens = [100, 40]
    tables = q8.tables_for(lens, 21, 7, 5)
    p = pool_with(code, 128, 21, amp, [], 6)
    p.codes.view(torch.uint8)[20] = 0
    codes, scales = q8.host(p)
    bad, seen = tables.copy(), tables.copy()
    for at in ((0, 2), (1, 0)):
        bad[at], seen[at] = 999, 20  # the oracle reads a block of zeros
    codes[20], scales[20] = 0, 0
    for io in ("bf16", "f32"):
        q = q8.rows(2, 8, 128, io, 7, 0.3)
        out = q8.decode(p, q, bad, lens, 112, 0.09)
        assert pk.pa_get_device_error() == pk.PA_DEVERR_BLOCK
        check(p, q, lens, [1, 1], seen, codes, scales, out, range(2), 0.09, io, 112, q8.biased(code, io))
