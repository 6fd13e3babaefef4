"""8-bit decode's partitions, read off the workspace size: a batch that is planned
as one round of resident CTAs is no more than the SMs hold at once."""
import json
import os
import subprocess
import sys

import pytest

from paged_kv_cache_400_b200 import binding as bd

SMS = 148
# CTAs of a decode kernel that an SM holds: (head_dim, more than 8 heads a group, dtype) -> (bf16, fp32 queries)
HOLDS = {(128, False, bd.PA_Q8_INT8): (3, 3), (128, False, bd.PA_Q8_E4M3): (3, 3),
         (64, False, bd.PA_Q8_INT8): (4, 4), (64, False, bd.PA_Q8_E4M3): (4, 4),
         (128, True, bd.PA_Q8_INT8): (3, 2), (128, True, bd.PA_Q8_E4M3): (3, 2),
         (64, True, bd.PA_Q8_INT8): (2, 2), (64, True, bd.PA_Q8_E4M3): (3, 2)}
SHAPES = [(seqs, kv, kv * group, dim, dtype, length) for seqs, kv, length in
          [(1, 8, 9000), (1, 8, 131071), (6, 8, 2928), (28, 2, 10517), (18, 8, 2048), (64, 8, 8192), (3, 1, 700), (200, 8, 137)]
          for group in (1, 8, 9, 16) for dim in (64, 128) for dtype in (bd.PA_Q8_INT8, bd.PA_Q8_E4M3)]


def size_of(shape):
    seqs, kv, heads, dim, dtype, length = shape
    return bd.lib().pa_decode_q8_workspace_size(seqs, heads, bd.pa_pool_desc(8, kv, dim, 16, dtype), length)


def partitions(shape):
    """The number of partitions whose states and work list make up the size."""
    seqs, _, heads, dim, _, _ = shape
    up = lambda x: (x + 255) // 256 * 256
    for n in range(2, 70000):
        units = seqs * heads * n
        total = up(up(up(units * dim * 4) + units * 8) + seqs * n * 4) + 8
        if total >= size_of(shape):
            assert total == size_of(shape)
            return n
    raise AssertionError("no number of partitions has this size")


@pytest.mark.parametrize("seqs,kv,length", [(1, 8, 9000), (6, 8, 2928), (2, 4, 9000), (3, 8, 6000)])
@pytest.mark.parametrize("dim,wide,dtype", sorted(HOLDS))
def test_one_round_fits(dim, wide, dtype, seqs, kv, length):
    shape = (seqs, kv, kv * (16 if wide else 4), dim, dtype, length)
    n = partitions(shape)
    holds = max(HOLDS[dim, wide, dtype])  # the size covers both types of queries
    assert n * seqs * kv <= holds * SMS or length / n > 1024
    assert (n + 1) * seqs * kv > holds * SMS * 0.9 or length / n <= 144  # and fills the round


@pytest.mark.gpu
def test_sizes_without_a_device_are_the_devices():
    code = ("import json, sys; sys.path.insert(0, 'tests'); import test_q8_partitions as t; "
            "print(json.dumps([t.size_of(s) for s in t.SHAPES]))")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, check=True, timeout=300,
                         env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}).stdout
    assert json.loads(out.strip().splitlines()[-1]) == [size_of(s) for s in SHAPES]
