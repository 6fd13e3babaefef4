"""Calls of a step with nothing between them: tables that move lengths over a
partition boundary, then at once a decode that takes its partitions from the
work list. Lengths read too early would drop the last partition or leave a row
unwritten."""
import pytest
import torch

import paged_kv_cache_400_b200 as pk

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, HKV, G, D, MOST = 64, 8, 4, 128, 8192
W = MOST // 16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Setup:
    """64 requests whose lengths end on partition boundaries (1024 tokens for 8-bit
    pools, 2048 for bf16 ones), over a pool of few blocks that they share."""

    def __init__(self, kind, in_place):
        self.kind, self.in_place = kind, in_place
        g = torch.Generator(device=DEV).manual_seed(3)
        self.N = 600
        part = 1024 if kind == "int8" else pk.pa_decode_partition_tokens(
            B, HKV * G, torch.empty(1, 2, HKV, 16, D, dtype=torch.bfloat16), MOST)
        self.lens0 = i32([part * (b % 3) + (0 if b % 5 else part - 1) for b in range(B)])
        self.tables = torch.randint(0, 500, (B, W), generator=g, device=DEV).to(torch.int32)
        self.tables0 = self.tables.clone()
        self.ring, self.state0 = torch.arange(4000, dtype=torch.int32, device=DEV) % 100 + 500, i32([7, 100, 0, 0])
        self.state, self.state_out = self.state0.clone(), self.state0.clone()
        self.lens = self.lens0.clone()
        self.lens_out = self.lens if in_place else torch.empty_like(self.lens)
        self.qs = torch.empty(B + 1, dtype=torch.int32, device=DEV)
        self.slots = torch.empty(B * 16, dtype=torch.int64, device=DEV)  # in place: two launches
        self.tws = pk.alloc_tables_workspace(B)
        self.q = torch.randn(B, HKV * G, D, generator=g, device=DEV).to(torch.bfloat16)
        self.out = torch.empty_like(self.q)
        if kind == "int8":
            self.pool = pk.Q8Pool(self.N, HKV, D)
            self.pool.codes.copy_(torch.randint(-127, 128, self.pool.codes.shape, generator=g, device=DEV))
            self.pool.scales.fill_(0.01)
        else:
            self.pool = torch.randn(self.N, 2, HKV, 16, D, generator=g, device=DEV).to(torch.bfloat16)
        self.ws = pk.alloc_workspace(B, HKV * G, self.pool, MOST)

    def reset(self):
        self.lens.copy_(self.lens0), self.tables.copy_(self.tables0), self.state.copy_(self.state0)
        self.lens_out.copy_(self.lens0), self.out.fill_(float("nan"))

    def tables_call(self, op, ask):
        so = self.state if self.in_place else self.state_out
        if op == "extend":
            pk.pa_tables_extend(self.tables, self.lens, ask, self.ring, self.state, self.lens_out, self.qs, self.slots,
                                so, self.N, 16, self.tws)
        else:
            pk.pa_tables_release(self.tables, self.lens, ask, self.ring, self.state, self.lens_out, so, self.N, self.tws)

    def decode(self):
        f = pk.pa_decode_q8 if self.kind == "int8" else pk.pa_decode
        f(self.out, self.q, self.pool, self.tables, self.lens_out, D ** -0.5, MOST, self.ws)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("op", ["extend", "release"])
@pytest.mark.parametrize("kind", ["int8", "bf16"])
def test_decode_at_once_behind_tables(kind, op, in_place):
    s = Setup(kind, in_place)
    ask = i32([1] * B) if op == "extend" else i32([int(b % 4 == 1) for b in range(B)])
    s.reset()
    s.tables_call(op, ask)
    torch.cuda.synchronize()
    want_lens = s.lens_out.clone()
    s.decode()
    torch.cuda.synchronize()
    want = s.out.clone()
    old = s.lens0 + 1 if op == "extend" else torch.where(ask != 0, 0, s.lens0)
    assert torch.equal(want_lens, old.to(torch.int32)) and torch.isfinite(want).all()
    for _ in range(40):
        s.reset()
        torch.cuda.synchronize()
        s.tables_call(op, ask)
        s.decode()
        torch.cuda.synchronize()
        assert torch.equal(s.lens_out, want_lens) and torch.equal(s.out, want)
    assert pk.pa_get_device_error() == 0
