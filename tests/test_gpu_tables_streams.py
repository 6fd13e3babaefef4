"""Step tables on a stream that is not the current one, with no workspace given."""
import numpy as np
import pytest
import torch

import paged_kv_cache_400_b200 as pk
from oracle import tables as ot

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x, np.int64).tolist(), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("batch", [5000, 4096])
def test_workspace_of_a_call_on_a_side_stream(batch, handle):
    """The side stream is held up, and meanwhile the current stream allocates and
    fills as many bytes as the workspace has: the call's sums must not lie there."""
    r = np.random.RandomState(batch)
    W, N = 6, batch * 6
    lens, new = r.randint(0, 40, batch), r.randint(0, 20, batch)
    perm = r.permutation(N)
    used = ot.pages(lens)
    t = np.full((batch, W), -1, np.int64)
    at = 0
    for b, n in enumerate(used):
        t[b, :n] = perm[at:at + n]
        at += n
    free = perm[at:]
    ring = np.concatenate([free, np.full(at, -1)])
    state = [0, len(free)]
    want_t, want_r = t.tolist(), ring.tolist()
    e_lens, e_qs, e_slots, e_state, e_err = ot.extend(want_t, lens.tolist(), new.tolist(), want_r, *state, N,
                                                      int(new.sum()), 0)
    done = (r.rand(batch) < 0.5).astype(int)
    r_lens, r_state, r_err = ot.release(want_t, e_lens, done.tolist(), want_r, *e_state[:2], N)
    dt, dl, dn, dd, dr, ds = i32(t), i32(lens), i32(new), i32(done), i32(ring), i32(state + [0, 0])
    mid, out, qs, so = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (batch, batch, batch + 1, 4))
    slots = torch.empty(int(new.sum()), dtype=torch.int64, device=DEV)
    size = pk.alloc_tables_workspace(batch).numel()
    side = torch.cuda.Stream()
    st = side.cuda_stream if handle else side
    torch.cuda.synchronize()

    def noise():
        return [torch.full((size,), 0x7f, dtype=torch.uint8, device=DEV) for _ in range(8)]

    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    pk.pa_tables_extend(dt, dl, dn, dr, ds, mid, qs, slots, so, N, 0, stream=st)
    kept = noise()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    pk.pa_tables_release(dt, mid, dd, dr, so, out, so, N, stream=st)
    kept += noise()
    torch.cuda.synchronize()
    assert len(kept) == 16 and all(bool((k == 0x7f).all()) for k in kept)
    assert mid.tolist() == e_lens and qs.tolist() == e_qs and slots.tolist() == e_slots and dt.tolist() == want_t
    assert out.tolist() == r_lens and so.tolist() == r_state and dr.tolist() == want_r
    assert e_err == r_err == 0 and pk.pa_get_device_error() == 0


def test_workspace_on_the_default_stream_by_handle():
    ring, state = pk.make_free_ring(8)
    lens, qs, slots = i32([0, 0]), i32([0] * 3), torch.zeros(2, dtype=torch.int64, device=DEV)
    pk.pa_tables_extend(i32([[-1] * 4] * 2), lens, i32([1, 1]), ring, state, lens, qs, slots, state, 8, stream=0)
    assert slots.tolist() == [0, 16] and lens.tolist() == [1, 1] and state.tolist() == [2, 6, 2, 0]
