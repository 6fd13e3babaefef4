"""Block tables, lengths and slot maps built on the GPU: equal to the oracle's
and to the host block manager's, entry by entry."""
import numpy as np
import pytest
import torch

import paged_kv_cache_400_b200 as pk
from oracle import tables as ot

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x, np.int64).tolist(), dtype=torch.int32, device=DEV)


def make(lens, width, num_blocks, seed=0, ring_size=None, head=None):
    """Tables of distinct blocks for the lengths, the rest of the blocks in a ring that starts at head."""
    r = np.random.RandomState(seed)
    perm = r.permutation(num_blocks).tolist()
    t = np.full((len(lens), width), -1, np.int64)
    for b, n in enumerate(lens):
        k = min(max(ot.pages(int(n)), 0), width)
        t[b, :k] = [perm.pop() for _ in range(k)]
    size = ring_size or num_blocks
    ring = np.full(size, -1, np.int64)
    head = r.randint(size) if head is None else head
    for i, x in enumerate(perm):
        ring[(head + i) % size] = x
    return t, ring, head, len(perm)


def check_extend(lens, new, width, num_blocks, row_tokens=0, num_slots=None, seed=0, alias=False, count=None,
                 head=None, edit=None):
    B = len(lens)
    t, ring, h, c = make(lens, width, num_blocks, seed, head=head)
    c = c if count is None else count
    if edit:
        edit(t, ring)
    if num_slots is None:
        num_slots = B * row_tokens if row_tokens else max(0, int(sum(x for x in new if x > 0))) + 5
    want_t = t.tolist()
    want = ot.extend(want_t, [int(x) for x in lens], [int(x) for x in new], ring.tolist(), h, c, num_blocks, num_slots,
                     row_tokens)
    dt, dl, dr, ds = i32(t).reshape(B, width), i32(lens), i32(ring), i32([h, c, 77, 78])
    lo = dl if alias else torch.full((B,), -9, dtype=torch.int32, device=DEV)
    so = ds if alias else torch.full((4,), -9, dtype=torch.int32, device=DEV)
    qs = torch.full((B + 1,), -9, dtype=torch.int32, device=DEV)
    slots = torch.full((num_slots,), -9, dtype=torch.int64, device=DEV)
    pk.pa_tables_extend(dt, dl, i32(new), dr, ds, lo, qs, slots, so, num_blocks, row_tokens,
                        pk.alloc_tables_workspace(B))
    assert pk.pa_get_device_error() == want[4]
    assert so.tolist() == want[3]
    assert lo.tolist() == want[0]
    assert qs.tolist() == want[1]
    assert dt.tolist() == want_t
    assert slots.tolist() == want[2]
    assert dr.tolist() == ring.tolist()
    return want


def check_release(lens, done, width, num_blocks, seed=0, ring_size=None, alias=False, edit=None, head=None, count=None):
    B = len(lens)
    t, ring, h, c = make(lens, width, num_blocks, seed, ring_size, head)
    c = c if count is None else count
    if edit:
        edit(t, ring)
    want_ring = ring.tolist()
    want = ot.release(t.tolist(), [int(x) for x in lens], [int(x) for x in done], want_ring, h, c, num_blocks)
    dt, dl, dr, ds = i32(t).reshape(B, width), i32(lens), i32(ring), i32([h, c, 77, 78])
    lo = dl if alias else torch.full((B,), -9, dtype=torch.int32, device=DEV)
    so = ds if alias else torch.full((4,), -9, dtype=torch.int32, device=DEV)
    pk.pa_tables_release(dt, dl, i32(done), dr, ds, lo, so, num_blocks, pk.alloc_tables_workspace(B))
    assert pk.pa_get_device_error() == want[2]
    assert so.tolist() == want[1]
    assert lo.tolist() == want[0]
    assert dr.tolist() == want_ring
    assert dt.tolist() == t.tolist()
    return want


SIZES = [1, 2, 31, 33, 256, 1000, 1024, 1025, 2048, 2049, 5000]


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("batch", SIZES)
def test_extend_decode_step(batch, alias):
    r = np.random.RandomState(batch)
    lens = r.randint(0, 300, batch)
    check_extend(lens, np.ones(batch, int), 19, int(ot.pages(300)) * batch + 40, 1, seed=batch, alias=alias)


@pytest.mark.parametrize("batch", SIZES)
def test_extend_prompts_packed(batch):
    """Zero to 90 tokens each (sparse batches among them), on fresh and running requests."""
    r = np.random.RandomState(batch + 1)
    lens = np.where(r.rand(batch) < 0.5, 0, r.randint(0, 50, batch))
    new = np.where(r.rand(batch) < 0.3, 0, r.randint(0, 91, batch))
    check_extend(lens, new, 9, batch * 9 + 3, seed=batch, alias=batch % 2 == 0)


@pytest.mark.parametrize("batch,row", [(1, 7), (40, 33), (300, 16), (700, 40), (3000, 5)])
def test_extend_rows(batch, row):
    """Padded rows, some of them empty."""
    r = np.random.RandomState(batch)
    check_extend(r.randint(0, 60, batch), r.randint(0, row + 1, batch), 8, batch * 8, row, batch * row + 11, seed=batch)


@pytest.mark.parametrize("batch", [5, 1500, 4000])
def test_extend_few_long(batch):
    """One request takes most positions: the search meets many empty ones."""
    new = np.zeros(batch, int)
    new[batch // 2], new[batch - 1] = 20000, 17
    check_extend(np.zeros(batch, int), new, 1250, 1300, seed=1)


@pytest.mark.parametrize("row", [0, 4])
@pytest.mark.parametrize("batch", [6, 1500, 3000])
def test_extend_runs_out_of_blocks(batch, row):
    """Requests behind the ring's end get nothing; those that need no block go on."""
    r = np.random.RandomState(batch)
    lens, new = r.randint(0, 40, batch), r.randint(0, 5, batch)
    check_extend(lens, new, 4, batch * 4, row, seed=3, count=batch // 20 + 1)
    check_extend(lens, new, 4, batch * 4, row, seed=3, count=0)


@pytest.mark.parametrize("batch", [9, 3000])
def test_extend_runs_out_of_slots(batch):
    r = np.random.RandomState(batch)
    check_extend(r.randint(0, 40, batch), r.randint(0, 9, batch), 4, batch * 4, 0, 3 * batch, seed=4)
    check_extend(r.randint(0, 40, batch), r.randint(0, 9, batch), 4, batch * 4, 0, 0, seed=4)


@pytest.mark.parametrize("row", [0, 3])
@pytest.mark.parametrize("batch", [12, 3000])
def test_extend_bad_requests(batch, row):
    r = np.random.RandomState(batch)
    lens, new = r.randint(0, 40, batch), r.randint(0, 4, batch)
    lens[1], new[3], lens[5], new[7] = -4, -1, 64, 65
    lens[8], new[8] = 2147483647, 2147483647
    check_extend(lens, new, 4, batch * 4, row, 4 * batch, seed=5)


def test_extend_bad_blocks_and_state():
    def edit(t, ring):
        t[0, 0], ring[3], ring[4] = -1, 999, -5
    check_extend([5, 16, 16, 16], [2, 1, 1, 1], 3, 40, 1, head=2, edit=edit)
    for h, c in ((-1, 3), (40, 3), (0, 41), (0, -1)):
        check_extend([5, 16, 15], [2, 1, 1], 3, 40, 0, 9, head=h % 40, count=c) if 0 <= h < 40 else None
    ds = i32([40, 3, 0, 0])
    lo, qs, sl = i32([0]), i32([0, 0]), torch.zeros(2, dtype=torch.int64, device=DEV)
    pk.pa_tables_extend(i32([[-1]]), i32([0]), i32([1]), i32(range(40)), ds, lo, qs, sl, ds, 40)
    assert pk.pa_get_device_error() == pk.PA_DEVERR_BLOCK
    assert ds.tolist() == [40, 3, 0, 1] and lo.tolist() == [0] and sl.tolist() == [-1, -1]


def test_empty_batch():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    ring, state = pk.make_free_ring(8)
    so, qs, sl = i32([9] * 4), i32([9]), torch.full((3,), 9, dtype=torch.int64, device=DEV)
    pk.pa_tables_extend(e.reshape(0, 4), e, e, ring, state, e, qs, sl, so, 8)
    assert so.tolist() == [0, 8, 0, 0] and qs.tolist() == [0] and sl.tolist() == [-1] * 3
    pk.pa_tables_release(e.reshape(0, 4), e, e, ring, state, e, so, 8)
    assert so.tolist() == [0, 8, 0, 0] and pk.pa_get_device_error() == 0


@pytest.mark.parametrize("share", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("batch", SIZES)
def test_release(batch, share):
    r = np.random.RandomState(batch)
    lens = np.where(r.rand(batch) < 0.1, 0, r.randint(0, 200, batch))
    check_release(lens, (r.rand(batch) < share) * r.randint(-3, 4, batch), 13, batch * 13 + 5, seed=batch,
                  alias=batch % 2 == 1)


@pytest.mark.parametrize("batch", [7, 1500, 3000])
def test_release_into_a_full_ring(batch):
    r = np.random.RandomState(batch)
    lens = r.randint(0, 60, batch)
    held = int(ot.pages(lens).sum())
    check_release(lens, np.ones(batch, int), 4, held + 10, seed=2, ring_size=10 + held // 2)


def test_release_bad_requests():
    def edit(t, ring):
        t[2, 1] = 40
    check_release([20, -1, 33, 64, 65, 7], [1, 1, 1, 1, 1, 0], 4, 40, edit=edit)
    check_release([20, 33], [1, 1], 4, 40, head=39, count=41)


@pytest.mark.parametrize("batch,row", [(40, 1), (700, 4), (2500, 3), (5000, 1)])
def test_captured_steps_in_place(batch, row):
    """Lengths and ring advanced in place by a replayed graph (one launch, two launches, sums in the
    workspace), then released by another that shares the workspace."""
    W, N = 4, batch * 4
    r = np.random.RandomState(batch)
    t, ring, h, c = make(np.zeros(batch, int), W, N, batch)
    o_t, o_l, o_r = t.tolist(), [0] * batch, ring.tolist()
    dt, dl, dr, ds = i32(t).reshape(batch, W), i32([0] * batch), i32(ring), i32([h, c, 0, 0])
    ask, qs = i32([0] * batch), i32([0] * (batch + 1))
    slots = torch.zeros(batch * row, dtype=torch.int64, device=DEV)
    ws = pk.alloc_tables_workspace(batch)
    up = lambda: pk.pa_tables_extend(dt, dl, ask, dr, ds, dl, qs, slots, ds, N, row, ws)
    down = lambda: pk.pa_tables_release(dt, dl, ask, dr, ds, dl, ds, N, ws)
    up(), down()  # nothing asked for: no state changes
    torch.cuda.synchronize()
    graphs = []
    for f in (up, down):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for step in range(6):
        if step == 3:
            done = (r.rand(batch) < 0.4).astype(int).tolist()
            ask.copy_(torch.tensor(done, dtype=torch.int32))
            graphs[1].replay()
            o_l, st, err = ot.release(o_t, o_l, done, o_r, h, c, N)
        else:
            new = r.randint(0, row + 1, batch).tolist()
            ask.copy_(torch.tensor(new, dtype=torch.int32))
            graphs[0].replay()
            o_l, start, o_s, st, err = ot.extend(o_t, o_l, new, o_r, h, c, N, batch * row, row)
            assert slots.tolist() == o_s and qs.tolist() == start
        h, c = st[:2]
        assert err == 0 and dl.tolist() == o_l and ds.tolist() == st and dr.tolist() == o_r
        assert dt.tolist() == o_t
    assert pk.pa_get_device_error() == 0


def test_same_blocks_as_the_host_block_manager():
    """Requests come, grow and leave: tables, lengths and slots stay the host block manager's."""
    r = np.random.RandomState(0)
    N, B, W = 120, 12, 12
    order = r.permutation(N).tolist()
    bm = pk.BlockManager(N, order)
    ring, state = pk.make_free_ring(N, order)
    tables = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    qs = torch.empty(B + 1, dtype=torch.int32, device=DEV)
    ws = pk.alloc_tables_workspace(B)
    have, ident, fresh = [0] * B, [None] * B, 0
    for step in range(60):
        done = [int(h > 0 and r.rand() < 0.1) for h in have]
        pk.pa_tables_release(tables, lens, i32(done), ring, state, lens, state, N, ws)
        for b in range(B):
            if done[b]:
                bm.free(ident[b])
                have[b], ident[b] = 0, None
        new = [int(r.randint(1, 70)) if h == 0 and r.rand() < 0.6 else int(h > 0) for h in have]
        room = bm.num_free()
        for b in range(B):  # what the step can hold
            need = ot.pages(have[b] + new[b]) - ot.pages(have[b])
            if need > room or have[b] + new[b] > W * 16:
                new[b] = 0
            else:
                room -= need
        slots = torch.empty(max(1, sum(new)), dtype=torch.int64, device=DEV)
        pk.pa_tables_extend(tables, lens, i32(new), ring, state, lens, qs, slots, state, N, 0, ws)
        want = []
        for b in range(B):
            if new[b] and have[b] == 0:
                fresh += 1
                ident[b] = fresh
                bm.allocate(fresh, new[b])
                want += bm.slots(fresh, 0, new[b]).tolist()
            elif new[b]:
                want.append(bm.append_slot(ident[b])[0])
            have[b] += new[b]
        assert pk.pa_get_device_error() == 0
        assert slots[: len(want)].tolist() == want
        assert lens.tolist() == have and state[1].item() == bm.num_free()
        host = tables.cpu().numpy()
        for b in range(B):
            if have[b]:
                assert host[b, : ot.pages(have[b])].tolist() == bm.block_table(ident[b])


def test_refusals():
    ring, state = pk.make_free_ring(8)
    a = dict(block_tables=i32([[-1] * 4] * 2), seq_lens=i32([0, 0]), new_tokens=i32([1, 1]), free_ring=ring,
             ring_state=state, seq_lens_out=i32([0, 0]), query_start=i32([0] * 3),
             slot_mapping=torch.zeros(4, dtype=torch.int64, device=DEV), ring_state_out=i32([0] * 4), num_blocks=8)
    pk.pa_tables_extend(**a)
    for bad in (dict(seq_lens=a["seq_lens"].long()), dict(new_tokens=i32([1])), dict(query_start=i32([0] * 2)),
                dict(ring_state_out=i32([0] * 3)), dict(slot_mapping=a["slot_mapping"].int()),
                dict(free_ring=ring.cpu()), dict(block_tables=i32([[-1] * 8] * 2)[:, ::2])):
        with pytest.raises(ValueError):
            pk.pa_tables_extend(**{**a, **bad})
    for bad in (dict(row_tokens=3), dict(row_tokens=-1), dict(num_blocks=0)):
        with pytest.raises(pk.PagedKVError) as e:
            pk.pa_tables_extend(**{**a, **bad})
        assert e.value.status == "INVALID_ARG"
    with pytest.raises(pk.PagedKVError) as e:
        pk.pa_tables_extend(**a, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    assert e.value.status == "WORKSPACE"
    with pytest.raises(ValueError):
        pk.alloc_tables_workspace((1 << 20) + 1)
