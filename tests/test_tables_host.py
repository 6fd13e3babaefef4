"""Device-side tables: host-side checks (no GPU) and the oracle against the
host block manager."""
import ctypes as C

import numpy as np

import paged_kv_cache_400_b200 as pk
from oracle import tables as ot
from paged_kv_cache_400_b200 import binding as bd

VP = C.c_void_p(16)  # never dereferenced: rejected before use


def test_workspace_size():
    L = bd.lib()
    assert L.pa_tables_workspace_size(-1) == 0 and L.pa_tables_workspace_size((1 << 20) + 1) == 0
    assert 0 < L.pa_tables_workspace_size(0) < L.pa_tables_workspace_size(1) < L.pa_tables_workspace_size(1 << 20)


def test_extend_refuses_on_host():
    L = bd.lib()
    need = L.pa_tables_workspace_size(4)

    def call(bt=VP, mb=4, sl=VP, nt=VP, ns=4, ring=VP, rs=8, st=VP, nb=8, lo=VP, qs=VP, sm=VP, n=64, row=0, so=VP,
             ws=VP, wb=need):
        return L.pa_tables_extend(bt, mb, sl, nt, ns, ring, rs, st, nb, lo, qs, sm, n, row, so, ws, wb, None)

    for kw in (dict(mb=0), dict(ns=-1), dict(rs=0), dict(nb=0), dict(n=-1), dict(row=-1), dict(row=17), dict(bt=None),
               dict(sl=None), dict(nt=None), dict(ring=None), dict(st=None), dict(lo=None), dict(qs=None),
               dict(sm=None), dict(so=None), dict(ws=C.c_void_p(18))):
        assert call(**kw) == 1, kw
    assert call(ns=(1 << 20) + 1) == 2 and call(mb=1 << 28) == 2
    assert call(rs=(1 << 30) + 1) == 2 and call(n=(1 << 30) + 1) == 2
    assert call(ws=None) == 9 and call(wb=need - 1) == 9


def test_release_refuses_on_host():
    L = bd.lib()
    need = L.pa_tables_workspace_size(4)

    def call(bt=VP, mb=4, sl=VP, fin=VP, ns=4, ring=VP, rs=8, st=VP, nb=8, lo=VP, so=VP, ws=VP, wb=need):
        return L.pa_tables_release(bt, mb, sl, fin, ns, ring, rs, st, nb, lo, so, ws, wb, None)

    for kw in (dict(mb=-1), dict(ns=-1), dict(rs=-1), dict(nb=0), dict(bt=None), dict(sl=None), dict(fin=None),
               dict(ring=None), dict(st=None), dict(lo=None), dict(so=None), dict(ws=C.c_void_p(17))):
        assert call(**kw) == 1, kw
    assert call(ns=(1 << 20) + 1) == 2
    assert call(ws=None) == 9 and call(wb=need - 4) == 9


def test_oracle_hands_out_the_block_managers_blocks():
    r = np.random.RandomState(1)
    N, B, W = 60, 6, 10
    bm = pk.BlockManager(N)
    ring, head, count = list(range(N)), 0, N
    tables, lens, ident, fresh = [[-1] * W for _ in range(B)], [0] * B, [None] * B, 0
    for _ in range(80):
        done = [int(n > 0 and r.rand() < 0.15) for n in lens]
        lens, st, err = ot.release(tables, lens, done, ring, head, count, N)
        head, count = st[:2]
        assert err == 0 and st[3] == 0
        for b in range(B):
            if done[b]:
                bm.free(ident[b])
        new = [int(r.randint(1, 40)) if n == 0 else int(n + 1 <= W * 16) for n in lens]
        had = list(lens)
        lens, start, slots, st, err = ot.extend(tables, lens, new, ring, head, count, N, sum(new), 0)
        head, count = st[:2]
        for b in range(B):
            got = slots[start[b]:start[b + 1]]
            if not got:
                continue
            if had[b] == 0:
                fresh += 1
                ident[b] = fresh
                bm.allocate(fresh, new[b])
                assert got == bm.slots(fresh, 0, new[b]).tolist()
            else:
                assert got == [bm.append_slot(ident[b])[0]]
            assert tables[b][: ot.pages(lens[b])] == bm.block_table(ident[b])
        assert count == bm.num_free()
