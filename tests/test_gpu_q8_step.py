"""The 8-bit cache and the device-side tables in use together: a step loop that
stays on the device, and the engine's step loop over 8-bit pools, each step's
results against the oracle."""
import numpy as np
import pytest
import torch

import paged_kv_cache_400_b200 as pk
from oracle import quantized as oq
from oracle import tables as ot
from paged_kv_cache_400_b200.engine import DecodeEngine, GraphedLayers

pytestmark = pytest.mark.gpu
DEV = "cuda"
HKV, G, D = 2, 4, 128
H = HKV * G
SCALE = D ** -0.5


def randn(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


class Cache:
    """The oracle's pool beside the device's."""

    def __init__(self, num_blocks, code):
        self.code = code
        self.codes = np.zeros((num_blocks, 2, HKV, 16, D), np.uint8)
        self.scales = np.zeros((num_blocks, 2, HKV), np.float32)

    def append(self, k, v, slots):
        oq.append(self.codes, self.scales, k.float().numpy(), v.float().numpy(), slots, self.code)

    def check_pool(self, pool, tables, lens):
        got_c, got_s = pool.codes.view(torch.uint8).cpu().numpy(), pool.scales.cpu().numpy()
        for t, n in zip(tables, lens):
            for pos in range(n):
                assert np.array_equal(got_c[t[pos // 16], :, :, pos % 16], self.codes[t[pos // 16], :, :, pos % 16])
            blk = np.asarray(t[: ot.pages(n)], int)
            assert np.array_equal(got_s[blk], self.scales[blk])

    def check_rows(self, out, q, table, length, decode):
        kv = oq.rows_of(self.codes, self.scales, table, length, self.code)
        ref, terms = oq.attention(q.double().numpy(), kv, SCALE, oq.scale_rows(self.scales, table, length))
        lim = oq.bound(ref, terms, D, length, "bf16", 2.0 ** -11, 2.0 ** -31, decode and self.code == "int8")
        err = np.abs(out.double().cpu().numpy() - ref)
        assert np.all(err <= lim), float((err / lim).max())


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_step_loop_on_the_device(code):
    """Admit, prefill, decode (one captured graph, lengths and ring updated in
    place, idle rows in the batch), release, admit again; the host only hands
    in the numbers of new tokens."""
    N, B, W = 40, 6, 10
    g = torch.Generator().manual_seed(3)
    r = np.random.RandomState(5)
    pool, cache = pk.Q8Pool(N, HKV, D, code), Cache(N, code)
    order = r.permutation(N).tolist()
    ring, state = pk.make_free_ring(N, order)
    o_ring, o_head, o_count = list(order), 0, N
    o_tables, o_lens = [[-1] * W for _ in range(B)], [0] * B
    tables = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    new = torch.zeros(B, dtype=torch.int32, device=DEV)
    qs = torch.empty(B + 1, dtype=torch.int32, device=DEV)
    tws = pk.alloc_tables_workspace(B)
    # the decode step's static buffers and its graph
    slots = torch.empty(B, dtype=torch.int64, device=DEV)
    q, out = (torch.zeros(B, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v = (torch.zeros(B, HKV, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ws = pk.alloc_workspace(B, H, pool, W * 16)

    def step():
        pk.pa_tables_extend(tables, lens, new, ring, state, lens, qs, slots, state, N, 1, tws)
        pk.pa_reshape_and_cache_q8(k, v, pool, slots)
        pk.pa_decode_q8(out, q, pool, tables, lens, SCALE, W * 16, ws)

    step()  # nothing asked for: kernels are set up, no state changes
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(3):
        ask = [int(r.randint(1, 60)) if n == 0 and r.rand() < 0.8 else 0 for n in o_lens]
        o_lens, start, o_slots, st, err = ot.extend(o_tables, o_lens, ask, o_ring, o_head, o_count, N, sum(ask), 0)
        o_head, o_count = st[:2]
        assert err == 0 and st[3] == 0
        T = sum(ask)
        if T:
            new.copy_(torch.tensor(ask, dtype=torch.int32))
            pslots = torch.empty(T, dtype=torch.int64, device=DEV)
            pk.pa_tables_extend(tables, lens, new, ring, state, lens, qs, pslots, state, N, 0, tws)
            pq, pkk, pv = randn(g, T, H, D), randn(g, T, HKV, D), randn(g, T, HKV, D)
            pk.pa_reshape_and_cache_q8(pkk.to(DEV), pv.to(DEV), pool, pslots)
            po = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
            pk.pa_prefill_q8(po, pq.to(DEV), pool, tables, lens, qs, SCALE, max(ask))
            cache.append(pkk, pv, o_slots)
            assert pslots.tolist() == o_slots and qs.tolist() == start
            for b in range(B):
                if ask[b]:
                    cache.check_rows(po[start[b]:start[b + 1]], pq[start[b]:start[b + 1]], o_tables[b], o_lens[b], False)
        for _ in range(20):
            ask = [int(n > 0) for n in o_lens]
            o_lens, start, o_slots, st, err = ot.extend(o_tables, o_lens, ask, o_ring, o_head, o_count, N, B, 1)
            o_head, o_count = st[:2]
            assert err == 0 and st[3] == 0
            new.copy_(torch.tensor(ask, dtype=torch.int32))
            hq, hk, hv = randn(g, B, H, D), randn(g, B, HKV, D) * 2, randn(g, B, HKV, D)
            q.copy_(hq), k.copy_(hk), v.copy_(hv)
            graph.replay()
            cache.append(hk, hv, o_slots)
            assert lens.tolist() == o_lens and slots.tolist() == o_slots and state.tolist() == st
            for b in range(B):
                if o_lens[b]:
                    cache.check_rows(out[b:b + 1], hq[b:b + 1], o_tables[b], o_lens[b], True)
                else:
                    assert not out[b].any()
        cache.check_pool(pool, o_tables, o_lens)
        done = [int(n > 0 and r.rand() < 0.5) for n in o_lens]
        o_lens, st, err = ot.release(o_tables, o_lens, done, o_ring, o_head, o_count, N)
        o_head, o_count = st[:2]
        new.copy_(torch.tensor(done, dtype=torch.int32))
        pk.pa_tables_release(tables, lens, new, ring, state, lens, state, N, tws)
        assert lens.tolist() == o_lens and state.tolist() == st
    assert pk.pa_get_device_error() == 0


@pytest.mark.parametrize("code,graphed,swap,cached", [("int8", False, 0, False), ("e4m3", True, 0, False),
                                                      ("int8", True, 12, False), ("e4m3", False, 0, True)])
def test_engine_over_8_bit_pools(code, graphed, swap, cached):
    """The step loop with preemption (recompute or swap), with prefix caching
    and with graphs: every step's outputs of both layers."""
    prompt = [30, 45, 17, 33, 50, 8]
    tokens = [[7] * 16 + list(range(100 * i, 100 * i + n - 16)) if n > 16 else list(range(n))
              for i, n in enumerate(prompt)] if cached else None
    eng = DecodeEngine(14, 2, H, HKV, D, [0, 0, 0, 1, 2, 3], prompt, [20, 25, 30, 12, 18, 9], 8, SCALE, DEV,
                       prompt_tokens=tokens, swap_host_blocks=swap, kv_code=code)
    run = GraphedLayers(eng, 6, 2).run if graphed else eng.run_layers
    g = torch.Generator().manual_seed(1)
    caches = [Cache(14, code) for _ in range(2)]
    hosts = [Cache(max(swap, 1), code) for _ in range(2)]
    preempted = steps = 0
    while True:
        idx = eng.schedule()
        if idx.done and not len(idx.running):
            break
        steps += 1
        assert steps < 200
        preempted += idx.record.preempted
        n, T = len(idx.running), len(idx.prompt_slots)
        if n == 0:
            continue
        x = [dict(q=randn(g, n, H, D), k_dec=randn(g, n, HKV, D), v_dec=randn(g, n, HKV, D),
                  k_prompt=randn(g, T, HKV, D), v_prompt=randn(g, T, HKV, D), q_prompt=randn(g, T, H, D))
             for _ in range(2)]
        if cached:  # requests with a common prefix bring the same K and V there
            reqs, pos = eng.prompt_positions(idx)
            for l in range(2):
                fixed = torch.Generator().manual_seed(50 + l)
                shared = randn(fixed, 2, 16, HKV, D)
                for i, (rq, ps) in enumerate(zip(reqs, pos)):
                    if ps < 16 and prompt[int(rq)] > 16:
                        x[l]["k_prompt"][i], x[l]["v_prompt"][i] = shared[0, ps], shared[1, ps]
        outs = run(idx, [{a: b.to(DEV) for a, b in d.items()} for d in x])
        for l in range(2):
            c, h = caches[l], hosts[l]
            for a, b in idx.swap_out:
                h.codes[b], h.scales[b] = c.codes[a], c.scales[a]
            for a, b in idx.swap_in:
                c.codes[b], c.scales[b] = h.codes[a], h.scales[a]
            for a, b in zip(idx.cow_src, idx.cow_dst):
                c.codes[b], c.scales[b] = c.codes[a], c.scales[a]
            c.append(x[l]["k_prompt"], x[l]["v_prompt"], idx.prompt_slots)
            row = {int(rq): i for i, rq in enumerate(idx.running)}
            at = 0
            for rq, n0, st in zip(idx.prompt_seqs, idx.prompt_lens, idx.prompt_starts):
                m = int(n0 - st)
                if m:
                    c.check_rows(eng.prefill_out[l][at:at + m], x[l]["q_prompt"][at:at + m],
                                 idx.block_tables[row[int(rq)]], int(n0), False)
                at += m
            c.append(x[l]["k_dec"], x[l]["v_dec"], idx.decode_slots)
            for i in range(n):
                c.check_rows(outs[l][i:i + 1], x[l]["q"][i:i + 1], idx.block_tables[i], int(idx.seq_lens[i]), True)
        if idx.done:
            break
    assert preempted > 0 or cached
    assert pk.pa_get_device_error() == 0
    eng.close()
