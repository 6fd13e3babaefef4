"""8-bit pools on the GPU: append and block copies bit for bit against the
oracle, attention within the bound that follows from its roundings."""
import numpy as np
import pytest
import torch

import paged_kv_cache_400_b200 as pk
from oracle import quantized as oq

pytestmark = pytest.mark.gpu
DEV = "cuda"
IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def make_pool(num_blocks, heads, dim, code, seed=0, spread=0.5):
    """A pool of random live codes (never NaN) and scales of differing size."""
    r = np.random.RandomState(seed)
    p = pk.Q8Pool(num_blocks, heads, dim, code)
    c = r.randint(0, 256, (num_blocks, 2, heads, 16, dim)).astype(np.uint8)
    c[c == (128 if code == "int8" else 127)] = 3
    if code == "e4m3":
        c[c == 255] = 130
    s = (np.exp(spread * r.randn(num_blocks, 2, heads)) / (60 if code == "int8" else 150)).astype(np.float32)
    p.codes.view(torch.uint8).copy_(torch.from_numpy(c))
    p.scales.copy_(torch.from_numpy(s))
    return p


def host(p):
    return p.codes.view(torch.uint8).cpu().numpy().copy(), p.scales.cpu().numpy().copy()


def rows(n, heads, dim, io, seed=0, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, dim, generator=g) * torch.exp(amp * torch.randn(n, 1, 1, generator=g))).to(IO[io])


def check_append(p, k, v, slots, want_error=0):
    codes, scales = host(p)
    oq.append(codes, scales, k.float().numpy(), v.float().numpy(), slots, p.code)
    rest = p.buf.clone()
    pk.pa_reshape_and_cache_q8(k.to(DEV), v.to(DEV), p, torch.as_tensor(slots, dtype=torch.int64, device=DEV))
    assert pk.pa_get_device_error() == want_error
    got_c, got_s = host(p)
    assert np.array_equal(got_s.view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(got_c, codes)
    raw = codes[0].size + 8 * p.num_kv_heads
    assert torch.equal(p.buf[:, raw:], rest[:, raw:])  # the padding stays


CODE = pytest.mark.parametrize("code", ["int8", "e4m3"])


# ---- append ----------------------------------------------------------------------
@CODE
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 128), (8, 128), (5, 64)])
def test_append_prompts(heads, dim, io, code):
    """Sequences with whole blocks, ragged ends, a start inside a block, one token."""
    p = make_pool(40, heads, dim, code, seed=heads)
    perm = np.random.RandomState(1).permutation(40)
    slots, at = [], 0
    for start, n in [(0, 16), (0, 1), (5, 60), (15, 1), (0, 33), (7, 9), (3, 2), (0, 47)]:
        pos = np.arange(start, start + n)
        slots += (perm[at + pos // 16] * 16 + pos % 16).tolist()
        at += pos[-1] // 16 + 1
    assert at <= 40
    check_append(p, rows(len(slots), heads, dim, io, 2), rows(len(slots), heads, dim, io, 3), slots)


@CODE
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_append_one_token_after_another(code, io):
    """A block filled in 16 calls of growing rows: its scale grows, earlier rows are coded again."""
    p = make_pool(4, 2, 128, code, seed=5)
    for r in range(16):
        k = rows(1, 2, 128, io, 10 + r) * 1.2 ** r
        v = rows(1, 2, 128, io, 50 + r) * (1.0 if r % 3 else 4.0)
        check_append(p, k, v, [2 * 16 + r])


@CODE
def test_append_many_sequences_one_token(code):
    """A decode step: 300 sequences, every row index, a token each (several tokens per warp)."""
    p = make_pool(300, 8, 128, code, seed=7)
    slots = np.random.RandomState(3).permutation(300) * 16 + np.random.RandomState(4).randint(0, 16, 300)
    check_append(p, rows(300, 8, 128, "bf16", 8), rows(300, 8, 128, "bf16", 9), slots)


@CODE
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 700])
def test_append_lengths_of_the_list(n, code):
    p = make_pool(64, 2, 64, code, seed=n)
    check_append(p, rows(n, 2, 64, "f32", 1), rows(n, 2, 64, "f32", 2), np.arange(3, 3 + n))


@CODE
def test_append_padding_and_order(code):
    """Padding between a block's tokens, rows in falling order, a row named twice."""
    p = make_pool(8, 2, 64, code, seed=1)
    slots = [-1, 16 + 9, -1, -1, 16 + 8, 16 + 7, -1, 16 + 9, -5, 48 + 0, -1, 48 + 2, 48 + 1, -1, 48 + 0, -1]
    check_append(p, rows(16, 2, 64, "bf16", 1), rows(16, 2, 64, "bf16", 2), slots)


@CODE
def test_append_zeros_tiny_huge(code):
    """Tiles of zeros, magnitudes below 2^-100, near the largest finite, and a tile that stays."""
    p = make_pool(8, 1, 64, code, seed=2)
    k = torch.zeros(64, 1, 64)
    k[16:32] = 1e-32
    k[32:48] = 3e38 * torch.linspace(-1, 1, 64)
    k[48] = 1e-38
    check_append(p, k, k.clone(), np.concatenate([np.arange(48), np.arange(49, 65)]))
    # growing from a scale of 0, and rows too small to change anything
    check_append(p, torch.full((1, 1, 64), 1.5), torch.full((1, 1, 64), 2.0 ** -101), [5])
    check_append(p, torch.full((1, 1, 64), 1e-6), torch.full((1, 1, 64), -3.0), [6])


@CODE
def test_append_non_finite(code):
    p = make_pool(4, 2, 64, code, seed=3)
    k, v = rows(5, 2, 64, "f32", 1), rows(5, 2, 64, "f32", 2)
    k[1, 0, 3], k[2, 1, 5], v[4, 0, 0] = float("nan"), float("inf"), -float("inf")
    check_append(p, k, v, [0, 1, 2, 35, 36], pk.PA_DEVERR_NONFINITE)


def test_append_bad_slots():
    p = make_pool(4, 2, 64, "int8", seed=4)
    k = rows(4, 2, 64, "f32", 1)
    codes, scales = host(p)
    oq.append(codes, scales, k.numpy(), k.numpy(), [16, -1, 17, -1], "int8")
    pk.pa_reshape_and_cache_q8(k.to(DEV), k.to(DEV), p, torch.tensor([16, 64, 17, 1 << 40], device=DEV))
    assert pk.pa_get_device_error() == pk.PA_DEVERR_SLOT
    assert np.array_equal(host(p)[0], codes) and np.array_equal(host(p)[1], scales)

@CODE
@pytest.mark.parametrize("lead", [0, 1, 14, 15, 16, 37])
def test_append_tokens_far_apart(lead, code):
    """A block's tokens over several windows of 32 entries, each within 31 of the one before; rows
    named again; a neighbour block in between."""
    p = make_pool(6, 2, 64, code, seed=4)
    slots = [-1] * lead + [16 + 3] + [-1] * 30 + [16 + 9] + [32 + i for i in range(16)] + [16 + 3] + [-1] * 30 \
        + [16 + 4, 16 + 0] + [-1] * 25 + [16 + 9] + [-1] * 40
    check_append(p, rows(len(slots), 2, 64, "f32", 2), rows(len(slots), 2, 64, "f32", 3), slots)


@CODE
@pytest.mark.parametrize("gap", [0, 7, 15, 16, 31, 60, 200])
def test_append_shared_prefix_in_one_call(gap, code):
    """Two requests of a step write the same blocks with the same values, at any distance."""
    p = make_pool(40, 2, 128, code, seed=5)
    k, v = rows(32 + gap + 40, 2, 128, "bf16", 6), rows(32 + gap + 40, 2, 128, "bf16", 7)
    k[32 + gap:64 + gap], v[32 + gap:64 + gap] = k[:32], v[:32]
    slots = list(range(32)) + list(range(100, 100 + gap)) + list(range(32)) + list(range(400, 408))
    check_append(p, k, v, slots)


@CODE
def test_copies_take_scales(code):
    p = make_pool(12, 3, 64, code, seed=6)
    want = p.buf.clone()
    want[[7, 2]] = want[[1, 11]]
    pk.pa_copy_blocks(p, torch.tensor([1, 11], dtype=torch.int32, device=DEV),
                      torch.tensor([7, 2], dtype=torch.int32, device=DEV))
    assert pk.pa_get_device_error() == 0 and torch.equal(p.buf, want)
    far = pk.Q8Pool.wrap(torch.zeros(5, p.buf.shape[1], dtype=torch.uint8).pin_memory(), 3, 64, code)
    src, dst = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([7, 0, 3], [4, 0, 2]))
    pk.pa_copy_blocks_between(far, p, src, dst)
    torch.cuda.synchronize()
    assert torch.equal(far.buf[[4, 0, 2]], p.buf[[7, 0, 3]].cpu())
    back = make_pool(12, 3, 64, code, seed=9)
    pk.pa_copy_blocks_between(back, far, dst, src)
    assert pk.pa_get_device_error() == 0 and torch.equal(back.buf[[7, 0, 3]], p.buf[[7, 0, 3]])


# ---- decode ----------------------------------------------------------------------
def tables_for(lens, num_blocks, width=None, seed=0):
    r = np.random.RandomState(seed)
    need = [(n + 15) // 16 for n in lens]
    width = width or max(1, max(need))
    t = np.full((len(lens), width), -1, np.int32)
    perm = r.permutation(num_blocks)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t


def poison(p, tables, lens):
    """Everything no sequence owns becomes NaN where a code can be one, and large otherwise."""
    codes, scales = host(p)
    bad = 127 if p.code == "e4m3" else 129
    live = np.zeros((p.num_blocks, 16), bool)
    for t, n in zip(tables, lens):
        pos = np.arange(n)
        live[t[pos // 16], pos % 16] = True
    codes = np.where(live[:, None, None, :, None], codes, np.uint8(bad))
    scales = np.where(live.any(1)[:, None, None], scales, np.float32(np.nan))
    p.codes.view(torch.uint8).copy_(torch.from_numpy(codes))
    p.scales.copy_(torch.from_numpy(scales))
    return codes, scales


def check_rows(got, q, lens, news, starts, codes, scales, tables, p, io, scale, p_rounding, chain,
               p_floor=2.0 ** -31, biased=False):
    got = got.double().cpu().numpy()
    for b, (n, new) in enumerate(zip(lens, news)):
        r = slice(starts[b], starts[b] + new)
        if n == 0:
            assert not got[r].any()
            continue
        kv = oq.rows_of(codes, scales, tables[b], n, p.code)
        ref, terms = oq.attention(q[r].double().numpy(), kv, scale, oq.scale_rows(scales, tables[b], n))
        err = np.abs(got[r] - ref)
        lim = oq.bound(ref, terms, p.head_dim, min(n, chain), io, p_rounding, p_floor, biased)
        assert np.all(err <= lim), (b, n, float((err / lim).max()))


def decode(p, q, tables, lens, max_len, scale, stream=None):
    q = q.to(DEV)
    out = torch.full_like(q, float("nan"))
    ws = pk.alloc_workspace(len(lens), q.shape[1], p, max_len)
    if ws is not None:
        ws.fill_(255)
    pk.pa_decode_q8(out, q, p, torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                    scale, max_len, ws, stream)
    return out


def biased(code, io):
    return code == "int8" and io == "bf16"  # decode sums such codes as code + 128


def check_decode(heads_kv, group, dim, code, io, lens, max_len=None, spread=0.5, seed=0, want_error=0):
    max_len = max_len or max(1, max(lens))
    width = (max_len + 15) // 16
    blocks = sum((n + 15) // 16 for n in lens) + 3
    p = make_pool(blocks, heads_kv, dim, code, seed, spread)
    tables = tables_for(lens, blocks, width, seed)
    codes, scales = poison(p, tables, lens)
    q = rows(len(lens), heads_kv * group, dim, io, seed + 1, 0.3)
    out = decode(p, q, tables, lens, max_len, dim ** -0.5)
    assert pk.pa_get_device_error() == want_error
    # a chain of sums: 32 blocks of 16 tokens in a warp, its 4 warps, the partitions
    check_rows(out, q, lens, [1] * len(lens), range(len(lens)), codes, scales, tables, p, io, dim ** -0.5,
               2.0 ** -11 if io == "bf16" else 2.0 ** -22, 32 * 16 + 4 + (max_len + 127) // 128,
               biased=biased(code, io))


LENS = [1, 0, 15, 16, 17, 31, 33, 64, 65, 100, 128, 129, 255, 511, 513]


@CODE
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads_kv,group", [(1, 1), (3, 2), (2, 4), (1, 7), (2, 8), (1, 9), (2, 16)])
def test_decode_shapes(heads_kv, group, dim, io, code):
    check_decode(heads_kv, group, dim, code, io, LENS, seed=group)


@CODE
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads_kv,group,dim", [(8, 4, 128), (2, 1, 64), (1, 12, 128)])
def test_decode_partitions(heads_kv, group, dim, io, code):
    """Long sequences beside short and empty ones: partitions, the work list, the merge."""
    check_decode(heads_kv, group, dim, code, io, [5000, 1, 0, 2047, 2048, 2049, 127, 129, 3333, 16], seed=3)
    check_decode(heads_kv, group, dim, code, io, [300], max_len=9000, seed=4)
    check_decode(heads_kv, group, dim, code, io, [20011], seed=5)


@CODE
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_decode_scales_far_apart(code, io):
    """Tile scales over some 30 binades, V and K each for itself."""
    check_decode(2, 4, 128, code, io, [1, 16, 40, 200, 1000], spread=5.0, seed=11)
    check_decode(2, 1, 64, code, io, [1, 16, 40, 200, 1000], spread=5.0, seed=12)


@CODE
def test_decode_zero_scales(code):
    p = make_pool(20, 2, 128, code, 1)
    lens = [100, 33]
    tables = tables_for(lens, 20, 7)
    p.scales[torch.from_numpy(tables[0, :3]).long().to(DEV)] = 0          # zero K and V tiles
    p.scales[torch.from_numpy(tables[1, :3]).long().to(DEV), 1] = 0       # every V tile zero
    codes, scales = host(p)
    q = rows(2, 8, 128, "bf16", 3)
    out = decode(p, q, tables, lens, 112, 0.1)
    assert pk.pa_get_device_error() == 0
    check_rows(out, q, lens, [1, 1], [0, 1], codes, scales, tables, p, "bf16", 0.1, 2.0 ** -11, 100,
               biased=biased(code, "bf16"))
    assert not out[1].any()


@CODE
@pytest.mark.parametrize("max_len", [64, 5000])
def test_decode_bad_blocks_and_lengths(code, max_len):
    p = make_pool(40, 2, 64, code, 1)
    lens = [40, 64, -3, max_len + 1, 33]
    tables = tables_for([40, 64, 16, 16, 33], 40, (max_len + 15) // 16)
    good = tables.copy()
    q = rows(5, 4, 64, "f32", 3)
    out = decode(p, q, tables, lens, max_len, 0.1)
    assert pk.pa_get_device_error() == pk.PA_DEVERR_SEQLEN
    assert not out[2:4].any() and torch.isfinite(out).all()
    codes, scales = host(p)
    ok = [0, 1, 4]
    check_rows(out[ok], q[ok], [40, 64, 33], [1] * 3, range(3), codes, scales, good[ok], p, "f32", 0.1, 2.0 ** -22, 64)
    tables[0, 1], tables[4, 0] = 40, -7
    out2 = decode(p, q, tables, [40, 64, 0, 0, 33], max_len, 0.1)
    assert pk.pa_get_device_error() == pk.PA_DEVERR_BLOCK
    assert torch.equal(out2[1], out[1]) and torch.isfinite(out2).all()


@CODE
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("heads_kv,group,dim", [(8, 2, 128), (8, 1, 64), (8, 9, 128)])
def test_decode_large_ragged_batch(heads_kv, group, dim, io, code):
    """More partitions than three rounds of CTAs: the list of the plan kernel, empty sequences among them."""
    r = np.random.RandomState(2)
    lens = r.randint(0, 40, 300)
    lens[[3, 77, 150, 299]] = [2100, 2049, 2048, 4000]
    check_decode(heads_kv, group, dim, code, io, lens.tolist(), max_len=4096, seed=6)


@CODE
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
def test_decode_many_short_sequences(dim, io, code):
    """A warp for each sequence and KV head: lengths over the ring's stages, empty and longest ones."""
    r = np.random.RandomState(3)
    lens = r.randint(0, 70, 130)
    lens[:6] = [0, 1, 512, 511, 497, 64]
    check_decode(4, 3, dim, code, io, lens.tolist(), max_len=512, seed=7)
    check_decode(4, 9, dim, code, io, np.minimum(lens, 30).tolist(), max_len=30, seed=8)


@CODE
@pytest.mark.parametrize("max_len", [200, 3000])
def test_decode_scale_of_any_sign(code, max_len):
    lens = [40, 200, 1, 17]
    p = make_pool(30, 2, 64, code, 4)
    tables = tables_for(lens, 30, (max_len + 15) // 16)
    codes, scales = host(p)
    q = rows(4, 8, 64, "bf16", 3)
    for scale in (-0.2, 0.0, 5.0):
        out = decode(p, q, tables, lens, max_len, scale)
        assert pk.pa_get_device_error() == 0
        check_rows(out, q, lens, [1] * 4, range(4), codes, scales, tables, p, "bf16", scale, 2.0 ** -11, 200,
                   biased=biased(code, "bf16"))


@CODE
@pytest.mark.parametrize("max_len", [200, 3000])
def test_decode_non_finite_queries_stay_in_their_head(code, max_len):
    lens = [40, 200, 1, 17]
    p = make_pool(30, 2, 64, code, 4)
    tables = tables_for(lens, 30, (max_len + 15) // 16)
    q = rows(4, 8, 64, "f32", 3)
    want = decode(p, q, tables, lens, max_len, 0.1)
    q[1, 2, 5], q[3, 7, 0], q[0, 4, 1] = float("nan"), float("inf"), -float("inf")
    got = decode(p, q, tables, lens, max_len, 0.1)
    hit = torch.zeros(4, 8, dtype=torch.bool)
    hit[1, 2] = hit[3, 7] = hit[0, 4] = True
    assert torch.equal(got[~hit], want[~hit]) and not torch.isfinite(got[hit]).all(-1).any()
    assert pk.pa_get_device_error() == 0


def test_calls_on_two_streams_at_once():
    """Two requests' steps side by side, each with buffers and a workspace of its own."""
    lens = [3000, 70, 1500, 900]
    sets = []
    for i in range(2):
        p = make_pool(400, 4, 128, "int8", 20 + i)
        sets.append((p, torch.from_numpy(tables_for(lens, 400, 188, i)).to(DEV), rows(4, 16, 128, "bf16", 30 + i).to(DEV),
                     rows(40, 4, 128, "bf16", 40 + i).to(DEV), pk.alloc_workspace(4, 16, p, 3008), torch.cuda.Stream()))
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    slots = torch.arange(16 * 399 - 24, 16 * 400 - 24, device=DEV).repeat(3)[:40]

    def step(s, n):
        p, t, q, k, ws, _ = s
        outs = []
        for _ in range(n):
            pk.pa_reshape_and_cache_q8(k, k, p, slots)
            o = torch.empty_like(q)
            pk.pa_decode_q8(o, q, p, t, dl, 0.09, 3008, ws)
            outs.append(o)
        return outs

    torch.cuda.synchronize()
    want = [step(s, 1)[0] for s in sets]
    torch.cuda.synchronize()
    got = []
    for s in sets:
        with torch.cuda.stream(s[5]):
            got.append(step(s, 10))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, o) for o in g)
    assert pk.pa_get_device_error() == 0


def test_decode_high_block_ids():
    """Blocks whose bytes lie behind 2^32."""
    n = (1 << 32) // pk.Q8Pool.block_bytes(8, 128) + 40
    p = pk.Q8Pool(n, 8, 128, "int8")
    small = make_pool(40, 8, 128, "int8", 2)
    p.buf[n - 40:] = small.buf
    lens = [300, 17]
    t = tables_for(lens, 40)
    q = rows(2, 32, 128, "bf16", 1)
    hi = np.where(t >= 0, t + (n - 40), -1).astype(np.int32)
    a, b = decode(p, q, hi, lens, 304, 0.1), decode(small, q, t, lens, 304, 0.1)
    assert pk.pa_get_device_error() == 0 and torch.equal(a, b)
    k = rows(17, 8, 128, "bf16", 5).to(DEV)
    slots = torch.arange(17, device=DEV) + 16 * (n - 3)
    pk.pa_reshape_and_cache_q8(k, k, p, slots)
    pk.pa_reshape_and_cache_q8(k, k, small, slots - 16 * (n - 40))
    assert pk.pa_get_device_error() == 0 and torch.equal(p.buf[n - 40:], small.buf)


def test_decode_is_reproducible_and_runs_on_a_stream_and_in_a_graph():
    lens = [5000, 77, 0, 1234, 2500, 600, 31, 4096]
    p = make_pool(sum((n + 15) // 16 for n in lens), 4, 128, "e4m3", 8)
    tables = tables_for(lens, p.num_blocks, 313)
    q = rows(8, 16, 128, "bf16", 9)
    a = decode(p, q, tables, lens, 5000, 0.09)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        b = decode(p, q, tables, lens, 5000, 0.09)
    st.synchronize()
    assert torch.equal(a, b)
    dq, dt = q.to(DEV), torch.from_numpy(tables).to(DEV)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, ws = torch.empty_like(dq), pk.alloc_workspace(8, 16, p, 5000)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.pa_decode_q8(out, dq, p, dt, dl, 0.09, 5000, ws)
    for _ in range(3):
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)
    dl.copy_(torch.tensor([1, 2, 3, 40, 0, 600, 31, 4000], dtype=torch.int32))
    dt[2, 0] = dt[3, 1]
    g.replay()
    c = decode(p, q, dt.cpu().numpy(), dl.tolist(), 5000, 0.09)
    assert torch.equal(out, c) and pk.pa_get_device_error() == 0


def test_decode_refusals():
    p = make_pool(8, 2, 64, "int8", 1)
    q = rows(1, 4, 64, "bf16", 1).to(DEV)
    t = torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    ln = torch.ones(1, dtype=torch.int32, device=DEV)
    o = torch.empty_like(q)
    for a in [(o.float(), q), (o.half(), q.half()), (o, q[:, :, :32]), (o, q.cpu()),
              (o, q.transpose(1, 2).contiguous().transpose(1, 2))]:
        with pytest.raises(ValueError):
            pk.pa_decode_q8(a[0], a[1], p, t, ln, 0.1, 16)
    for bad in [(t.long(), ln), (t, ln.long()), (t[0], ln), (t, ln[:0])]:
        with pytest.raises(ValueError):
            pk.pa_decode_q8(o, q, p, bad[0], bad[1], 0.1, 16)
    with pytest.raises(ValueError):
        pk.pa_decode(o, q, p, t, ln, 0.1, 16)
    wide = torch.zeros(1, 600, dtype=torch.int32, device=DEV)
    with pytest.raises(pk.PagedKVError) as e:
        pk.pa_decode_q8(o, q, p, wide, ln, 0.1, 9600)
    assert e.value.status == "WORKSPACE"


# ---- prefill ---------------------------------------------------------------------
def prefill(p, q, tables, lens, start, scale, max_new, out=None):
    q = q.to(DEV)
    out = torch.full_like(q, float("nan")) if out is None else out
    pk.pa_prefill_q8(out, q, p, torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                     torch.tensor(start, dtype=torch.int32, device=DEV), scale, max_new)
    return out


def check_prefill(heads_kv, group, code, lens, news, spread=0.5, seed=0, scale=128 ** -0.5):
    blocks = sum((n + 15) // 16 for n in lens) + 3
    p = make_pool(blocks, heads_kv, 128, code, seed, spread)
    tables = tables_for(lens, blocks, None, seed)
    codes, scales = poison(p, tables, lens)
    start = np.concatenate([[0], np.cumsum(news)]).tolist()
    q = rows(start[-1] + 5, heads_kv * group, 128, "bf16", seed + 1, 0.3)  # five rows behind the last sequence
    out = prefill(p, q, tables, lens, start, scale, max(news))
    assert pk.pa_get_device_error() == 0
    assert torch.isnan(out[start[-1]:]).all()
    # a probability times its V scale as fp16, sums over the whole sequence
    check_rows(out, q, lens, news, start, codes, scales, tables, p, "bf16", scale, 2.0 ** -11, max(lens))


@CODE
@pytest.mark.parametrize("heads_kv,group", [(1, 1), (3, 2), (2, 4), (1, 8), (2, 16)])
def test_prefill_prompts(heads_kv, group, code):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 100, 129, 200, 257]
    check_prefill(heads_kv, group, code, lens, lens, seed=group)


@CODE
@pytest.mark.parametrize("heads_kv,group", [(2, 1), (2, 4), (1, 16)])
def test_prefill_chunks(heads_kv, group, code):
    """New tokens behind cached contexts, single tokens and empty requests among them."""
    check_prefill(heads_kv, group, code, [700, 16, 33, 65, 1, 0, 500, 64, 128, 1025], [300, 1, 17, 64, 1, 0, 1, 0, 33, 70],
                  seed=2)


@CODE
def test_prefill_scales_far_apart(code):
    for seed in (3, 11, 12):
        check_prefill(2, 4, code, [1, 16, 40, 200, 900], [1, 16, 20, 100, 60], spread=5.0, seed=seed)


@CODE
def test_prefill_many_sequences(code):
    """More sequences than the launch sorts by length, more units than SMs."""
    r = np.random.RandomState(5)
    lens = r.randint(1, 150, 200)
    check_prefill(2, 8, code, lens.tolist(), (1 + (lens - 1) * r.rand(200)).astype(int).tolist(), seed=4)


@CODE
def test_prefill_zero_scales(code):
    p = make_pool(20, 2, 128, code, 1)
    lens = [130, 33]
    tables = tables_for(lens, 20, 9)
    p.scales[torch.from_numpy(tables[0, [0, 1, 4]]).long().to(DEV)] = 0   # zero K and V tiles
    p.scales[torch.from_numpy(tables[1, :3]).long().to(DEV), 1] = 0       # every V tile zero
    codes, scales = host(p)
    q = rows(163, 8, 128, "bf16", 3)
    for scale in (0.1, 0.0):
        out = prefill(p, q, tables, lens, [0, 130, 163], scale, 130)
        assert pk.pa_get_device_error() == 0
        check_rows(out, q, lens, lens, [0, 130], codes, scales, tables, p, "bf16", scale, 2.0 ** -11, 130)
        assert not out[130:].any()


@CODE
def test_prefill_bad_blocks_and_lengths(code):
    p = make_pool(60, 2, 128, code, 1)
    lens, news = [100, 90, 33, 300, 64], [50, 90, 40, 10, 64]             # 2: more new tokens than tokens; 3: too long
    tables = tables_for([100, 90, 33, 16, 64], 60, 8)
    start = np.concatenate([[0], np.cumsum(news)]).tolist()
    q = rows(start[-1], 4, 128, "bf16", 3)
    out = prefill(p, q, tables, lens, start, 0.1, 90)
    assert pk.pa_get_device_error() == pk.PA_DEVERR_SEQLEN
    codes, scales = host(p)
    assert torch.isnan(out[start[2]:start[4]]).all()
    for b in (0, 1, 4):
        check_rows(out[start[b]:start[b + 1]], q[start[b]:start[b + 1]], [lens[b]], [news[b]], [0], codes, scales,
                   tables[b:b + 1], p, "bf16", 0.1, 2.0 ** -11, 100)
    tables[0, 2], tables[1, 0] = 60, -1
    out2 = prefill(p, q, tables, [100, 90, 40, 10, 64], start, 0.1, 90)
    assert pk.pa_get_device_error() == pk.PA_DEVERR_BLOCK
    assert torch.equal(out2[start[4]:], out[start[4]:]) and torch.isfinite(out2[:start[2]]).all()


def test_prefill_agrees_with_decode_and_runs_in_a_graph():
    """A single new token is a decode step; a captured call replays with new lengths and tables."""
    lens = [400, 77, 16, 1, 250]
    p = make_pool(60, 4, 128, "int8", 8)
    tables = tables_for(lens, 60, 26)
    q = rows(5, 16, 128, "bf16", 9)
    a = prefill(p, q, tables, lens, range(6), 0.09, 1)
    b = decode(p, q, tables, lens, 416, 0.09)
    codes, scales = host(p)
    for x in (a, b):
        check_rows(x, q, lens, [1] * 5, range(5), codes, scales, tables, p, "bf16", 0.09, 2.0 ** -11, 400,
                   biased=True)
    dq, dt = q.to(DEV), torch.from_numpy(tables).to(DEV)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ds = torch.arange(6, dtype=torch.int32, device=DEV)
    out = torch.empty_like(dq)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.pa_prefill_q8(out, dq, p, dt, dl, ds, 0.09, 4)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a)
    dl.copy_(torch.tensor([300, 77, 16, 4, 200], dtype=torch.int32))
    ds.copy_(torch.tensor([0, 1, 1, 1, 5, 5], dtype=torch.int32))
    out.fill_(0)
    g.replay()
    want = prefill(p, q, dt.cpu().numpy(), dl.tolist(), ds.tolist(), 0.09, 4, torch.zeros_like(dq))
    assert torch.equal(out, want) and pk.pa_get_device_error() == 0


def test_prefill_refusals():
    p = make_pool(8, 2, 128, "int8", 1)
    q = rows(3, 4, 128, "bf16", 1).to(DEV)
    t = torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    ln, st = torch.full((1,), 3, dtype=torch.int32, device=DEV), torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    o = torch.empty_like(q)
    for a in [(o, q.float()), (o.float(), q), (o[:2], q), (o, q.cpu())]:
        with pytest.raises(ValueError):
            pk.pa_prefill_q8(a[0], a[1], p, t, ln, st, 0.1, 3)
    with pytest.raises(ValueError):
        pk.pa_prefill_q8(o, q, p, t, ln, st[:1], 0.1, 3)
    small = make_pool(8, 2, 64, "int8", 1)
    with pytest.raises(pk.PagedKVError) as e:
        pk.pa_prefill_q8(o[..., :64].contiguous(), q[..., :64].contiguous(), small, t, ln, st, 0.1, 3)
    assert e.value.status == "UNSUPPORTED"
    with pytest.raises(pk.PagedKVError) as e:
        pk.pa_prefill_q8(o, q, p, t, ln, st, -0.1, 3)
    assert e.value.status == "INVALID_ARG"
