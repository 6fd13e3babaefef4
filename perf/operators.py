"""Cases that time the 8-bit cache operators and the device-side block tables, each next to a plain
form made of elementary torch operations.

Operators (calls of paged_kv_cache_400_b200):
  append   pa_reshape_and_cache_q8   new K/V rows coded in 8 bits into their slots
  decode   pa_decode_q8              single-token attention over the 8-bit cache
  prefill  pa_prefill_q8             causal attention of new tokens over the 8-bit cache
  extend   pa_tables_extend          blocks taken, tables and slot maps built from request lengths
  release  pa_tables_release         finished requests' blocks back to the free ring

An 8-bit pool is one uint8 buffer [num_blocks][block_bytes]; a block holds codes
[2][num_kv_heads][16][head_dim] and, after them, fp32 scales [2][num_kv_heads] (K, V), padded to a
multiple of 128 bytes. A code stands for code * scale of its (block, K|V, head).

Coding of a tile (block, K|V, head), A = the largest finite |x| of its rows in the call, M = 127
(int8) or 448 (e4m3), all in fp32: A below 2^-100 counts as 0; a tile whose row 0 is written starts
afresh with scale A * (1/M); otherwise the scale only grows, for int8 to A * (1/M), for e4m3 by the
smallest power of two that makes room for A, and the rows kept are coded again at the grown scale.
A code is x * (1/scale) rounded to the nearest value of the type, ties to even.
"""
import math

import numpy as np
import torch

own = False
BS = 16
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
MOST = {"int8": 127.0, "e4m3": 448.0}
TINY = 2.0 ** -100


# ---- cases --------------------------------------------------------------------------------------
def listed():
    return [
        # one new token of each of 256 running requests, into blocks that hold 0..15 tokens already
        dict(name="append_decode_b256", op="append", form="decode", batch=256, tokens=256, kv_heads=8, dim=128,
             io="bf16", code="int8", lens=11),
        # whole prompts of a step's admitted requests, 8192 tokens in all, ragged ends
        dict(name="append_prompts_8k", op="append", form="prompts", batch=15, tokens=8192, kv_heads=8, dim=128,
             io="bf16", code="e4m3", lens=12),
        # the smallest call: four short requests, fp32, as many KV heads as query heads
        dict(name="decode_tiny_f32", op="decode", batch=4, kv_heads=2, group=1, dim=64, io="f32", code="int8",
             shape="tiny", max_len=48, lens=1),
        # a full decode batch with grouped heads, lengths lognormal (median 1000) in [16, 8192]
        dict(name="decode_gqa_b256", op="decode", batch=256, kv_heads=8, group=4, dim=128, io="bf16", code="int8",
             shape="lognormal", max_len=8192, lens=2),
        # as many KV heads as query heads, lengths uniform in [128, 2048]
        dict(name="decode_mha_b64", op="decode", batch=64, kv_heads=32, group=1, dim=128, io="bf16", code="e4m3",
             shape="uniform", max_len=2048, lens=3),
        # one request with a long context: the sequence axis has to be split
        dict(name="decode_long_b1", op="decode", batch=1, kv_heads=8, group=4, dim=128, io="bf16", code="int8",
             shape="full", max_len=131071, lens=4),
        # a few short prompts attended after their append
        dict(name="prefill_prompts_b5", op="prefill", batch=5, kv_heads=8, group=4, new=203, context=0, io="bf16",
             code="e4m3", dim=128, lens=5),
        # a chunked-prefill step: 512-token chunks after cached contexts of up to 4096 tokens
        dict(name="prefill_chunked_b16", op="prefill", batch=16, kv_heads=8, group=4, new=512, context=4096,
             io="bf16", code="int8", dim=128, lens=6),
        # the decode step's tables: one token for each of 256 requests
        dict(name="extend_decode_b256", op="extend", form="rows", batch=256, new=1, context=2048, lens=7),
        # admission of many prompts at once, packed slot map of about half a million tokens
        dict(name="extend_prompts_b1000", op="extend", form="packed", batch=1000, new=1024, context=0, lens=8),
        # a few requests of a decode batch finish
        dict(name="release_b256", op="release", batch=256, context=2048, share=0.05, lens=9),
        # a large batch is dropped at once
        dict(name="release_b4096", op="release", batch=4096, context=4096, share=0.7, lens=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "decode", "prefill", "prefill", "extend", "extend",
                     "release"])
    seed = rng.randrange(1 << 30)
    if op == "append":
        form = rng.choice(["decode", "prompts"])
        tokens = _log(rng, 1, 8192)
        if form == "decode":
            tokens = min(tokens, 1024)
        return dict(op=op, form=form, batch=tokens if form == "decode" else _log(rng, 1, min(64, tokens)),
                    tokens=tokens, kv_heads=rng.choice([1, 2, 3, 4, 8]), dim=rng.choice([64, 128]),
                    io=rng.choice(["bf16", "f32"]), code=rng.choice(["int8", "e4m3"]), lens=seed)
    if op == "decode":
        kv = rng.choice([1, 2, 4, 5, 8, 32])
        batch = _log(rng, 1, 256)
        group = rng.choice([1, 2, 3, 4, 7, 8] + ([16] if kv < 32 else []))
        most = max(1, min(32768, 10000000 // (kv * max(4, group) * batch)))
        return dict(op=op, batch=batch, kv_heads=kv, group=group, dim=rng.choice([64, 128, 128]),
                    io=rng.choice(["bf16", "bf16", "f32"]), code=rng.choice(["int8", "e4m3"]),
                    shape=rng.choice(["uniform", "lognormal", "full"]),
                    max_len=_log(rng, 1, most), lens=seed)
    if op == "prefill":
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, batch=_log(rng, 1, min(16, 512 // (kv * group))), kv_heads=kv, group=group,
                    new=_log(rng, 1, 500), context=rng.choice([0, _log(rng, 1, 2000)]), io="bf16",
                    code=rng.choice(["int8", "e4m3"]), dim=128, lens=seed)
    if op == "extend":
        form = rng.choice(["rows", "packed"])
        batch = _log(rng, 1, 4096)
        return dict(op=op, form=form, batch=batch, new=1 if form == "rows" and rng.random() < 0.6 else
                    _log(rng, 1, max(1, min(2000, 400000 // batch))),
                    context=rng.choice([0, _log(rng, 1, 4096)]), lens=seed)
    return dict(op=op, batch=_log(rng, 1, 4096), context=_log(rng, 1, 4000), share=rng.choice([0.03, 0.3, 1.0]),
                lens=seed)


# ---- sizes that follow from a case alone ----------------------------------------------------------
def _seq_lens(c):
    r = np.random.RandomState(c["lens"])
    n, top = c["batch"], c["max_len"]
    if c["shape"] == "tiny":
        return np.array([5, 16, 17, 33])[:n]
    if c["shape"] == "full":
        return np.full(n, top)
    if c["shape"] == "uniform":
        return r.randint(max(1, top // 16), top + 1, n)
    # median 1000 and clipped to [16, 8192] at the largest bound; in proportion below it
    return np.clip(np.rint(np.exp(r.normal(math.log(max(1.0, top / 8.192)), 0.8, n))), min(16, top), top).astype(int)


def _query_lens(c):
    r = np.random.RandomState(c["lens"])
    if c["context"]:
        new = np.full(c["batch"], c["new"])
        new[r.rand(c["batch"]) < 0.2] = max(1, c["new"] // 3)
        return new, r.randint(0, c["context"] + 1, c["batch"])
    return r.randint(max(1, c["new"] // 8), c["new"] + 1, c["batch"]), np.zeros(c["batch"], int)


def _append_lens(c):
    """(tokens held before, new tokens) of each request."""
    r = np.random.RandomState(c["lens"])
    if c["form"] == "decode":
        return r.randint(0, 200, c["batch"]), np.ones(c["batch"], int)
    cuts = np.sort(r.choice(np.arange(1, c["tokens"]), c["batch"] - 1, replace=False)) if c["batch"] > 1 else []
    new = np.diff(np.concatenate([[0], cuts, [c["tokens"]]])).astype(int)
    # most prompts start at 0, some go on behind a cached prefix that ends inside a block
    return np.where(r.rand(c["batch"]) < 0.7, 0, r.randint(0, 40, c["batch"])), new


def _table_lens(c):
    r = np.random.RandomState(c["lens"])
    old = r.randint(0, c["context"] + 1, c["batch"])
    if c["op"] == "release":
        return old, (r.rand(c["batch"]) < c["share"]).astype(int)
    if c["new"] == 1:
        return old, np.ones(c["batch"], int)
    return old, r.randint(0, c["new"] + 1, c["batch"])


def _pages(n):
    return (np.asarray(n) + BS - 1) // BS


def _block_bytes(c):
    raw = 2 * c["kv_heads"] * BS * c["dim"]
    return raw, (raw + 8 * c["kv_heads"] + 127) // 128 * 128


def work(case):
    c = case
    io = 4 if c.get("io") == "f32" else 2
    if c["op"] == "append":
        old, new = _append_lens(c)
        t, h, d = int(new.sum()), c["kv_heads"], c["dim"]
        tiles = int((_pages(old + new) - old // BS).sum()) * 2 * h
        return {"bytes": t * h * d * 2 * (io + 1) + 8 * t + 8 * tiles, "flops": 4 * t * h * d}
    if c["op"] == "decode":
        n = _seq_lens(c)
        h, d, heads = c["kv_heads"], c["dim"], c["kv_heads"] * c["group"]
        return {"bytes": int(n.sum()) * h * d * 2 + int(_pages(n).sum()) * (8 * h + 4) + 2 * c["batch"] * heads * d * io,
                "flops": 4 * int(n.sum()) * heads * d}
    if c["op"] == "prefill":
        new, ctx = _query_lens(c)
        h, d, heads = c["kv_heads"], c["dim"], c["kv_heads"] * c["group"]
        pairs = int((new * ctx + new * (new + 1) // 2).sum())
        return {"bytes": int((new + ctx).sum()) * h * d * 2 + int(_pages(new + ctx).sum()) * (8 * h + 4)
                + 2 * int(new.sum()) * heads * d * io, "flops": 4 * pairs * heads * d}
    old, new = _table_lens(c)
    if c["op"] == "extend":
        t = int(new.sum())
        fresh = int((_pages(old + new) - _pages(old)).sum())
        slots = c["batch"] * c["new"] if c["form"] == "rows" else t
        return {"bytes": 16 * c["batch"] + 8 * fresh + 8 * slots, "flops": 0}
    return {"bytes": 12 * c["batch"] + 8 * int((_pages(old) * new).sum()), "flops": 0}


# ---- inputs ----------------------------------------------------------------------------------------
def _tables(lens, num_blocks, width, g):
    """Random distinct blocks for every request, -1 behind them."""
    lens = torch.as_tensor(np.asarray(_pages(lens)), device=DEV)
    perm = torch.randperm(num_blocks, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(width, device=DEV)
    used = at < lens[:, None]
    t = torch.full(used.shape, -1, dtype=torch.int32, device=DEV)
    t[used] = perm[: int(lens.sum())]
    return t, perm


def _views(buf, c):
    raw, _ = _block_bytes(c)
    n, h = buf.shape[0], c["kv_heads"]
    codes = buf[:, :raw].view(CODES[c["code"]]).unflatten(1, (2, h, BS, c["dim"]))
    scales = buf[:, raw:raw + 8 * h].view(torch.float32).view(n, 2, h)
    return codes, scales


def _filled_pool(c, num_blocks, g):
    """A pool whose tiles hold coded normal values; amplitudes differ from tile to tile."""
    raw, total = _block_bytes(c)
    buf = torch.zeros(num_blocks, total, dtype=torch.uint8, device=DEV)
    codes, scales = _views(buf, c)
    step = max(1, (1 << 27) // raw)
    for i in range(0, num_blocks, step):
        x = torch.randn(min(step, num_blocks - i), 2, c["kv_heads"], BS, c["dim"], generator=g, device=DEV)
        a = torch.exp(0.3 * torch.randn(x.shape[:3], generator=g, device=DEV))
        s = x.abs().amax((3, 4)) * (1.0 / MOST[c["code"]])
        y = x * (1.0 / s)[..., None, None]
        codes[i:i + step] = (y.round().to(torch.int8) if c["code"] == "int8" else
                             y.clamp(-448, 448).to(torch.float8_e4m3fn))
        scales[i:i + step] = s * a
    return buf


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + c["lens"])
    s = {"case": c}
    if c["op"] in ("extend", "release"):
        _prepare_tables(c, s, g)
        return s
    if c["op"] == "append":
        old, new = _append_lens(c)
        blocks = int(_pages(old + new).sum()) + 64
        s["buf"] = _filled_pool(c, blocks, g)
        table, _ = _tables(old + new, blocks, int(_pages(old + new).max()), g)
        seq = torch.as_tensor(np.repeat(np.arange(c["batch"]), new), device=DEV)
        pos = torch.as_tensor(np.concatenate([np.arange(a, a + n) for a, n in zip(old, new)]), device=DEV)
        s["slots"] = table[seq, pos // BS].long() * BS + pos % BS
        shape = (len(seq), c["kv_heads"], c["dim"])
        amp = torch.exp(0.5 * torch.randn(len(seq), 1, 1, generator=g, device=DEV))
        s["k"] = (torch.randn(shape, generator=g, device=DEV) * amp).to(TYPES[c["io"]])
        s["v"] = (torch.randn(shape, generator=g, device=DEV) * amp).to(TYPES[c["io"]])
    else:
        if c["op"] == "decode":
            lens, rows, s["max_len"] = _seq_lens(c), c["batch"], c["max_len"]
        else:
            new, ctx = _query_lens(c)
            lens, rows = new + ctx, int(new.sum())
            start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
            s["query_start"] = torch.as_tensor(start, device=DEV)
            s["max_new"] = int(new.max())
        blocks = int(_pages(lens).sum()) + 32
        s["buf"] = _filled_pool(c, blocks, g)
        width = int(_pages(max(int(lens.max()), s.get("max_len", 0))))
        s["tables"], _ = _tables(lens, blocks, width, g)
        s["lens"] = torch.as_tensor(lens.astype(np.int32), device=DEV)
        s["q"] = torch.randn(rows, c["kv_heads"] * c["group"], c["dim"], generator=g, device=DEV).to(TYPES[c["io"]])
        s["scale"] = 1.0 / math.sqrt(c["dim"])
        s["out"] = torch.empty_like(s["q"])
    if own:
        import paged_kv_cache_400_b200 as pk
        s["pool"] = pk.Q8Pool.wrap(s["buf"], c["kv_heads"], c["dim"], c["code"])
        if c["op"] == "decode":
            s["ws"] = pk.alloc_workspace(c["batch"], c["kv_heads"] * c["group"], s["pool"], c["max_len"])
    return s


def _prepare_tables(c, s, g):
    old, new = _table_lens(c)
    width = int(_pages((old + new if c["op"] == "extend" else old).max())) + 1
    held = int(_pages(old).sum())
    spare = int((_pages(old + new) - _pages(old)).sum()) if c["op"] == "extend" else 0
    blocks = held + spare + 100
    table, perm = _tables(old, blocks, width, g)
    free = perm[held:]
    ring = torch.full((blocks,), -1, dtype=torch.int32, device=DEV)
    head = int(torch.randint(0, blocks, (1,), generator=g, device=DEV))  # the ring wraps for most heads
    ring[(head + torch.arange(len(free), device=DEV)) % blocks] = free
    s.update(tables=table, lens=torch.as_tensor(old.astype(np.int32), device=DEV), ring=ring, num_blocks=blocks,
             state=torch.tensor([head, len(free), 0, 0], dtype=torch.int32, device=DEV),
             lens_out=torch.empty(c["batch"], dtype=torch.int32, device=DEV),
             state_out=torch.empty(4, dtype=torch.int32, device=DEV))
    if c["op"] == "release":
        s["done"] = torch.as_tensor(new.astype(np.int32), device=DEV)
    else:
        s["new"] = torch.as_tensor(new.astype(np.int32), device=DEV)
        s["query_start"] = torch.empty(c["batch"] + 1, dtype=torch.int32, device=DEV)
        slots = c["batch"] * c["new"] if c["form"] == "rows" else int(new.sum()) + 37
        s["slots"] = torch.empty(slots, dtype=torch.int64, device=DEV)
    if own:
        import paged_kv_cache_400_b200 as pk
        s["ws"] = pk.alloc_tables_workspace(c["batch"])


# ---- one pass --------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    form = {"append": _append, "decode": _decode, "prefill": _prefill, "extend": _extend, "release": _release}
    return form[c["op"]](c, s)


def _append(c, s):
    codes, scales = _views(s["buf"], c)
    if own:
        import paged_kv_cache_400_b200 as pk
        pk.pa_reshape_and_cache_q8(s["k"], s["v"], s["pool"], s["slots"])
        return {"codes": codes, "scales": scales}
    top = MOST[c["code"]]
    int8 = c["code"] == "int8"
    code = (lambda x: x.round().clamp(-top, top)) if int8 else \
        (lambda x: x.clamp(-top, top).to(torch.float8_e4m3fn).float())
    blk, tile = torch.unique(s["slots"] // BS, return_inverse=True)
    row = s["slots"] % BS
    x = torch.zeros(len(blk), 2, c["kv_heads"], BS, c["dim"], device=DEV)
    x[tile, 0, :, row] = s["k"].float()
    x[tile, 1, :, row] = s["v"].float()
    fresh_row = torch.zeros(len(blk), BS, dtype=torch.bool, device=DEV)
    fresh_row[tile, row] = True
    a = x.abs().amax((3, 4))
    a = torch.where(a < TINY, 0.0, a)
    old = scales[blk]
    first = a * (1.0 / top)
    if int8:
        grown = torch.maximum(old, first)
    else:
        m, e = torch.frexp(a / (old * top))
        k = torch.where(m > 0.5, e, e - 1).clamp_min(0)
        grown = torch.where(a > old * top, torch.ldexp(old, k), old)
        grown = torch.where(old == 0, first, grown)
    new = torch.where(fresh_row[:, 0, None, None], first, grown)
    inv = torch.where(new > 0, 1.0 / new, 0.0)
    kept = codes[blk].float()
    ratio = torch.where(old == new, 1.0, torch.where(new > 0, old / new, 0.0))
    again = torch.where((old < new)[..., None, None] & ~fresh_row[:, None, None, :1, None],
                        code(kept * ratio[..., None, None]), kept)
    y = torch.where(fresh_row[:, None, None, :, None], code(x * inv[..., None, None]), again)
    codes[blk] = y.to(codes.dtype)
    scales[blk] = new
    return {"codes": codes, "scales": scales}


def _decode(c, s):
    if own:
        import paged_kv_cache_400_b200 as pk
        pk.pa_decode_q8(s["out"], s["q"], s["pool"], s["tables"], s["lens"], s["scale"], s["max_len"], s["ws"])
        return s["out"]
    codes, scales = _views(s["buf"], c)
    b, h, g, d = c["batch"], c["kv_heads"], c["group"], c["dim"]
    lens = s["lens"].long()
    seq = torch.repeat_interleave(torch.arange(b, device=DEV), lens)
    pos = torch.arange(len(seq), device=DEV) - (lens.cumsum(0) - lens)[seq]
    blk, row = s["tables"][seq, pos // BS].long(), pos % BS
    k = codes[blk, 0, :, row].float() * scales[blk, 0][..., None]
    v = codes[blk, 1, :, row].float() * scales[blk, 1][..., None]
    q = s["q"].float().view(b, h, g, d)
    sc = (q[seq] @ k[..., None])[..., 0] * s["scale"]                       # [tokens][h][g]
    at = seq[:, None, None].expand_as(sc)
    m = torch.full((b, h, g), -math.inf, device=DEV).scatter_reduce_(0, at, sc, "amax")
    p = torch.exp(sc - m[seq])
    l = torch.zeros(b, h, g, device=DEV).index_add_(0, seq, p)
    o = torch.zeros(b, h, g, d, device=DEV).index_add_(0, seq, p[..., None] * v[:, :, None])
    return (o / l[..., None]).view(b, h * g, d).to(s["q"].dtype)


def _prefill(c, s):
    if own:
        import paged_kv_cache_400_b200 as pk
        pk.pa_prefill_q8(s["out"], s["q"], s["pool"], s["tables"], s["lens"], s["query_start"], s["scale"],
                         s["max_new"])
        return s["out"]
    codes, scales = _views(s["buf"], c)
    b, h, g, d = c["batch"], c["kv_heads"], c["group"], c["dim"]
    lens, start = s["lens"].long(), s["query_start"].long()
    new = start[1:] - start[:-1]
    n, t = s["max_new"], s["tables"].shape[1] * BS
    blk = s["tables"].long().clamp_min(0)                                    # behind the end: masked below
    kv = codes[blk].float() * scales[blk][..., None, None]                   # [b][pages][2][h][16][d]
    k, v = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, b, h, t, d)
    i = torch.arange(n, device=DEV)
    here = i < new[:, None]
    rows = torch.where(here, start[:-1, None] + i, 0)
    q = s["q"].float()[rows].view(b, n, h, g, d).permute(0, 2, 3, 1, 4).reshape(b, h, g * n, d)
    sc = (q @ k.transpose(2, 3)).view(b, h, g, n, t) * s["scale"]
    p = (lens - new)[:, None] + i                                            # position of each query
    sc.masked_fill_((torch.arange(t, device=DEV) > p[..., None])[:, None, None], -math.inf)
    e = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = (e.view(b, h, g * n, t) @ v).view(b, h, g, n, d) / e.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, h * g, d)
    return o[here].to(s["q"].dtype)


def _extend(c, s):
    step = c["new"] if c["form"] == "rows" else 0
    if own:
        import paged_kv_cache_400_b200 as pk
        pk.pa_tables_extend(s["tables"], s["lens"], s["new"], s["ring"], s["state"], s["lens_out"], s["query_start"],
                            s["slots"], s["state_out"], s["num_blocks"], step, s["ws"])
        return [s["tables"], s["lens_out"], s["query_start"], s["slots"], s["state_out"]]
    b, w = s["tables"].shape
    old, new = s["lens"].long(), s["new"].long()
    had, need = (old + BS - 1) // BS, (old + new + BS - 1) // BS
    take = need - had
    first = take.cumsum(0) - take
    head, count = s["state"][0].long(), s["state"][1].long()
    e = torch.arange(w, device=DEV)
    fresh = (e >= had[:, None]) & (e < need[:, None])
    ids = s["ring"][(head + first[:, None] + e - had[:, None]) % s["ring"].numel()]
    s["tables"].copy_(torch.where(fresh, ids, s["tables"]))
    s["lens_out"].copy_(old + new)
    s["query_start"][0] = 0
    s["query_start"][1:] = new.cumsum(0)
    s["slots"].fill_(-1)
    seq = torch.repeat_interleave(torch.arange(b, device=DEV), new)
    i = torch.arange(len(seq), device=DEV) - (new.cumsum(0) - new)[seq]
    pos = old[seq] + i
    slot = s["tables"][seq, pos // BS].long() * BS + pos % BS
    s["slots"][seq * step + i if step else torch.arange(len(seq), device=DEV)] = slot
    total = take.sum()
    s["state_out"].copy_(torch.stack([(head + total) % s["ring"].numel(), count - total, new.sum(), 0 * total]))
    return [s["tables"], s["lens_out"], s["query_start"], s["slots"], s["state_out"]]


def _release(c, s):
    if own:
        import paged_kv_cache_400_b200 as pk
        pk.pa_tables_release(s["tables"], s["lens"], s["done"], s["ring"], s["state"], s["lens_out"], s["state_out"],
                             s["num_blocks"], s["ws"])
        return [s["ring"], s["lens_out"], s["state_out"]]
    done = s["done"] != 0
    had = torch.where(done, (s["lens"].long() + BS - 1) // BS, 0)
    e = torch.arange(s["tables"].shape[1], device=DEV)
    back = s["tables"][e < had[:, None]]                                     # in request and table order
    head, count = s["state"][0].long(), s["state"][1].long()
    s["ring"][(head + count + torch.arange(len(back), device=DEV)) % s["ring"].numel()] = back
    s["lens_out"].copy_(torch.where(done, 0, s["lens"]))
    s["state_out"].copy_(torch.stack([head, count + len(back), 0 * head, 0 * head]))
    return [s["ring"], s["lens_out"], s["state_out"]]


# ---- the definitions in 64 bits ----------------------------------------------------------------------
def exact(case, seed):
    c = case
    if c["op"] in ("extend", "release"):
        return None  # whole numbers only
    s = prepare(c, seed)
    codes, scales = _views(s["buf"], c)
    if c["op"] == "append":
        return _exact_append(c, s, codes, scales)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    h, g = c["kv_heads"], c["group"]
    lens = s["lens"].tolist()
    start = s["query_start"].tolist() if c["op"] == "prefill" else list(range(c["batch"] + 1))
    for b, n in enumerate(lens):
        blk = s["tables"][b, : (n + BS - 1) // BS].long()
        kv = codes[blk].double() * scales[blk].double()[..., None, None]     # [pages][2][h][16][d]
        kv = kv.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n]               # [2][h][n][d]
        q = s["q"][start[b]:start[b + 1]].double()
        new = len(q)
        q = q.view(new, h, g, -1).permute(1, 2, 0, 3).reshape(h, g * new, -1)
        w = torch.matmul(q, kv[0].transpose(1, 2)).view(h, g, new, n) * s["scale"]
        last = torch.arange(n - new, n, device=DEV)
        w = w.masked_fill(torch.arange(n, device=DEV) > last[:, None], -math.inf)
        w = torch.softmax(w, -1).view(h, g * new, n)
        o = torch.matmul(w, kv[1]).view(h, g, new, -1).permute(2, 0, 1, 3)
        out[start[b]:start[b + 1]] = o.reshape(new, h * g, -1)
    return out


def _nearest_e4m3(x):
    """Nearest e4m3 value, ties to even, of values within +-448 (64-bit arithmetic)."""
    _, e = torch.frexp(x)
    unit = torch.ldexp(torch.ones_like(x), torch.clamp(e - 1, min=-6) - 3)
    return torch.clamp(torch.round(x / unit) * unit, -448, 448)


def _exact_append(c, s, codes, scales):
    top = MOST[c["code"]]
    near = torch.round if c["code"] == "int8" else _nearest_e4m3
    value = codes.double()
    scale = scales.double()
    slots = s["slots"].tolist()
    owner = {}
    for t, slot in enumerate(slots):
        owner.setdefault(slot // BS, []).append((slot % BS, t))
    for blk, rows in owner.items():
        r = torch.tensor([x for x, _ in rows], device=DEV)
        t = torch.tensor([x for _, x in rows], device=DEV)
        new = torch.stack([s["k"][t], s["v"][t]]).double().transpose(1, 2)   # [2][h][rows][d]
        a = new.abs().amax((2, 3))
        was = scale[blk]
        if 0 in [x for x, _ in rows]:
            now = a / top
        elif c["code"] == "int8":
            now = torch.maximum(was, a / top)
            value[blk] = near(value[blk] * (was / now)[..., None, None])
        else:
            k = torch.clamp(torch.ceil(torch.log2(a / (was * top))), min=0)
            now = was * 2.0 ** k
            value[blk] = near(value[blk] * (2.0 ** -k)[..., None, None])
        scale[blk] = now
        value[blk][:, :, r] = near(new / now[..., None, None])
    return {"codes": value, "scales": scale}
