"""Oracle of the 8-bit pools: codes, append, attention.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

A tile is the 16 rows of one (block, K|V, head); an element is code * scale of
its tile. The append rule is defined step by step in binary32 (numpy float32
arithmetic is correctly rounded), so its results are compared bit for bit.
Attention is fp64 over the values that codes and scales stand for, and comes
with the two magnitudes that error bounds need.
"""
from __future__ import annotations

import numpy as np

F32 = np.float32
TINY = F32(2.0 ** -100)
MOST = {"int8": F32(127), "e4m3": F32(448)}

# value of each e4m3 byte from the format's definition (no infinity; 0x7f, 0xff NaN)
_MAG = np.array([(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)])
_MAG[127] = np.nan
E4M3_VALUES = np.concatenate([_MAG, -_MAG])


def decode(codes: np.ndarray, code: str) -> np.ndarray:
    """uint8 codes -> fp64 values."""
    return codes.view(np.int8).astype(np.float64) if code == "int8" else E4M3_VALUES[codes]


def encode(x: np.ndarray, code: str) -> np.ndarray:
    """fp32 values -> nearest codes (ties to even, saturating), uint8."""
    x = np.asarray(x, F32)
    if code == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    mag = np.minimum(np.abs(x).astype(np.float64), 448.0)
    hi = np.searchsorted(_MAG[:127], mag)                    # first value >= mag
    lo = np.maximum(hi - 1, 0)
    up, down = _MAG[hi] - mag, mag - _MAG[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (pick | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def grown(s: F32, a: F32, code: str) -> F32:
    """Scale of a tile of scale s that gains rows of largest magnitude a."""
    inv = F32(1) / MOST[code]
    if code == "int8":
        return max(s, a * inv)
    room = s * MOST[code]
    if not a > room:
        return s
    if s == 0:
        return a * inv
    (ma, ea), (mr, er) = np.frexp(a), np.frexp(room)         # m 2^e, m in [0.5, 1)
    return F32(np.ldexp(s, int(ea) - int(er) + int(ma > mr)))


def append(codes: np.ndarray, scales: np.ndarray, k: np.ndarray, v: np.ndarray, slots, code: str) -> None:
    """In place: codes uint8 [N][2][Hkv][16][D], scales fp32 [N][2][Hkv];
    k, v fp32 [T][Hkv][D]; negative slots are padding."""
    rows = {}
    for t, s in enumerate(int(x) for x in slots):
        if s >= 0:
            rows.setdefault(s // 16, {})[s % 16] = t         # a row named twice: the later token
    inv_most = F32(1) / MOST[code]
    for blk, at in rows.items():
        r = np.array(sorted(at))
        t = np.array([at[i] for i in r])
        for kv, src in enumerate((k, v)):
            for h in range(codes.shape[2]):
                x = src[t, h].astype(F32)
                mag = np.abs(x)
                a = F32(np.max(np.where(np.isfinite(x), mag, F32(0))))
                a = F32(0) if a < TINY else a
                old = F32(scales[blk, kv, h])
                fresh = 0 in at
                new = a * inv_most if fresh else F32(grown(old, a, code))
                if not fresh and new > old:
                    keep = np.array([i for i in range(16) if i not in at], int)
                    ratio = old / new
                    c = codes[blk, kv, h, keep]
                    codes[blk, kv, h, keep] = encode(decode(c, code).astype(F32) * ratio, code)
                inv = F32(1) / new if new > 0 else F32(0)
                x = np.where(np.isnan(x), F32(0), np.clip(x, -np.finfo(F32).max, np.finfo(F32).max))
                with np.errstate(over="ignore"):
                    codes[blk, kv, h, r] = encode(x * inv, code)
                scales[blk, kv, h] = new


def rows_of(codes, scales, table, length: int, code: str) -> np.ndarray:
    """[2][Hkv][length][D] fp64 values of a sequence's tokens."""
    blk = np.asarray(table[: (length + 15) // 16], np.int64)
    x = decode(codes[blk], code) * scales[blk].astype(np.float64)[..., None, None]
    return x.transpose(1, 2, 0, 3, 4).reshape(2, x.shape[2], -1, x.shape[4])[:, :, :length]


def scale_rows(scales, table, length: int) -> np.ndarray:
    """[2][Hkv][length] fp64: the K and V scale of each of a sequence's tokens."""
    return scales[np.asarray(table[: (length + 15) // 16], np.int64)].astype(np.float64).repeat(16, 0)[:length].transpose(
        1, 2, 0)


def attention(q: np.ndarray, kv: np.ndarray, scale: float, scales: np.ndarray):
    """Causal attention of the last len(q) of kv's tokens: q fp64 [n][H][D], kv
    fp64 [2][Hkv][L][D], scales [2][Hkv][L] from scale_rows. Returns out and what
    bound() needs, each [n][H][D] or [n][H][1]:
      mag   the sum of p |v|
      big   the largest scale * sum |q_d k_d| over the tokens seen
      low   the largest p * v_scale times the sum of the |V codes| (tiles of
            scale 0 aside)
      big1  the largest scale * k_scale * sum |q_d|
      mag1  the sum of p * v_scale"""
    n, H, D = q.shape
    G, L = H // kv.shape[1], kv.shape[2]
    out, mag, big, low = np.empty((n, H, D)), np.empty((n, H, D)), np.empty((n, H, 1)), np.empty((n, H, D))
    big1, mag1 = np.empty((n, H, 1)), np.empty((n, H, 1))
    seen = np.arange(L) <= (L - n + np.arange(n))[:, None]
    for h in range(H):
        (k, v), (ks, vs) = kv[:, h // G], scales[:, h // G]
        s = np.where(seen, scale * (q[:, h] @ k.T), -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out[:, h], mag[:, h] = p @ v, p @ np.abs(v)
        big[:, h, 0] = np.where(seen, abs(scale) * (np.abs(q[:, h]) @ np.abs(k).T), 0).max(1)
        big1[:, h, 0] = abs(scale) * np.abs(q[:, h]).sum(1) * np.where(seen, ks, 0).max(1)
        mag1[:, h, 0] = p @ vs
        low[:, h] = (p * vs).max(1, keepdims=True) * (seen @ (np.abs(v) / np.where(vs > 0, vs, 1)[:, None]))
    return out, (mag, big, low, big1, mag1)


def bound(ref, terms, dim: int, length: int, io: str, p_rounding: float, p_floor: float, biased: bool) -> np.ndarray:
    """What an output may be off by: the output's rounding, and of the sum of
    p |v| the rounding of each probability (p_rounding), the scores' errors
    (fp32 sums of dim terms; the exponent's argument passes a few roundings of
    its own size; fp32 queries keep 22 bits), 2^-20 for 2^x and the logarithm
    of the V scale, and the fp32 sums over at most `length` terms in a chain.
    p_floor: smallest spacing of the type that holds p * v_scale, relative to
    the largest of them: each such product may be off by half of it, whatever
    its own size, and multiplies a V code. fp16 products whose largest is at
    least 2^7 lie on a grid of 2^-24 there: 2^-31.
    biased: the sums over codes are formed over code + 128 <= 255 and 128 times
    the sum of the other factor is taken off, so their fp32 errors are relative
    to 255 sum |q_d| k_scale and to 255 sum p v_scale in place of sum |q_d k_d|
    and sum p |v|; the subtraction rounds once more at that size."""
    mag, big, low, big1, mag1 = terms
    if biased:
        big, chain = 255 * big1, 255 * mag1
    else:
        chain = mag
    score = (dim + 16) * 2.0 ** -24 + (2.0 ** -22 if io == "f32" else 0.0)
    eps = p_rounding + 2 * score * big + 16 * 2.0 ** -24 * big + 2.0 ** -20
    return ((2.0 ** -8 if io == "bf16" else 2.0 ** -23) * np.abs(ref) + eps * mag
            + (length + 16) * 2.0 ** -24 * chain + p_floor / 2 * low + 1e-30)
