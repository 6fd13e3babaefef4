"""Oracle of the step tables built on the device.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

One request after another, in plain Python integers: extend takes blocks from
the head of the free ring, release gives a finished request's blocks back to
its tail in table order ("如何通过PagedAttention实现LLM高性能推理：实战指南" §2.2:
the free blocks are a deque).
"""
from __future__ import annotations

BLOCK = 16


def pages(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def extend(tables, lens, new, ring, head, count, num_blocks, num_slots, row_tokens):
    """tables (list of lists) is changed in place. Returns lens_out, query_start,
    slots, state_out, error bits."""
    width = len(tables[0]) if tables else 1
    slots, start, out, refused, errors = [-1] * num_slots, [0], [], 0, 0
    state = [head, count]
    if not (0 <= head < len(ring) and 0 <= count <= len(ring)):
        errors |= 2
        head = count = 0
    asked_blocks = asked_tokens = taken = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        if L < 0 or n < 0 or L + n > width * BLOCK or (row_tokens and n > row_tokens):
            errors |= 4
            refused += 1
            out.append(L)
            start.append(start[-1])
            continue
        need = pages(L + n) - pages(L)
        asked_blocks += need
        asked_tokens += n
        if (need and asked_blocks > count) or (not row_tokens and n and asked_tokens > num_slots):
            refused += 1
            out.append(L)
            start.append(start[-1])
            continue
        for e in range(pages(L), pages(L + n)):
            tables[b][e] = ring[(head + taken) % len(ring)]
            taken += 1
        for i in range(n):
            blk = tables[b][(L + i) // BLOCK]
            at = b * row_tokens + i if row_tokens else start[-1] + i
            if 0 <= blk < num_blocks:
                slots[at] = blk * BLOCK + (L + i) % BLOCK
            else:
                errors |= 2
        out.append(L + n)
        start.append(start[-1] + n)
    if state == [head, count]:
        state = [(head + taken) % len(ring), count - taken]
    return out, start, slots, state + [start[-1], refused], errors


def release(tables, lens, finished, ring, head, count, num_blocks):
    """ring (a list) is changed in place. Returns lens_out, state_out, error bits."""
    width = len(tables[0]) if tables else 1
    room, state, errors = len(ring) - count, [head, count], 0
    if not (0 <= head < len(ring) and 0 <= count <= len(ring)):
        errors |= 2
        room = 0
    out, refused, asked, back = [], 0, 0, 0
    for b, (L, done) in enumerate(zip(lens, finished)):
        out.append(L)
        if not done:
            continue
        if L < 0 or L > width * BLOCK:
            errors |= 4
            refused += 1
            continue
        asked += pages(L)
        if asked > room:
            refused += 1
            continue
        out[b] = 0
        for e in range(pages(L)):
            ring[(head + count + back) % len(ring)] = tables[b][e]
            if not 0 <= tables[b][e] < num_blocks:
                errors |= 2
            back += 1
    return out, [state[0], state[1] + back, 0, refused], errors
