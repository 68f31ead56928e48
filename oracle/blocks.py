"""Block pool oracle (test infrastructure only): forking, growing and compacting
rows of block tables, one row and one block at a time.

[KVB] §思想: sequences share physical blocks through their block tables (beam
search); [SM] §PagedAttention 批处理: a block is taken only when the last one is
full.  A pool is block_tables [n_rows, width], lens [n_rows] and refs
[num_blocks] (holders of each block, 0: free), all NumPy integers; every function
changes them in place.

Readings (the pages fix no order): free blocks are taken from the lowest id on, in
row order; a partial last block stays with its lowest row when every holder ends
in it, and every other row gets a copy.
"""
import numpy as np


def n_blocks(tokens, bs=16):
    return -(-int(tokens) // bs)


def held(tables, lens, r, bs=16):
    """The entries of row r."""
    return [int(e) for e in tables[r, :n_blocks(lens[r], bs)]]


def _lowest_free(refs):
    free = np.flatnonzero(refs == 0)
    return int(free[0]) if len(free) else -1


def fork(parents, keep, tables, lens, refs, bs=16):
    """Returns (pairs [n_rows, 2], rows cut for want of a block)."""
    n = len(lens)
    before = [held(tables, lens, r, bs) for r in range(n)]
    had = [int(x) for x in lens]
    after, new = [], []
    for j in range(n):
        p = int(parents[j])
        have = had[p] if 0 <= p < n else 0
        k = -1 if keep is None else int(keep[j])
        m = have if k < 0 else min(have, k)
        new.append(m)
        after.append(before[p][:n_blocks(m, bs)] if m else [])
    for row in after:
        for e in row:
            if e >= 0:
                refs[e] += 1
    for row in before:
        for e in row:
            if e >= 0:
                refs[e] -= 1
    ends = [after[j][-1] if new[j] % bs and after[j][-1] >= 0 else -1 for j in range(n)]
    need = []
    for j in range(n):
        same = [i for i in range(n) if ends[i] == ends[j]]
        if ends[j] >= 0 and not (len(same) == refs[ends[j]] and same[0] == j):
            need.append(j)
    pairs = np.full((n, 2), -1, np.int64)
    free = [int(b) for b in np.flatnonzero(refs == 0)]
    cut = []
    for k, j in enumerate(need):
        refs[ends[j]] -= 1
        if k < len(free):
            refs[free[k]] = 1
            pairs[j] = ends[j], free[k]
            after[j][-1] = free[k]
        else:
            after[j][-1] = -1
            new[j] -= new[j] % bs
            cut.append(j)
    for j in range(n):
        width = max(len(before[j]), len(after[j]))
        tables[j, :width] = after[j] + [-1] * (width - len(after[j]))
        lens[j] = new[j]
    return pairs, cut


def grow(q_lens, tables, lens, refs, bs=16):
    """Returns (ctx_lens, slots, rows that did not grow)."""
    ctx = lens.copy()
    slots, stay = [], []
    free = [int(b) for b in np.flatnonzero(refs == 0)]
    asked = 0
    for r, q in enumerate(int(x) for x in q_lens):
        a, b = n_blocks(lens[r], bs), n_blocks(lens[r] + q, bs)
        if b > tables.shape[1]:
            stay.append(r)
            slots += [-1] * q
            continue
        asked += b - a
        if b > a and asked > len(free):
            stay.append(r)
            slots += [-1] * q
            continue
        for c in range(a, b):
            e = free[asked - (b - a) + c - a]
            tables[r, c] = e
            refs[e] = 1
        for i in range(q):
            pos = int(lens[r]) + i
            slots.append(int(tables[r, pos // bs]) * bs + pos % bs)
        lens[r] += q
    return ctx, np.asarray(slots, np.int64), stay


def compact(tables, lens, refs, max_pairs=None, bs=16):
    """Returns (block_map, moves [n, 2], live blocks)."""
    live = int((refs > 0).sum())
    holes = [b for b in range(live) if refs[b] <= 0]
    movers = [b for b in range(live, len(refs)) if refs[b] > 0]
    moves = list(zip(movers, holes))[:max_pairs]
    block_map = np.where(refs > 0, np.arange(len(refs)), -1)
    for src, dst in moves:
        block_map[src] = dst
        refs[dst], refs[src] = refs[src], 0
    for r in range(len(lens)):
        for c in range(n_blocks(lens[r], bs)):
            if tables[r, c] >= 0:
                tables[r, c] = block_map[tables[r, c]]
    return block_map, np.asarray(moves, np.int64).reshape(-1, 2), live


def check(tables, lens, refs, held_outside=None, bs=16):
    """The pool's invariants: refs counts the entries (and what is held outside),
    and a block that a row will write next has no other holder."""
    count = np.zeros(len(refs), np.int64) if held_outside is None else held_outside.astype(np.int64).copy()
    for r in range(len(lens)):
        for e in held(tables, lens, r, bs):
            if e >= 0:
                count[e] += 1
    assert np.array_equal(count, refs)
    for r in range(len(lens)):
        if lens[r] % bs:
            e = held(tables, lens, r, bs)[-1]
            assert e < 0 or refs[e] == 1, f"row {r} shares the block it will write"
