"""Plain restatement of the step plan, one token at a time (test infrastructure)."""

import numpy as np

SEQ, BLOCK, QUERY, NO_BLOCKS = 0x8, 0x2, 0x40, 0x80


def plan_step(ctx, new, tables, free, head, num_tokens, bs, num_blocks):
    """(tables, cu, lens, slots, positions, head, error bits) of one step."""
    tables = np.array(tables, np.int32)
    b, width = tables.shape
    err = 0
    if not 0 <= head <= len(free):
        err |= BLOCK
        head = min(max(head, 0), len(free))
    cu, lens = [0], []
    slots = np.full(num_tokens, -1, np.int64)
    positions = np.zeros(num_tokens, np.int32)
    at, taken, start = head, head, 0
    for r in range(b):
        c, n = int(ctx[r]), int(new[r])
        if c < 0 or n < 0:
            err |= SEQ
            c, n = max(c, 0), 0
        old, full = -(-c // bs), -(-(c + n) // bs)
        placed = True
        if c + n > width * bs:
            err |= SEQ
            placed = False
        elif start + n > num_tokens:
            err |= QUERY
            placed = False
        else:
            at += full - old
            if full > old and at > len(free):
                err |= NO_BLOCKS
                placed = False
        if placed:
            if full > old:
                taken = at
            for k in range(full - old):
                tables[r, old + k] = free[at - (full - old) + k]
        for i in range(n):
            if start + i >= num_tokens:
                break
            p = c + i
            positions[start + i] = p
            if placed:
                blk = int(tables[r, p // bs])
                if 0 <= blk < num_blocks:
                    slots[start + i] = blk * bs + p % bs
                else:
                    err |= BLOCK
        start += n
        cu.append(min(start, num_tokens))
        lens.append(c + (n if placed else 0))
    return (tables, np.array(cu, np.int32), np.array(lens, np.int32), slots, positions, taken, err)
