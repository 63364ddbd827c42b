"""Page bookkeeping of a step, a sequence and a page at a time (lists on the
host, no code of the library)."""
from __future__ import annotations


TOP = 2 ** 31 - 1


def step(table, seq_len, new, free, count, page, window=0, sinks=0, released=None, num_slots=None):
    """Updates `table` (rows of page ids) and `free` (a list of the stack's
    capacity) in place; returns (q_start, positions, seq_len, count, released,
    slots, errors)."""
    B, cap, width = len(seq_len), len(free), len(table[0])
    keep = -(-sinks // page)
    errors = []
    if count > cap:
        errors.append(count)
        count = cap
    count = max(count, 0)
    back, held, gone_after = [], [], []
    for b in range(B):
        L = max(seq_len[b], 0)
        h = -(-L // page)
        if h > width:
            errors.append(h)
            h = width
        held.append(h)
        gone = max(keep, released[b]) if window else 0
        if new[b] < 0:
            cols = [c for c in range(h) if not window or c < keep or c >= gone]
            after = 0
        elif window:
            cols = [c for c in range(gone, h) if (c + 1) * page <= L - window + 1]
            after = gone + len(cols)
        else:
            cols, after = [], 0
        gone_after.append(after)
        back += [table[b][c] for c in cols]
    stack = free[:count] + back
    if len(stack) > cap:
        errors.append(len(stack))
        stack = stack[:cap]
    avail = len(stack)
    q_start, positions, after_len, wanted, served = [0], [], [], 0, []
    for b in range(B):
        L, n = max(seq_len[b], 0), new[b]
        q_start.append(q_start[-1] + max(n, 0))
        need = -(-(L + max(n, 0)) // page) - -(-L // page)
        fits = n >= 0 and -(-L // page) <= width
        if fits and (-(-(L + n) // page) > width or L + n > TOP):
            errors.append(-(-(L + n) // page))
            fits = False
        # packed tokens behind the slots, or behind what an int32 counts
        if n > 0 and q_start[-1] > (TOP if num_slots is None else num_slots):
            if fits:
                errors.append(q_start[-1])
            fits = False
        ok = False
        if fits:
            wanted += need
            ok = need == 0 or wanted <= avail
        served.append(ok)
        positions.append(L if ok else -1)
        after_len.append(0 if n < 0 else L + n if ok else L)
        if ok:
            for c in range(held[b], held[b] + need):
                table[b][c] = stack.pop()
    for i, x in enumerate(back):
        if count + i < cap:
            free[count + i] = x
    slots = None
    if num_slots is not None:
        slots = [-1] * num_slots
        for b in range(B):
            if served[b]:
                for i in range(max(new[b], 0)):
                    t = max(seq_len[b], 0) + i
                    slots[q_start[b] + i] = table[b][t // page] * page + t % page
    q_start = [min(x, TOP) for x in q_start]
    return q_start, positions, after_len, len(stack), gone_after if window else None, slots, errors
