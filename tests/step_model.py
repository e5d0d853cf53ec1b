"""A step's tables, one sequence and one block after the other (tests only): the plain
statement of what ``pa_step_tables`` computes, on numpy arrays."""
import numpy as np

from paged_kv_cache_395_b200 import pa

BS = 16


def step(tables, lens, news, free, count, T, refs=None):
    """Returns (tables, lens, free, count, refs, slots, positions, row_starts, flags)."""
    tables, free = tables.copy(), free.copy()
    refs = None if refs is None else refs.copy()
    B, M = tables.shape
    N, flags = len(free), 0
    if count < 0 or count > N:
        flags |= pa.PA_EFLAG_FREE_LIST
        count = min(max(count, 0), N)
    stack = [int(x) for x in free[:count]]
    good = [lens[b] >= 0 and news[b] >= -1 and int(lens[b]) + max(int(news[b]), 0) <= M * BS for b in range(B)]
    if not all(good):
        flags |= pa.PA_EFLAG_BAD_LENGTH
    # finished sequences
    entries = []
    for b in range(B):
        if good[b] and news[b] == -1:
            entries += [int(x) for x in tables[b, :-(-int(lens[b]) // BS)]]
    if any(not 0 <= x < N for x in entries):
        flags |= pa.PA_EFLAG_BAD_BLOCK
    entries = [x for x in entries if 0 <= x < N]
    if refs is not None:
        left = [entries.count(x) for x in entries]
        for i, x in enumerate(entries):
            if refs[x] < left[i]:
                flags |= pa.PA_EFLAG_FREE_LIST
        keep = [refs[x] == left[i] and x not in entries[i + 1:] for i, x in enumerate(entries)]
        for x in set(entries):
            refs[x] = max(0, int(refs[x]) - entries.count(x))
        entries = [x for x, k in zip(entries, keep) if k]
    for x in entries:
        if len(stack) >= N:
            flags |= pa.PA_EFLAG_FREE_LIST
            break
        stack.append(x)
    free[:len(stack)] = stack
    # the others
    starts = [0]
    for b in range(B):
        starts.append(starts[-1] + max(0, int(news[b])))
    slots, pos = np.full(T, -1, np.int64), np.full(T, -1, np.int32)
    out = np.array(lens, np.int32).copy()
    asked = 0
    have = len(stack)
    for b in range(B):
        n, L = int(news[b]), int(lens[b])
        if good[b] and n == -1:
            out[b] = 0
        if not good[b] or n <= 0:
            continue
        if starts[b + 1] > T:
            flags |= pa.PA_EFLAG_BAD_LENGTH
            continue
        if L % BS:
            x = int(tables[b, L // BS])
            if not 0 <= x < N:
                flags |= pa.PA_EFLAG_BAD_BLOCK
                continue
            if refs is not None and refs[x] > 1:
                flags |= pa.PA_EFLAG_BAD_LENGTH
                continue
        old, need = -(-L // BS), -(-(L + n) // BS) - -(-L // BS)
        asked += need
        if need and asked > have:
            flags |= pa.PA_EFLAG_OUT_OF_BLOCKS
            continue
        for j in range(old, old + need):
            x = stack.pop()
            tables[b, j] = x
            if refs is not None:
                refs[x] = 1
        for i in range(n):
            p = L + i
            slots[starts[b] + i] = int(tables[b, p // BS]) * BS + p % BS
            pos[starts[b] + i] = p
        out[b] = L + n
    return tables, out, free, len(stack), refs, slots, pos, np.minimum(starts, T).astype(np.int32), flags
