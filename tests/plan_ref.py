"""A plain reference of the planned step: Python integers, one request after the other."""


def plan(seq, new, table, free, num_free, bs, T, finished=None):
    """Lists of whole numbers (table and free are changed); returns slots, positions, cu, seq, num_free, served, ok."""
    B, cols, cap, ok = len(seq), len(table[0]), len(free), True
    up = lambda n: -(-n // bs)
    seq = [max(x, 0) for x in seq]
    num_free = min(max(num_free, 0), cap)
    for b in range(B):
        if finished and finished[b]:
            for c in range(min(up(seq[b]), cols)):
                if num_free < cap:
                    free[num_free] = table[b][c]
                    num_free += 1
                else:
                    ok = False
            seq[b] = 0
    top, want, rows, taken = num_free, 0, 0, 0
    slots, positions, cu, served = [-1] * T, [0] * T, [0], []
    for b in range(B):
        n = max(new[b], 0)
        have, need = up(seq[b]), up(seq[b] + n) - up(seq[b])
        fits = have + need <= cols
        if not fits:
            need = 0
        good = fits and (need == 0 or want + need <= top) and rows + n <= T
        if good:
            for i in range(need):
                table[b][have + i] = free[top - 1 - want - i]
            taken = max(taken, want + need) if need else taken
        want += need
        for i in range(n):
            if rows + i < T:
                p = seq[b] + i
                positions[rows + i] = p
                slots[rows + i] = table[b][p // bs] * bs + p % bs if good else -1
        rows += n
        cu.append(min(rows, T))
        if good:
            seq[b] += n
        served.append(good)
        ok = ok and good
    return slots, positions, cu, seq, top - taken, served, ok
