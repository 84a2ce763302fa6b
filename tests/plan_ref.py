"""The page plan's definition with refusals: an allocator on the host that takes one sequence after the other."""


def plan(lens, new, table, free, count, page, tokens, groups=None, prefix=None):
    """(table, cu_new, positions, slots, lens, pages left, whether anything was refused)."""
    table = [list(r) for r in table]
    B, width = len(lens), len(table[0])
    reach = width * page
    left = min(max(count, 0), len(free))
    refused = left != count
    cu, after, taken, had = [0], [], [], []
    for b, (n, m) in enumerate(zip(lens, new)):
        known = 0 <= n <= reach                 # what a length outside the table says is not used for anything
        if not known or m < 0 or n + m > reach:
            refused, m = True, 0
        held = -(-n // page) if known else 0
        need = -(-(n + m) // page) - held if known else 0
        ok = need <= left
        for i in range(need):
            table[b][held + i] = free[left - 1 - i] if ok else -1
        if ok:
            left -= need
        else:
            refused = True
        had.append(n if known else -1)
        taken.append(m)
        after.append(n + m if ok else n)
        cu.append(cu[-1] + m)
    for a, z, n in zip(groups or [], (groups or [])[1:], prefix or []):
        for b in range(a + 1, z):
            if not 0 < n <= had[b]:
                continue
            for j in range(n // page):
                idle = had[a] == 0 and taken[a] == 0
                whole = had[a] >= 0 and (j + 1) * page <= after[a]   # the first's page, filled after this step
                if (idle or whole) and table[a][j] >= 0:
                    table[b][j] = table[a][j]
    positions, slots = [], []
    for b in range(B):
        for p in range(lens[b], lens[b] + taken[b]):
            at = table[b][p // page]
            positions.append(p)
            slots.append(at * page + p % page if after[b] > p and at >= 0 else -1)
    pad = [-1] * max(0, tokens - len(positions))
    return table, cu, (positions + pad)[:tokens], (slots + pad)[:tokens], after, left, refused
