"""The fork of requests' pages, one request and one page after another."""
from __future__ import annotations


def fork(rows, lens, table, refs, free, count, new_table, page):
    """Lists in, lists out; refs, free and new_table are changed.  Returns new_lens, copies (src, dst, rows), info."""
    B, width = len(rows), len(table[0])
    lens = [min(max(n, 0), width * page) for n in lens]
    count = min(max(count, 0), len(free))
    good = lambda p: 0 <= p < len(refs)  # noqa: E731
    rows = [r if 0 <= r < B else -1 for r in rows]
    children = [rows.count(p) for p in range(B)]
    for p, c in enumerate(children):
        if c > 1:
            for j in range(lens[p] // page):
                if good(table[p][j]):
                    refs[table[p][j]] += c - 1
    freed = []
    # Nobody left: found out after all have let go, noted at the last one's place.
    for j in range(width):
        ends = [(p, table[p][j]) for p in range(B) if children[p] == 0 and j < -(-lens[p] // page) and good(table[p][j])]
        for i, (p, x) in enumerate(ends):
            refs[x] -= 1
        for i, (p, x) in enumerate(ends):
            if refs[x] < 0 and x not in [y for _, y in ends[i + 1:]]:
                freed.append(x)
                refs[x] = 0
    top = free[:count] + freed
    free[count:count + len(freed)] = freed[:len(free) - count]
    new_lens, copies, taken, refused = [0] * B, [(-1, -1, 0)] * B, 0, 0
    for b, r in enumerate(rows):
        if r < 0:
            continue
        whole, part = lens[r] // page, lens[r] % page
        first = rows.index(r) == b
        for j in range(whole + (part > 0 and first)):
            new_table[b][j] = table[r][j]
        new_lens[b] = lens[r]
        if part and not first:
            if taken < len(top):
                x = top[len(top) - 1 - taken]
                taken += 1
                new_table[b][whole] = x
                copies[b] = (table[r][whole], x, part)
            else:
                refused += 1
                new_lens[b] = 0
                for j in range(whole):
                    if good(table[r][j]):
                        refs[table[r][j]] -= 1
    return new_lens, copies, [len(freed), taken, min(len(top), len(free)) - taken, refused]
