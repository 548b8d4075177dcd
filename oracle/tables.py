"""Oracle: block tables, the free-page ring and the token list of a step, request by request.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain Python integers.
A request of x positions holds one page per N * P positions begun (the widened
page of SGLang "Decode context parallelism", "Virtual KV layout").
"""

from __future__ import annotations

from . import layout

BAD_PAGE_INDEX, BAD_LENGTH, NO_PAGES, TOO_MANY_TOKENS, BAD_POOL = 2, 16, 128, 256, 512


def update(seq_lens, new_lens, table, max_pages, ring, head, count, N, I, P, T=None):
    """One step on Python lists (seq_lens, table, ring are changed in place).

    Returns (head, count, tokens, cu, status): tokens = [(pos, req, owner, row, slot)], all lists
    untouched and no tokens if status is not 0.
    """
    B, cap, span = len(seq_lens), len(ring), N * P
    status = 0

    def pages(x):
        return (x + span - 1) // span

    take = give = grown = 0
    for a, n in zip(seq_lens, new_lens):
        if a < 0 or n < 0 or max(a, n) > (1 << 62) // B:
            status |= BAD_LENGTH
        elif max(pages(a), pages(n)) > max_pages:
            status |= BAD_PAGE_INDEX
        else:
            take += max(0, pages(n) - pages(a))
            give += max(0, pages(a) - pages(n))
            grown += max(0, n - a)
    if not (0 <= head < cap and 0 <= count <= cap) or give > cap - count:
        status |= BAD_POOL
    elif take > count:
        status |= NO_PAGES
    if T is not None and grown > T:
        status |= TOO_MANY_TOKENS
    if status:
        return head, count, [], [0] * (B + 1), status
    free = [ring[(head + i) % cap] for i in range(count)]
    back = []
    tokens, cu = [], [0]
    for b in range(B):
        a, n = seq_lens[b], new_lens[b]
        for k in range(pages(a), pages(n)):
            table[b][k] = free.pop(0)
        for k in range(pages(n), pages(a)):
            back.append(table[b][k])
            table[b][k] = -1
        for p in range(a, n):
            row = int(layout.local_row(p, N, I))
            tokens.append((p, b, int(layout.owner(p, N, I)), row, table[b][row // P] * P + row % P))
        cu.append(len(tokens))
        seq_lens[b] = n
    new_head = (head + count - len(free)) % cap
    for i, page in enumerate(back):
        ring[(head + count + i) % cap] = page
    return new_head, len(free) + len(back), tokens, cu, 0
