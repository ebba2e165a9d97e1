"""The page plan from its definition: Python lists, one request after the other."""


def pages_for(n, page):
    return -(-n // page)


def plan(q_len, kv_len, first, table, free, n_free, *, page_size, n_tokens, drop=None):
    """A dict of lists as PagePlan names them."""
    B, W, cap = len(q_len), len(table[0]) if table else 0, len(free)
    q, old = [max(x, 0) for x in q_len], [max(x, 0) for x in kv_len]
    n_free = max(n_free, 0)
    stack, rows, kept, start = list(free[:n_free]), [], [], []
    fits = all(pages_for(n, page_size) <= W for n in old) and sum(q) <= n_tokens
    for b in range(B):
        pages = pages_for(old[b], page_size)
        d = 0 if drop is None else pages if drop[b] < 0 else min(drop[b], pages)
        ends = drop is not None and drop[b] < 0
        kept.append(max(old[b] - d * page_size, 0))
        start.append(0 if ends else first[b] + old[b] - kept[b])
        fits = fits and pages_for(kept[b] + q[b], page_size) <= W
        if fits:
            stack += table[b][:d]
            rows.append(table[b][d:pages])
    fits = fits and len(stack) <= cap
    lack = 0
    if fits:
        wants = [pages_for(kept[b] + q[b], page_size) - len(rows[b]) for b in range(B)]
        lack = max(sum(wants) - len(stack), 0)
    if not fits or lack:
        same = list(free[:min(n_free, cap)])
        return dict(cu_q=[0] * (B + 1), positions=[0] * n_tokens, slots=[-1] * n_tokens, kv_len=old, first=list(first),
                    block_table=[list(r) for r in table], free_pages=same + [-1] * (cap - len(same)), n_free=[n_free],
                    missing=[lack if fits else -1])
    cu, positions, slots = [0], [], []
    for b in range(B):
        rows[b] = rows[b] + [stack.pop() for _ in range(wants[b])]
        for place in range(kept[b], kept[b] + q[b]):
            positions.append(start[b] + place)
            slots.append(rows[b][place // page_size] * page_size + place % page_size)
        cu.append(cu[-1] + q[b])
    rest = n_tokens - cu[-1]
    return dict(cu_q=cu, positions=positions + [0] * rest, slots=slots + [-1] * rest,
                kv_len=[k + n for k, n in zip(kept, q)], first=start, block_table=[r + [-1] * (W - len(r)) for r in rows],
                free_pages=stack + [-1] * (cap - len(stack)), n_free=[len(stack)], missing=[0])
