"""Plain 64-bit forms of the prompt, draft-tree and page calls (imported by
their test modules), written from the formulas in include/kvq.h; nothing here
calls the library."""
import numpy as np

import score_ref as ref

ROW, CHANNEL = ref.ROW, ref.CHANNEL


def chains(parents, n):
    """For each of n nodes the nodes from it up to its root."""
    got = []
    for i in range(n):
        p = int(parents[i])
        got.append([i] + (got[p] if 0 <= p < i else []))
    return got


def random_parents(r, B, T, wide=6):
    """Each node follows one of the `wide` before it; some are roots (-1, or a
    value outside [0, i))."""
    p = np.full((B, T), -1, np.int32)
    for b in range(B):
        for i in range(1, T):
            p[b, i] = i - 1 - r.integers(0, min(i, wide))
            if r.random() < 0.08:
                p[b, i] = r.choice([-1, i, T + 3, -(2 ** 31), 2 ** 31 - 1])
    return p


def tree_keys(case, parents, nodes, b):
    """For each node of sequence b the keys (cache rows) it sees."""
    L, n, W = case.lens[b], int(nodes[b]), case.window
    P, up = L - n, chains(parents[b], n)
    got = []
    for chain in up:
        far = len(chain) - 1
        lo = max(0, P + far - W + 1) if W > 0 else 0
        near = chain[:W] if W > 0 else chain
        got.append(list(range(lo, P)) + sorted(P + j for j in near))
    return got


def attend_tree(cache: ref.Cache, parents, nodes, sink=None):
    """out, lse and what the tolerances need, as score_ref.attend."""
    c = cache.case
    B, dv = len(c.lens), (c.dv or c.d) if c.latent else c.d
    out = np.zeros((B, c.c, c.hq, dv))
    absv, f16 = np.zeros_like(out), np.zeros_like(out)
    lse = np.full((B, c.c, c.hq), -np.inf)
    size = np.zeros((B, c.c, c.hq))
    for b in range(B):
        keys = tree_keys(c, parents, nodes, b)
        for h in range(c.hkv):
            k, v = cache.values(b, h, "k"), cache.values(b, h, "v")
            for hq in range(h * c.group, (h + 1) * c.group):
                for i, at in enumerate(keys):
                    q = cache.q[b, i, hq].astype(np.float64)
                    s = k[at] @ q * c.scale
                    size[b, i, hq] = (np.abs(k[at]) @ np.abs(q)).max() * c.scale
                    if c.softcap > 0:
                        s = c.softcap * np.tanh(s / c.softcap)
                    m = s.max()
                    p = np.exp(s - m)
                    lse[b, i, hq] = m + np.log(p.sum())
                    p /= p.sum()
                    f = 1.0 if sink is None else 1.0 / (1.0 + np.exp(float(sink[hq]) - lse[b, i, hq]))
                    out[b, i, hq] = p @ v[at] * f
                    absv[b, i, hq] = p @ np.abs(v[at]) * f
                    # (the roundings of weights and scaled values to f16: score_ref.attend)
                    f16[b, i, hq] = (2.0 ** -10 * absv[b, i, hq]
                                     + 2.0 ** -24 * len(at) * cache.largest(b, h, 0, c.lens[b]))
    return out, lse, absv, f16, size


def accept(parents, nodes, drafts, chosen):
    """The accepted path of each tree, and the token after it."""
    paths, after = [], []
    for b in range(parents.shape[0]):
        n = int(nodes[b])
        path = [0] if n > 0 else []
        while path:
            cur = path[-1]
            kids = [i for i in range(cur + 1, n) if parents[b, i] == cur and drafts[b, i] == chosen[b, cur]]
            if not kids:
                break
            path.append(kids[0])
        paths.append(path)
        after.append(int(chosen[b, path[-1]]) if path else -1)
    return paths, after


class Pages:
    """The page bookkeeping of kvq_pages_step, one sequence and page at a time."""

    SEQ_LEN, NO_BLOCKS, BLOCK_ID = 0x4, 0x40, 0x2

    def __init__(self, bs, width, num_blocks, max_tokens):
        self.bs, self.width, self.nb, self.room = bs, width, num_blocks, max_tokens

    def step(self, held, start, new, table, free, count, parents=None):
        """Returns table, free list, count, lens, cu, slots, positions, flags."""
        table, free, flags = table.copy(), free.copy(), 0
        B, bs = len(held), self.bs
        up = lambda n: -(-int(n) // bs)  # noqa: E731
        valid = [0 <= held[b] <= self.width * bs and 0 <= start[b] <= held[b] and new[b] >= 0 for b in range(B)]
        refused, tokens = [not v for v in valid], 0
        for b in range(B):
            if not valid[b]:
                flags |= self.SEQ_LEN
                continue
            tokens += int(new[b])
            if int(start[b]) + int(new[b]) > self.width * bs or (new[b] > 0 and tokens > self.room):
                refused[b] = True
                flags |= self.SEQ_LEN
        stack = [int(x) for x in free[:count]]
        for b in range(B):  # what comes back
            if not refused[b]:
                for p in range(up(start[b] + new[b]), up(held[b])):
                    stack.append(int(table[b, p]))
        supply, asked = len(stack), 0
        for b in range(B):  # who gets pages
            if valid[b]:
                more = max(0, up(int(start[b]) + int(new[b])) - up(held[b]))
                asked += more
                if not refused[b] and more > 0 and asked > supply:
                    refused[b] = True
                    flags |= self.NO_BLOCKS
        slots, pos = np.full(self.room, -1, np.int64), np.zeros(self.room, np.int64)
        cu, lens, at = np.zeros(B + 1, np.int32), np.array(held, np.int32), 0
        for b in range(B):
            if not refused[b]:
                for p in range(up(held[b]), up(start[b] + new[b])):
                    table[b, p] = stack.pop()
                lens[b] = start[b] + new[b]
                depth = None if parents is None else [len(c) - 1 for c in chains(parents[b], parents.shape[1])]
                for i in range(int(new[b])):
                    row = int(start[b]) + i
                    page = int(table[b, row // bs])
                    if 0 <= page < self.nb:
                        slots[at] = page * bs + row % bs
                    else:
                        flags |= self.BLOCK_ID
                    pos[at] = start[b] + depth[i] if depth is not None and i < len(depth) else row
                    at += 1
            cu[b + 1] = at
        if len(stack) > count:
            free[count:len(stack)] = stack[count:]
        return table, free, len(stack), lens, cu, slots, pos, flags
