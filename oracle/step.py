"""A decoding step's tables, the verification of drafted tokens, and what stays of the step, fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Written sequence by sequence, from the definitions: pages are popped from and pushed onto a list,
masks are sets of ancestors, verification keeps the whole left-over distribution and its sum after
every drafted token that goes.
"""

import numpy as np


def plan(free, lens, counts, table, rows, page, pages, parents=None, words=0, shift=None):
    """free: list of free pages (the last given out first); table [B][width] int array. Returns a
    dict of the outputs, `free` and `table` after the call; the arguments stay."""
    free, table = list(free), np.array(table, dtype=np.int64)
    B, width = table.shape if table.ndim == 2 else (len(lens), 0)
    out = {"slots": np.full(rows, -1, np.int64), "positions": np.zeros(rows, np.int64), "kv_lens": [],
           "status": [], "tree": np.zeros((rows, words), np.uint32)}
    offsets, out_of_pages = [0], False
    for b in range(B):
        n, c = max(0, int(lens[b])), max(0, int(counts[b]))
        first = offsets[-1]
        offsets.append(first + c)
        status = 0
        need = -(-(n + c) // page) - -(-n // page)
        if n + c > width * page:
            status = 2
        elif c and first + c > rows:
            status = 3
        elif need:
            out_of_pages = out_of_pages or need > len(free)
            status = 1 if out_of_pages else 0
        out["status"].append(status)
        out["kv_lens"].append(0 if status else n + c)
        if status:
            continue
        for j in range(-(-n // page), -(-(n + c) // page)):
            table[b, j] = free.pop()
        seen, depth = [], []  # ancestors as a whole number's bits, steps to the root
        for i in range(c):
            r, token = first + i, n + i
            p = table[b, token // page]
            if 0 <= p < pages:
                out["slots"][r] = p * page + token % page
            up = i - 1 if parents is None else int(parents[r])
            chained = i > 0 and 0 <= up < i
            seen.append((seen[up] if chained else 0) | 1 << i)
            depth.append(depth[up] + 1 if chained else 0)
            out["positions"][r] = n + depth[i] + (0 if shift is None else int(shift[b]))
            for w in range(words):
                out["tree"][r, w] = seen[i] >> (32 * w) & 0xffffffff
            if parents is None and not words:
                seen[i] = 0  # (nobody looks)
    out["q_offsets"] = np.minimum(offsets, rows)
    out["free"], out["table"] = free, table
    return out


def keep(free, lens, kept, table, page, q_offsets=None, status=None):
    """(new lengths, free list, moves): moves as (sequence, place j of those kept)."""
    back, ends, moves = [], [], []
    for b in range(len(lens)):
        n = max(0, int(lens[b]))
        c = 0 if q_offsets is None or (status is not None and status[b]) else int(q_offsets[b + 1] - q_offsets[b])
        k = max(0, min(int(kept[b]), c))
        end = 0 if kept[b] < 0 else n + k
        ends.append(end)
        back += [int(x) for x in table[b][-(-end // page):-(-(n + c) // page)]]
        moves += [(b, j) for j in range(1, k)]
    return np.array(ends), list(free) + back[::-1], moves


def distribution(x, kind, T):
    """The probabilities of a row, or None where its logits (greedy: its values) make none."""
    x = np.asarray(x, dtype=np.float64)
    if kind == "probabilities" and T > 0:
        return x
    if np.isnan(x).any() or (x == np.inf).any():
        return None
    if x.max() == -np.inf:
        return None
    if not T > 0:
        if kind == "probabilities" and x.max() <= 0:
            return None
        return (np.arange(x.size) == np.argmax(x)).astype(np.float64)
    e = np.exp((x - x.max()) / T) if np.isfinite(T) else (x > -np.inf).astype(np.float64)
    return e / e.sum()


def sample(w, u):
    """(first i with cumsum(w)_i > u sum(w), distance to the nearest border relative to the sum)."""
    c = np.cumsum(w)
    if not c[-1] > 0 or not np.isfinite(c[-1]):
        return -1, 1.0
    goal = max(0.0, u if u == u else 0.0) * c[-1]
    hit = np.nonzero(c > goal)[0]
    i = int(hit[0]) if hit.size else int(np.nonzero(w > 0)[0][-1])
    inner = c[np.nonzero(w > 0)[0][:-1]]
    return i, float(np.min(np.abs(inner - goal)) / c[-1]) if inner.size else 1.0


def verify(target, tokens, uniforms, offsets, draft=None, parents=None, temperature=None, target_kind="logits",
           draft_kind="logits"):
    """(kept, tokens, path, margins [sequences][2]): margins are the smallest distances of a sequence's
    decisions to their borders, relative to what is compared: of the tests, of the new token."""
    M = len(tokens)
    kept, out, path, margins = [], np.full(M, -1), np.full(M, -1), np.ones((len(offsets) - 1, 2))
    for b in range(len(offsets) - 1):
        margin = margins[b]
        lo, n = int(offsets[b]), int(offsets[b + 1] - offsets[b])
        if n == 0:
            kept.append(0)
            continue
        T = 1.0 if temperature is None else float(temperature[b])
        greedy = not T > 0
        at, k = 0, 1
        path[lo] = 0
        while True:
            whole = distribution(target[lo + at], target_kind, T)
            children = [r for r in range(at + 1, n) if (r - 1 if parents is None else parents[lo + r]) == at]
            q = None
            p, S, found, bad = whole, 1.0, None, whole is None
            for r in children:
                x, u = int(tokens[lo + r]), float(uniforms[lo + r])
                if not 0 <= x < len(target[lo]) or bad:
                    continue
                if greedy:
                    if p[x] == 1.0:
                        found = r
                        break
                    continue
                if draft is not None and q is None:
                    q = distribution(draft[lo + at], draft_kind, T)
                    if q is None:
                        bad = True
                        continue
                if not np.isfinite(p[x]) or (q is not None and not np.isfinite(q[x])):
                    bad = True  # (probabilities: of logits all are finite)
                    continue
                # S is what is left of p's sum (1 at first): p / S against q
                left, right = (u * S * q[x], p[x]) if draft is not None else (u * S, p[x])
                if left != right:
                    margin[0] = min(margin[0], abs(left - right) / max(abs(left), abs(right)))
                if left < right:
                    found = r
                    break
                if draft is not None:
                    p = np.maximum(p - S * q, 0.0)
                    S = p.sum()
                else:
                    S -= p[x]
                    p = p.copy()
                    p[x] = 0.0
            if found is None:
                break
            out[lo + k - 1], path[lo + k] = tokens[lo + found], found
            at, k = found, k + 1
        if bad:
            new = -1
        elif q is not None and not np.isfinite(q).all():
            new = -1
        else:
            w = np.maximum(p, 0.0)
            new, margin[1] = sample(w if w.sum() > 0 else np.maximum(whole, 0.0), float(uniforms[lo]))
        out[lo + k - 1] = new
        kept.append(k)
    return np.array(kept), out, path, margins
