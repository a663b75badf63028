"""Plain 64-bit references of the tree-drafting operators, one row or one page
at a time, from their definitions.  Test infrastructure only."""
import math

import numpy as np


def sees(parents, k):
    """[k+1][k+1] bool: whether row r attends to tree row j; all False in rows of absent nodes."""
    m = np.zeros((k + 1, k + 1), bool)
    m[0, 0] = True
    for i in range(k):
        p = int(parents[i])
        if -1 <= p < i and m[p + 1, p + 1]:
            m[i + 1] = m[p + 1]
            m[i + 1, i + 1] = True
    return m


def attention(q, kc, vc, table, lens, parents, scale):
    """float64 arrays q [B][k+1][Hq][D], caches [P][Hkv][page][D].  Returns out, lse, and the bound's parts: the
    weighted sum of |v| and the largest sum |q||k| scale over each row's keys."""
    B, k1, hq, D = q.shape
    P, hkv, page, _ = kc.shape
    g = hq // hkv
    out, absv = np.zeros((B, k1, hq, D)), np.zeros((B, k1, hq, D))
    lse, dot = np.full((B, k1, hq), -np.inf), np.zeros((B, k1, hq))
    for b in range(B):
        n = int(lens[b])
        if n < 0 or n + k1 > table.shape[1] * page:
            continue
        see = sees(parents[b], k1 - 1)
        pos = np.arange(n + k1)
        ids, off = table[b][pos // page], pos % page
        for h in range(hq):
            K, V = kc[ids, h // g, off], vc[ids, h // g, off]
            for r in range(k1):
                if not see[r, r]:
                    continue
                cols = np.concatenate([np.arange(n), n + np.nonzero(see[r])[0]])
                s = (K[cols] * q[b, r, h]).sum(1) * scale
                m = s.max()
                w = np.exp(s - m)
                z = w.sum()
                out[b, r, h] = (w[:, None] * V[cols]).sum(0) / z
                absv[b, r, h] = (w[:, None] * np.abs(V[cols])).sum(0) / z
                lse[b, r, h] = m + math.log(z)
                dot[b, r, h] = (np.abs(K[cols]) * np.abs(q[b, r, h])).sum(1).max() * scale
    return out, lse, absv, dot


# Relative error of a probability that sv_verify_tree forms: its 2^f is good to 4.5e-12 (a table and a polynomial), a sum
# of such terms is no worse, and a probability is one over the other: 9e-12, and the roundings of 64 bits (1e-14).
KERNEL_ERROR = 1e-11


def walk(target, draft, tokens, parents, u, T, onehot, e=KERNEL_ERROR):
    """One sequence: (accepted_len, out_tokens [k+1], path [k], margin).  target [k+1][V], draft [R][V] or None, float64.

    margin: the least distance of a test or of the draw from its border, over what a computation whose probabilities
    have the relative error `e` can be off there; above 1 the result is settled.  `off` bounds the residual's error token
    by token: e r at first; max(0, r - q) is off by at most off + e q, or by nothing where q is larger beyond that, and its
    division by the sum F by another sum(off) / F of itself, so that a residual of two nearly equal rows (a small F) is
    known less well."""
    k, V = len(tokens), target.shape[1]
    bad = False
    R = 0 if draft is None else draft.shape[0]
    for i in range(k):
        p = int(parents[i])
        if p == -2:
            continue
        bad |= p < -2 or p >= i or not 0 <= tokens[i] < V
        if 0 <= p < i:
            bad |= parents[p] == -2 or (not onehot and T != 0 and p + 1 >= R)
    if bad:
        return -1, [-1] * (k + 1), [-1] * k, np.inf
    at, path, margin = -1, [], np.inf
    while True:
        kids = [i for i in range(k) if parents[i] == at]
        row = target[at + 1]
        hit = None
        if T == 0:
            y = int(np.argmax(row))
            hit = next((i for i in kids if tokens[i] == y), None)
        else:
            r = np.exp((row - row.max()) / T)
            r /= r.sum()
            off = e * r
            q = None
            if kids and not onehot:
                d = draft[at + 1]
                q = np.exp((d - d.max()) / T)
                q /= q.sum()
            for i in kids:
                x = tokens[i]
                a, c = u[i] * (1.0 if q is None else q[x]), r[x]
                margin = min(margin, abs(a - c) / max(2 * e * a + off[x], 1e-300))
                if a < c:
                    hit = i
                    break
                if q is None:
                    r, off = r.copy(), off.copy()
                    r[x] = off[x] = 0.0
                else:
                    r, off = np.maximum(0.0, r - q), np.where(r + off < q - e * q, 0.0, off + e * q)
                F, off_F = r.sum(), off.sum()
                if F <= off_F:
                    return None, None, None, 0.0  # nothing is known of what is left
                r, off = r / F, (off + r * (off_F / F)) / F
            if hit is None:
                C = np.cumsum(r)
                goal = u[k] * C[-1]
                y = min(V - 1, int(np.searchsorted(C, goal, side="right")))
                margin = min(margin, float((np.abs(C - goal) / (np.cumsum(off) + u[k] * off.sum() + 1e-14)).min()))
        if hit is None:
            toks = [int(tokens[i]) for i in path] + [y]
            return len(path), toks + [-1] * (k + 1 - len(toks)), path + [-1] * (k - len(path)), margin
        path.append(hit)
        at = hit


def resize(want, table, count, refs, page):
    """In place, on numpy arrays; returns status."""
    n, width = table.shape
    goal = [count[b] if want[b] < 0 else -(-int(want[b]) // page) for b in range(n)]
    ok = [0 <= count[b] <= width and g <= width for b, g in enumerate(goal)]
    for b in range(n):
        while ok[b] and count[b] > goal[b]:
            count[b] -= 1
            refs[table[b, count[b]]] -= 1
            table[b, count[b]] = -1
    free = [i for i in range(len(refs)) if refs[i] == 0]
    out = False
    for b in range(n):
        need = goal[b] - count[b] if ok[b] else 0
        if need <= 0:
            continue
        if out or need > len(free):
            out, ok[b] = True, False
            continue
        for _ in range(need):
            i = free.pop(0)
            refs[i], table[b, count[b]] = 1, i
            count[b] += 1
    return np.array(ok, np.int32)


def fork(src, dst, kc, vc, table, count, refs, lens, page):
    """In place, caches [layers][P]...; returns status."""
    n = len(lens)
    named = [d for d in dst if 0 <= d < n]
    ok = []
    for i, (s, d) in enumerate(zip(src, dst)):
        fine = 0 <= s < n and 0 <= d < n and list(dst).index(d) == i and s not in named and lens[s] >= 0
        ok.append(fine and count0(count, d) and -(-int(lens[s]) // page) <= count[s])
    free = [i for i in range(len(refs)) if refs[i] == 0]
    for i, (s, d) in enumerate(zip(src, dst)):
        if not ok[i]:
            continue
        whole, begun = divmod(int(lens[s]), page)
        if begun and not free:
            ok[i] = False
            continue
        table[d, :whole] = table[s, :whole]
        for x in table[s, :whole]:
            refs[x] += 1
        if begun:
            new = free.pop(0)
            refs[new], table[d, whole] = 1, new
            kc[:, new], vc[:, new] = kc[:, table[s, whole]], vc[:, table[s, whole]]
        count[d], lens[d] = whole + (begun > 0), lens[s]
    return np.array(ok, np.int32)


def count0(count, d):
    return count[d] == 0
