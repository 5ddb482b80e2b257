"""The 4-bit page format, its attention, forks, compaction and beam selection in
64 bits on the host, written from their definitions."""
import numpy as np

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_E = np.arange(127)
SCALES = np.where(_E >= 8, (8 + _E % 8) * 2.0 ** (_E // 8 - 10.0), (_E % 8) * 2.0 ** -9)


def nearest(x, grid):
    """Place of the nearest grid value (ascending, from 0), ties to the even place."""
    x = np.minimum(x, grid[-1])
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    below, above = x - grid[hi - 1], grid[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)


def rounded(x, e=0):
    """What x [..., D] stands as in the pages, and the scales' places."""
    y = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 16) * 2.0 ** -e
    # a / 6 against the scales: a against six times them, which is exact
    s = nearest(np.abs(y).max(-1, keepdims=True), 6 * SCALES)
    step = SCALES[s]
    code = np.where(step > 0, nearest(np.abs(y) / np.where(step > 0, step, 1), CODES), 0)
    return (np.sign(y) * CODES[code] * step * 2.0 ** e).reshape(x.shape), s[..., 0]


def unpack_block(block, page, D, e=(0, 0)):
    """Keys and values [page, D] of one head's block of bytes."""
    g = np.asarray(block).reshape(page // 16, 18 * D)
    out = []
    for j in (0, 1):
        part = g[:, j * 9 * D: (j + 1) * 9 * D]
        codes = part[:, : 8 * D].reshape(page, D // 2)
        s = part[:, 8 * D:].reshape(page, D // 16)
        x = np.empty((page, D))
        for k in (0, 1):
            c = (codes >> (4 * k)) & 15
            x[:, k::2] = np.where(c >= 8, -1.0, 1.0) * CODES[c & 7]
        out.append(x * np.repeat(SCALES[s], 16, axis=1) * 2.0 ** e[j])
    return out


def unpack(pages, table, n, page, D, e=(0, 0)):
    """Keys and values [n, Hkv, D] of a sequence's first n positions; NaN where
    the table names no page.  pages: [n_pages, Hkv, block]."""
    Hkv = pages.shape[1]
    k = np.full((n, Hkv, D), np.nan)
    v = np.full((n, Hkv, D), np.nan)
    for i in range(-(-n // page)):
        if not 0 <= table[i] < len(pages):
            continue
        t = slice(i * page, min(n, (i + 1) * page))
        for h in range(Hkv):
            a, b = unpack_block(pages[table[i], h], page, D, e)
            k[t, h], v[t, h] = a[: t.stop - t.start], b[: t.stop - t.start]
    return k, v


def attention(q, k, v, sees, scale):
    """q [N, Hq, D]; k, v [n, Hkv, D] (NaN keys: no page); sees [N, n].  Returns
    out, lse, the sums of weight times |value|, and the largest scale * sum |q k|."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mass = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    lse, amp = np.full((N, Hq), -np.inf), np.zeros((N, Hq))
    there = ~np.isnan(k[:, 0, 0]) if len(k) else np.zeros(0, bool)
    for h in range(Hq):
        kk, vv = np.nan_to_num(k[:, h // G]), np.nan_to_num(v[:, h // G])
        z = np.where(sees & there, q[:, h] @ kk.T * scale, -np.inf)
        if z.shape[1] == 0:
            continue
        m = z.max(1, keepdims=True)
        ok = np.isfinite(m[:, 0])
        p = np.exp(z - np.where(np.isfinite(m), m, 0))
        total = p.sum(1, keepdims=True)
        w = p / np.where(total > 0, total, 1)
        out[:, h], mass[:, h] = w @ vv, w @ np.abs(vv)
        lse[ok, h] = (m[:, 0] + np.log(np.where(total[:, 0] > 0, total[:, 0], 1)))[ok]
        amp[:, h] = (np.abs(q[:, h]) @ np.abs(kk).T * scale).max(1)
    return out, lse, mass, amp


def fork(table, length, parent, need, page, n_pages):
    """New table, lengths, pages held, copies (from, to), as the definition has it."""
    W = table.shape[1]
    B2 = len(parent)
    row = [int(p) if 0 <= p < len(length) else -1 for p in parent]
    ln = [int(length[r]) if r >= 0 and 0 <= length[r] <= W * page else 0 for r in row]
    full = [n // page for n in ln]
    opened = [int(table[r, f]) if r >= 0 and n % page else -1 for r, f, n in zip(row, full, ln)]
    opened = [o if 0 <= o < n_pages else -1 for o in opened]
    closed = {int(table[r, i]) for r, f in zip(row, full) if r >= 0 for i in range(f)}
    held = {x for x in closed if 0 <= x < n_pages}
    keep, seen = [], set()
    for o in opened:
        keep.append(o >= 0 and o not in closed and o not in seen)
        if o >= 0:
            seen.add(o)
    held |= {o for o, k in zip(opened, keep) if k}
    free = [i for i in range(n_pages) if i not in held]
    new, copies, at = np.full((B2, W), -1, np.int32), [], 0
    for j in range(B2):
        if row[j] < 0:
            continue
        pages = -(-min(max(int(need[j]), ln[j]), W * page) // page)
        kept = full[j] + keep[j]
        for i in range(pages):
            if i < kept:
                x = int(table[row[j], i])
                new[j, i] = x if 0 <= x < n_pages else -1
            else:
                if at < len(free):
                    new[j, i] = free[at]
                    if i == full[j] and opened[j] >= 0:
                        copies.append((opened[j], free[at]))
                at += 1
    return new, np.array(ln, np.int32), len(held) + min(at, len(free)), copies


def compact(table, n_pages):
    held = sorted({int(x) for x in table.ravel() if 0 <= x < n_pages})
    n = len(held)
    free = [i for i in range(n) if i not in set(held)]
    to = {x: x for x in held if x < n}
    to.update(zip([x for x in held if x >= n], free))
    new = np.array([[to.get(int(x), -1) for x in r] for r in table], np.int32).reshape(table.shape)
    return new, n, [(a, b) for a, b in to.items() if a != b]


def beams(logits, scores, finished, eos, T, M):
    """Scores, parents, tokens, finished [B, M] and all candidates' totals."""
    B, K, V = logits.shape
    out = (np.full((B, M), -np.inf), np.full((B, M), -1), np.full((B, M), -1), np.ones((B, M), int))
    every = []
    for b in range(B):
        found = []
        for k in range(K):
            s = float(scores[b, k])
            if not s > -np.inf:
                continue
            if finished is not None and finished[b, k]:
                found.append((-s, k, eos, 1))
                continue
            z = logits[b, k].astype(np.float64) / T
            m = z.max()
            if not np.isfinite(m):
                continue
            t = s + (z - (m + np.log(np.exp(z - m).sum())))
            for x in np.lexsort((np.arange(V), -t))[: M + 1]:
                if t[x] > -np.inf:
                    found.append((-t[x], k, int(x), int(x == eos)))
        found.sort()
        every.append([-x[0] for x in found])
        for i, (x, k, t, f) in enumerate(found[:M]):
            out[0][b, i], out[1][b, i], out[2][b, i], out[3][b, i] = -x, b * K + k, t, f
    return out, every
