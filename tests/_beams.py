"""Plain forms of the calls around beams, trees and rotary positions, from their definitions: 64 bits, request by request."""
from __future__ import annotations

import math

import numpy as np

EPS = 2.0 ** -24


def continuations(x, starts, scores=None, weights=None, ended=None):
    """For each request the list of (weight * total, row, rank in its row, token, total), best first: everything it has."""
    out = []
    for b in range(len(starts) - 1):
        got = []
        for r in range(starts[b], starts[b + 1]):
            score = 0.0 if scores is None else float(scores[r])
            weight = 1.0 if weights is None else float(weights[r])
            if not math.isfinite(score) or not (0 < weight < math.inf):
                continue
            if ended is not None and ended[r] >= 0:
                got.append((weight * score, r, 0, int(ended[r]), score))
                continue
            row = x[r].astype(np.float64) + 0.0
            if np.isnan(row).any() or (row == np.inf).any() or (row == -np.inf).all():
                continue
            top = row.max()
            norm = math.log(math.fsum(np.exp(row - top).tolist())) + top
            order = np.argsort(-row, kind="stable")
            order = order[row[order] > -np.inf][:64]
            got += [(weight * (score + (row[v] - norm)), r, k, int(v), score + (row[v] - norm)) for k, v in enumerate(order)]
        got.sort(key=lambda c: (-c[0], c[1], c[2]))
        out.append(got)
    return out


def slack(x):
    """How far the call's log sum exp may be from the exact one, for logits of size up to |x|: a term's argument is rounded once
    (at most 2^-24 of it, and terms with arguments below -24 are together below 2^18 2^-24 of the sum), the exponential 2^-22, 37 additions
    in fp32 (32 in a lane, 5 in a warp), parts rounded to 2^-33 each; log2 e is 1.4e-8 off, of a spread of 2 max|x|."""
    finite = x[np.isfinite(x)].astype(np.float64)
    size = float(np.abs(finite).max()) if finite.size else 0.0
    return (24 + 4 + 37 + 1) * EPS + 2.8e-8 * size


def check_selection(x, starts, n_out, got, scores=None, weights=None, ended=None):
    """(parents, tokens, totals) against the definition.  Totals of different rows that are nearer to one another than the call's
    sums are exact may change places; the continuations of one row may not."""
    parents, tokens, totals = (t.cpu().numpy() for t in got)
    off = slack(x)
    for b, want in enumerate(continuations(x, starts, scores, weights, ended)):
        n = min(n_out, len(want))
        assert np.all(parents[b, n:] == -1) and np.all(tokens[b, n:] == -1) and np.all(totals[b, n:] == -np.inf), b
        by = {(c[1], c[3]): c for c in want}
        used = {}
        for k in range(n):
            r, v = int(parents[b, k]), int(tokens[b, k])
            assert (r, v) in by, (b, k, r, v)
            order, _, rank, _, total = by[r, v]
            assert rank == used.get(r, 0), (b, k, r, v)     # a row's own continuations in their order, none left out
            used[r] = rank + 1
            w = 1.0 if weights is None else float(weights[r])
            tol = off * max(w, *(1.0 if weights is None else float(weights[c[1]]) for c in want[k:k + 1])) + 1e-14 * abs(order)
            assert abs(order - want[k][0]) <= 2 * tol, (b, k, order, want[k])
            assert abs(float(totals[b, k]) - total) <= off + abs(total) * EPS, (b, k)


def fork_counts(parents, state_of, counts):
    """(state_of_out, counts, status)."""
    n_states, m = len(counts), len(parents)
    none = (np.full(m, -1, np.int32), counts.copy())
    state = [s if 0 <= s < n_states else -1 for s in state_of]
    if any(q >= len(state) for q in parents):
        return none + (2,)
    alive = sorted({q for q in parents if q >= 0})
    rows = [state[q] for q in alive if state[q] >= 0]
    if len(set(rows)) < len(rows):
        return none + (2,)
    free = [r for r in range(n_states) if r not in set(rows)]
    out, new, seen = [], counts.copy(), set()
    for q in parents:
        if q < 0 or state[q] < 0:
            out.append(-1)
        elif q not in seen:
            out.append(state[q])
            seen.add(q)
        else:
            if not free:
                return none + (1,)
            out.append(free.pop(0))
            new[out[-1]] = counts[state[q]]
    return np.array(out, np.int32), new, 0


def fork_pages(parents, lens, held, page, table, shares, ring, state, table_out):
    """What kvq8_paged_fork gives, sequence by sequence: table_out, lens_out, held_out, shares, ring, ring state, copy list, status."""
    m, n, pages = len(parents), len(lens), len(ring)
    head, count = int(state[0]), int(state[1])
    zero = np.zeros(m, np.int32)
    none = (table_out.copy(), zero, zero, np.array(shares), ring.copy(), np.array(state), zero - 1, zero - 1, zero)
    bad = not (0 <= head < pages and 0 <= count <= pages) or any(q >= n for q in parents)
    bad = bad or any(not 0 <= h <= table.shape[1] for h in held)
    if bad or any(q >= 0 and not 0 <= lens[q] <= held[q] * page for q in parents):
        return none + (2,)
    table_out, lens_out, held_out = table_out.copy(), zero.copy(), zero.copy()
    src, dst, rows = zero - 1, zero - 1, zero.copy()
    holders = np.array(shares, np.int64)          # beyond the first
    seen, ring, ring0 = set(), ring.copy(), ring.copy()
    taken = 0
    change = {}

    def add(pg, by):
        if 0 <= pg < pages:
            change[pg] = change.get(pg, 0) + by

    for q in range(n):
        for k in range(held[q]):
            add(int(table[q, k]), -1)
    for i, q in enumerate(parents):
        if q < 0:
            continue
        need = -(-int(lens[q]) // page)
        table_out[i, :need] = table[q, :need]
        lens_out[i], held_out[i] = lens[q], need
        part = int(lens[q]) % page
        first = q not in seen
        seen.add(q)
        tail = int(table[q, need - 1]) if part else -1
        if part and not (first and (not 0 <= tail < pages or shares[tail] == 0)):
            if taken == count:
                return none + (1,)
            table_out[i, need - 1] = ring0[(head + taken) % pages]
            src[i], dst[i], rows[i] = tail, ring0[(head + taken) % pages], part
            taken += 1
            need -= 1
        for k in range(need):
            add(int(table[q, k]), 1)
    freed = []
    for pg in sorted(change):
        holders[pg] += change[pg]
        if holders[pg] < 0:
            holders[pg] = 0
            freed.append(pg)
    for k, pg in enumerate(freed):
        ring[(head + count + k) % pages] = pg
    return (table_out, lens_out, held_out, holders.astype(np.int32), ring,
            np.array([(head + taken) % pages, count - taken + len(freed)]), src, dst, rows, 0)


def rotated(x, angles, pairs):
    """x [n][heads][hd] in 64 bits, turned by angles [n][rot / 2]."""
    x = x.astype(np.float64).copy()
    half = angles.shape[1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    c, s = np.cos(angles)[:, None], np.sin(angles)[:, None]
    u, v = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = u * c - v * s, v * c + u * s
    return x


def angles_of(positions, freq, axis_of=None):
    """[n][rot / 2] in turns reduced in whole numbers, then radians: positions [axes][n] of any size."""
    two_pi = 2 * math.pi
    half, n = len(freq), positions.shape[1]
    out = np.zeros((n, half))
    for i in range(half):
        a = 0 if axis_of is None else int(axis_of[i])
        if not 0 <= a < len(positions):
            continue
        num, den = float(freq[i]).as_integer_ratio()
        for t in range(n):
            turns = int(positions[a, t]) * num * _INV_TAU
            out[t, i] = (turns % (den << 256)) / (den << 256) * two_pi
    return out


_INV_TAU = int("18428883373056725475459024596439793651824491331936921676307065986443608256856")  # 2^256 / (2 pi)
