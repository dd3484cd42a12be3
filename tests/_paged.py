"""Plain 64-bit forms of the paged serving calls, from their definitions, and input makers for the tests."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def starts_of(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def i32(v, device="cuda"):
    return torch.as_tensor(np.asarray(v, dtype=np.int32), device=device)


def masks64(words, device="cuda"):
    return torch.as_tensor(np.asarray(words, dtype=np.uint64).view(np.int64), device=device)


def tree_words(n, rng):
    words = []
    for i in range(n):
        up = 0 if i == 0 else words[int(rng.integers(0, i))]
        words.append(up | (1 << i))
    return words


def tables(lens, n_new, held, table, ring, state, page, n_rows):
    """What kvq8_paged_tables gives, request by request."""
    n, pages = len(lens), len(ring)
    head, count = int(state[0]), int(state[1])
    same = (table.copy(), ring.copy(), np.array(held), np.array(state), np.zeros(n + 1, np.int32),
            np.full(n_rows, -1, np.int64), np.full(n_rows, -1, np.int32))
    bad = not (0 <= head < pages and 0 <= count <= pages)
    for b in range(n):
        bad |= lens[b] < 0 or n_new[b] < 0 or n_new[b] > lens[b] or not 0 <= held[b] <= table.shape[1]
        bad |= int(lens[b]) > table.shape[1] * page
    if bad or sum(int(x) for x in n_new) > n_rows:
        return same + (2,)
    need = [-(-int(x) // page) for x in lens]
    if count + sum(max(0, held[b] - need[b]) for b in range(n)) > pages:
        return same + (2,)
    if sum(max(0, need[b] - held[b]) for b in range(n)) > count:
        return same + (1,)
    table, ring = table.copy(), ring.copy()
    old = ring.copy()
    tail, slots, positions = head + count, [], []
    for b in range(n):
        for p in range(held[b], need[b]):
            table[b, p] = old[head % pages]
            head, count = head + 1, count - 1
        for p in range(need[b], held[b]):
            ring[tail % pages] = table[b, p]
            tail, count = tail + 1, count + 1
        for pos in range(lens[b] - n_new[b], lens[b]):
            slots.append(int(table[b, pos // page]) * page + pos % page)
            positions.append(pos)
    pad = [-1] * (n_rows - len(slots))
    return (table, ring, np.array(need, np.int32), np.array([head % pages, count], np.int32), starts_of(n_new),
            np.array(slots + pad, np.int64), np.array(positions + pad, np.int32), 0)


class Batch:
    """A paged cache of random values and a batch of windows over it."""

    def __init__(self, seed, hq, hkv, hd, page, lens, n_new, dtype=torch.bfloat16, tree=False, spare=2, pad_rows=0,
                 q_gain=1.0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.hd, self.page, self.lens, self.n_new = hq, hkv, hd, page, list(lens), list(n_new)
        self.scale, self.dtype = 1.0 / math.sqrt(hd), dtype
        held = [max(0, -(-n // page)) for n in lens]
        pages = sum(held) + spare
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(held + [1])), -7, dtype=np.int32)  # what is not held is no page
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (pages, hkv, page, hd)
        self.codes = [np.clip(np.rint(rng.standard_normal(shape) * 45), -127, 127).astype(np.int8) for _ in range(2)]
        self.scales = [(0.02 * np.exp(0.4 * rng.standard_normal(shape[:3] + (hd // 32,)))).astype(np.float16)
                       for _ in range(2)]
        # rows of a page behind the request's length hold anything
        for b, n in enumerate(lens):
            if n % page:
                for c, s in zip(self.codes, self.scales):
                    c[self.table[b, n // page], :, n % page:] = 127
                    s[self.table[b, n // page], :, n % page:] = np.float16(np.nan)
        self.starts = starts_of(n_new)
        rows = int(self.starts[-1]) + pad_rows
        self.q = torch.from_numpy(rng.standard_normal((rows, hq, hd)).astype(np.float32) * q_gain).to(dtype)
        self.words = None
        if tree:
            self.words = sum((tree_words(n, rng) for n in n_new), []) + [0] * pad_rows

    def cache(self):
        from speculative_verify_attention_gb300 import KVPagedCacheQ8
        k, v = (torch.from_numpy(c).cuda() for c in self.codes)
        ks, vs = (torch.from_numpy(s).cuda() for s in self.scales)
        return KVPagedCacheQ8.from_planes(k, ks, v, vs)

    def call(self, cache=None, out=None, **more):
        from speculative_verify_attention_gb300 import attn_verify_paged_q8
        cache = cache or self.cache()
        if out is None:
            out = torch.full(self.q.shape, 77.0, dtype=self.dtype, device="cuda")
        more.setdefault("max_rows", max(self.n_new))
        more.setdefault("softmax_scale", self.scale)
        more.setdefault("q", self.q.cuda())
        mask = None if self.words is None else masks64(self.words)
        attn_verify_paged_q8(more.pop("q"), cache, i32(self.table), i32(self.lens), i32(self.starts), window_mask=mask,
                             out=out, **more)
        return out

    def visible(self, b, t):
        """Keys of request b that its row t sees."""
        n, rows = self.lens[b], self.n_new[b]
        seen = np.arange(n) < n - rows
        for j in range(rows):
            if (j <= t) if self.words is None else (self.words[self.starts[b] + t] >> j) & 1:
                seen[n - rows + j] = True
        pages = self.table[b, np.arange(n) // self.page]
        return seen & (pages >= 0) & (pages < len(self.codes[0]))

    def values(self, b):
        """K and V of request b in 64 bits, [head][key][dim]; zeros on pages that there are not."""
        n = self.lens[b]
        pages, off = self.table[b, np.arange(n) // self.page], np.arange(n) % self.page
        good = (pages >= 0) & (pages < len(self.codes[0]))
        pages = np.where(good, pages, 0)
        out = []
        for c, s in zip(self.codes, self.scales):
            x = c[pages, :, off].astype(np.float64) * np.repeat(s[pages, :, off].astype(np.float64), 32, axis=-1)
            out.append(np.where(good[:, None, None], x, 0.0).transpose(1, 0, 2))
        return out

    def expect(self, scale=None, rows=None):
        """(row, head) -> (o, bound): the definition in 64 bits, and how far the call may be from it.

        The call rounds k, v and p to fp16 (half a step 2^-11 of each) and the result to its own type; q is exact
        (bf16 times a power of two fits fp16 but for values 2^-10 and more below the row's largest, off by at most
        2^-25 of it).  A score is off by at most ds = scale * (sum |q k| (2^-11 + hd 2^-24) + sum |k| max|q| 2^-24
        + sum |q| 2^-25), a weight relative to the sum of weights by 2 ds + 2^-11 to first order (1.1 covers the
        second, ds being below 0.05), and sums over the keys in fp32 by keys * 2^-24 and the exponential's
        approximation 2^-21."""
        scale = self.scale if scale is None else scale
        group, found = self.hq // self.hkv, {}
        for b in range(len(self.lens)):
            if not self.n_new[b]:
                continue
            k, v = self.values(b)
            for t in range(self.n_new[b]):
                r = int(self.starts[b]) + t
                if rows is not None and r not in rows:
                    continue
                seen = self.visible(b, t)
                for h in range(self.hq):
                    q = self.q[r, h].double().numpy()
                    kk, vv = k[h // group][seen], v[h // group][seen]
                    if not len(kk):
                        found[r, h] = (np.zeros(self.hd), np.zeros(self.hd))
                        continue
                    s = scale * (kk @ q)
                    p = np.exp(s - s.max())
                    w = p / p.sum()
                    o = w @ vv
                    ds = scale * (np.abs(kk) @ np.abs(q) * (2.0 ** -11 + self.hd * 2.0 ** -24)
                                  + np.abs(kk).sum(1) * np.abs(q).max() * 2.0 ** -24 + np.abs(q).sum() * 2.0 ** -25)
                    assert ds.max() < 0.05
                    rel = 1.1 * (2 * ds.max() + 2.0 ** -10) + len(kk) * 2.0 ** -24 + 2.0 ** -21
                    off = rel * (w @ np.abs(vv)) + len(kk) * 2.0 ** -30 * np.abs(vv).max(0)
                    found[r, h] = (o, off + (np.abs(o) + off) * HALF_STEP[self.dtype])
        return found

    def check(self, out, expected=None):
        got = out.double().cpu().numpy()
        worst = 0.0
        for (r, h), (o, off) in (expected or self.expect()).items():
            d = np.abs(got[r, h] - o)
            assert np.all(d <= off), (r, h, float((d - off).max()), float(d.max()))
            worst = max(worst, float((d / np.maximum(off, 1e-30)).max()))
        live = int(self.starts[-1])
        assert torch.all(out[live:] == 77.0) or out.shape[0] == live
        return worst


def adjusted(logits, starts, penalties=None, counts=None, state_of=None, tokens=None, words=None, bias=None,
             grammar=None, grammar_of=None):
    """(x, bound) of logits_adjust in 64 bits, row by row; rows of no request are NaN.  bias: list of [(token, value)]
    per request.  Six fp32 operations, each off by half a step of a number no larger than the sum of magnitudes."""
    x = logits.double().numpy().copy()
    n_rows, vocab = x.shape
    size = np.abs(np.where(np.isfinite(x), x, 0.0))
    done = np.zeros(n_rows, bool)
    for b in range(len(starts) - 1):
        for r in range(starts[b], starts[b + 1]):
            done[r] = True
            word = np.zeros(vocab, np.int64)
            st = b if state_of is None else state_of[b]
            if counts is not None and 0 <= st < len(counts):
                word = counts[st].astype(np.int64) & 0xffffffff
            c = word & 0x7fffffff
            for j in range(starts[b + 1] - starts[b]):
                t = r - starts[b]
                if tokens is not None and ((j <= t) if words is None else (words[r] >> j) & 1):
                    v = tokens[starts[b] + j]
                    if 0 <= v < vocab:
                        c[v] += 1
            if penalties is not None:
                rep, freq, pres = (float(z) for z in penalties[b])
                with np.errstate(invalid="ignore"):
                    y = np.where(x[r] > 0, x[r] / rep, x[r] * rep)
                    x[r] = np.where((c > 0) | (word >> 31 != 0), y, x[r]) - (freq * c + pres * (c > 0))
                size[r] = size[r] * max(rep, 1 / rep) + abs(freq) * c + abs(pres)
            if bias is not None:
                for v, val in dict(bias[b]).items():
                    if 0 <= v < vocab:
                        x[r, v] += np.float32(val)
                        size[r, v] += abs(val)
            if grammar is not None:
                g = r if grammar_of is None else grammar_of[r]
                if 0 <= g < len(grammar):
                    w = grammar[g].astype(np.int64) & 0xffffffff
                    allowed = (w[np.arange(vocab) // 32] >> (np.arange(vocab) % 32)) & 1
                    x[r] = np.where(allowed == 1, x[r], -np.inf)
    x[~done] = np.nan
    return x, 6 * 2.0 ** -24 * size
