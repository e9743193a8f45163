"""Plain 64-bit implementations of the paged-cache operators (numpy), written from their
definitions in include/mk.h, one row, head and token at a time."""
import math

import numpy as np


def rope(x, pos, freqs, interleaved, mscale):
    """x [heads, head_dim] rotated at one position."""
    y = np.array(x, dtype=np.float64)
    n = len(freqs)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        t = math.fmod(float(pos) * float(freqs[i]), 2 * math.pi)
        c, s = mscale * math.cos(t), mscale * math.sin(t)
        ya, yb = y[:, a].copy(), y[:, b].copy()
        y[:, a], y[:, b] = ya * c - yb * s, yb * c + ya * s
    return y


def attend(q, k, v, seen, scale, softcap):
    """One query head [d] over keys and values [t, d] of which `seen` [t] (bool) count: the
    output, the log-sum-exp, sum p |v|, and the largest scale * sum |q||k|."""
    k, v = k[seen], v[seen]
    if not len(k):
        return np.zeros(q.shape[0]), -math.inf, np.zeros(q.shape[0]), 0.0
    s = (k @ q) * scale
    size = (np.abs(k) @ np.abs(q)).max() * abs(scale)
    if softcap:
        s = softcap * np.tanh(s / softcap)
    m = s.max()
    p = np.exp(s - m)
    z = p.sum()
    return (p @ v) / z, m + math.log(z), (p @ np.abs(v)) / z, size


class Pages:
    """The state of mk_update_pages, one step at a time in Python: table [rows][width], lens, refs and a
    value per page (what its copies carry along)."""

    def __init__(self, rows, width, n_pages, page_size):
        self.table = -np.ones((rows, width), dtype=np.int32)
        self.lens = np.zeros(rows, dtype=np.int32)
        self.refs = np.zeros(n_pages, dtype=np.int32)
        self.ps = page_size

    def update(self, parents, reserve):
        """The copies [(src, dst)], or None where the call is refused."""
        rows, width = self.table.shape
        lens = np.zeros_like(self.lens)
        table = -np.ones_like(self.table)
        for r, p in enumerate(parents):
            if p < -1 or p >= rows:
                return None
            if p >= 0:
                lens[r] = self.lens[p]
                held = -(-int(lens[r]) // self.ps)
                table[r, :held] = self.table[p, :held]
        refs = self.refs.copy()
        for t, sign in ((self.table, -1), (table, 1)):
            for i in t.reshape(-1):
                if i >= 0:
                    refs[i] += sign
        free = [i for i in range(len(refs)) if refs[i] == 0]
        copies = []
        for r, p in enumerate(parents):
            m = int(reserve[r]) if p >= 0 else 0
            if m <= 0:
                continue
            held, ends = -(-int(lens[r]) // self.ps), -(-(int(lens[r]) + m) // self.ps)
            if ends > width:
                return None
            last = table[r, held - 1] if lens[r] % self.ps else -1
            if last >= 0 and refs[last] > 1:
                if not free:
                    return None
                new = free.pop(0)
                copies.append((int(last), new))
                refs[last] -= 1
                refs[new] = 1
                table[r, held - 1] = new
            for i in range(held, ends):
                if not free:
                    return None
                table[r, i] = free.pop(0)
                refs[table[r, i]] = 1
        self.table, self.lens, self.refs = table, lens, refs
        return copies


def select(logits, scores, ended, eos):
    """One group: [(token, beam, score, ended)] best first; logits [beams, vocab] float64."""
    offers = []
    beams, vocab = logits.shape
    for b in range(beams):
        if ended[b]:
            offers.append((-scores[b], b, 0, eos, scores[b]))
            continue
        x = logits[b]
        m = x.max()
        lse = m + math.log(np.exp(x - m).sum()) if m > -math.inf else 0.0
        order = sorted(range(vocab), key=lambda t: (-x[t], t))[:beams]
        for e, t in enumerate(order):
            s = scores[b] + (x[t] - lse) if x[t] > -math.inf else -math.inf
            offers.append((-s, b, e, t, s))
    offers.sort(key=lambda o: o[:3])
    return [(t, b, s, bool(ended[b]) or t == eos) for _, b, _, t, s in offers[:beams]]
