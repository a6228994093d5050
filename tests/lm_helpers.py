"""Plain 64-bit restatements of the cache, its attention and the log probabilities, and the inputs the
tests give them.  Everything is numpy on the host; nothing here shares code with the library."""
import numpy as np

BLOCK = 16


class Case:
    """A cache with its sequences: lens and news per sequence, pages dealt out in a shuffled order."""

    def __init__(self, seed, lens, news, kv_heads, dim, page, spare=2, v_spread=False):
        r = self.rng = np.random.default_rng(seed)
        self.lens, self.news = list(lens), list(news)
        self.H, self.D, self.P = kv_heads, dim, page
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = r.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.T = sum(news)
        self.q_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        shape = (self.pages, kv_heads, page, dim)
        self.codes = [r.integers(1, 256, shape, dtype=np.uint8) for _ in range(2)]
        self.scales = [r.uniform(0.004, 0.03, (self.pages, kv_heads, page // BLOCK)).astype(np.float32)
                       for _ in range(2)]
        if v_spread:  # value scales over many orders of magnitude
            self.scales[1] *= np.float32(10) ** r.uniform(-6, 2, self.scales[1].shape).astype(np.float32)

    def value(self, which, s, j):
        """[H, D] of position j of sequence s, or None where its page does not exist."""
        p = int(self.table[s, j // self.P])
        if not 0 <= p < self.pages:
            return None
        c = self.codes[which][p, :, j % self.P].astype(np.float64) - 128
        return c * self.scales[which][p, :, j % self.P // BLOCK].astype(np.float64)[:, None]

    def upload(self, torch, mnb, max_new=None, max_len=None):
        dev = [torch.from_numpy(x).cuda() for x in (*self.codes, *self.scales)]
        self.cache = mnb.KVCache(*dev)
        cu = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
        self.batch = mnb.KVBatch(cu(self.table), cu(self.lens), cu(self.q_start), self.T,
                                 max(self.news) if max_new is None else max_new,
                                 max(self.lens) if max_len is None else max_len)
        return self.cache, self.batch


def write_ref(c, k, v):
    """The write in its own arithmetic, binary32 step by step: (codes, scales) for keys and values."""
    f = np.float32
    codes, scales = [x.copy() for x in c.codes], [x.copy() for x in c.scales]
    with np.errstate(all="ignore"):
        for which, x in ((0, k), (1, v)):
            x = x.astype(f)
            for s, (n, length) in enumerate(zip(c.news, c.lens)):
                first = length - n
                for b in range(max(first, 0) // BLOCK, -(-length // BLOCK)) if n else ():
                    p = int(c.table[s, b * BLOCK // c.P])
                    if not 0 <= p < c.pages:
                        continue
                    row, blk = b * BLOCK % c.P, b * BLOCK % c.P // BLOCK
                    pos = np.arange(b * BLOCK, b * BLOCK + BLOCK)
                    new, old = (pos >= first) & (pos < length), pos < first
                    for h in range(c.H):
                        tok = x[c.q_start[s] + pos[new] - first, h]
                        s_new = np.max(np.abs(tok)) / f(127)
                        s_old = scales[which][p, h, blk]
                        sc = np.maximum(s_old, s_new) if old.any() else s_new
                        good = sc > 0 and sc < np.inf
                        q = codes[which][p, h, row:row + BLOCK]
                        if good:
                            inv = f(1) / sc
                            code = lambda y, m: np.clip(np.rint(y * m), -127, 127).astype(np.int64) + 128  # noqa: E731
                            if s_old != sc:
                                q[old] = code(q[old].astype(f) - f(128), s_old / sc)
                            q[new] = code(tok, inv)
                        else:
                            q[old | new] = 128
                        scales[which][p, h, blk] = sc
    return codes, scales


def attn_ref(c, q, scale, window=0):
    """(out, lse, tolerance) in 64 bits.  The tolerance, a key p_j = e^(s_j - m) / sum at a time: its FP16 rounding
    (2^-11 of it, or 2^-25 of the largest where it is subnormal), the binary32 dot product's roundings in the
    exponent (numerator and denominator), and the output's FP16 rounding."""
    T, Hq, D = q.shape
    G = Hq // c.H
    out, lse, tol = np.zeros(q.shape), np.full((T, Hq), -np.inf), np.full(q.shape, 2.0 ** -25)
    for s, (n, length) in enumerate(zip(c.news, c.lens)):
        if not n:
            continue
        kv = [[c.value(w, s, j) for j in range(length)] for w in (0, 1)]
        there = np.array([x is not None for x in kv[0]], bool)
        k, v = (np.array([x if x is not None else np.zeros((c.H, D)) for x in y]).reshape(length, c.H, D) for y in kv)
        for i in range(n):
            pos = length - n + i
            j = np.arange(length)
            sees = there & (j <= pos)
            if window:
                sees &= j > pos - window
            if not sees.any():
                continue
            t = c.q_start[s] + i
            for h in range(Hq):
                kh, vh, qh = k[sees, h // G], v[sees, h // G], q[t, h].astype(np.float64)
                x = kh @ qh * scale
                m = x.max()
                e = np.exp(x - m)
                den = e.sum()
                out[t, h] = e @ vh / den
                lse[t, h] = m + np.log(den)
                ds = 2.0 ** -24 * (D + 8) * (np.abs(kh) @ np.abs(qh) * scale).max() + 2.0 ** -21
                spread = e @ np.abs(vh) / den
                tol[t, h] += (2.0 ** -11 + 2 * ds) * spread + 2.0 ** -11 * np.abs(out[t, h]) \
                    + 2.0 ** -25 * len(x) * np.abs(vh).max()
    return out, lse, tol


def past_the_table(c, over):
    """Lengths of `over[s]` positions past the last page of the table, which gets no spare column.  Returns the
    table that a call is given; c keeps one with columns of missing pages for the references: a position past
    the table is one whose page does not exist."""
    full = c.table[:, :-1].copy()
    cap = full.shape[1] * c.P
    c.lens = [cap + o for o in over]
    more = -(-max(max(over), 0) // c.P)
    c.table = np.concatenate([full, np.full((len(c.lens), more + 1), -1, np.int32)], 1)
    return full


def attn_ref_rows(c, q, scale, window=0):
    """attn_ref for many rows: the same definition and tolerance, a sequence and head at a time."""
    T, Hq, D = q.shape
    G = Hq // c.H
    out, lse, tol = np.zeros(q.shape), np.full((T, Hq), -np.inf), np.full(q.shape, 2.0 ** -25)
    for s, (n, length) in enumerate(zip(c.news, c.lens)):
        if not n or length <= 0:
            continue
        j = np.arange(length)
        page = c.table[s, j // c.P].astype(np.int64)
        there = (page >= 0) & (page < c.pages)
        page = np.where(there, page, 0)
        pos = length - n + np.arange(n)
        sees = there & (j <= pos[:, None])
        if window:
            sees &= j > pos[:, None] - window
        rows = slice(c.q_start[s], c.q_start[s] + n)
        for h in range(Hq):
            k, v = ((c.codes[w][page, h // G, j % c.P].astype(np.float64) - 128)
                    * c.scales[w][page, h // G, j % c.P // BLOCK].astype(np.float64)[:, None] for w in (0, 1))
            k, v = np.where(there[:, None], k, 0), np.where(there[:, None], v, 0)
            qh = q[rows, h].astype(np.float64)
            x = np.where(sees, qh @ k.T * scale, -np.inf)
            some = sees.any(1)
            m = np.where(some, x.max(1), 0.0)
            e = np.exp(x - m[:, None])
            den = np.where(some, e.sum(1), 1.0)
            o = e @ v / den[:, None]
            with np.errstate(divide="ignore"):
                lse[rows, h] = np.where(some, m + np.log(den), -np.inf)
            out[rows, h] = o
            ds = 2.0 ** -24 * (D + 8) * np.where(sees, np.abs(qh) @ np.abs(k).T * abs(scale), 0).max(1) + 2.0 ** -21
            spread = e @ np.abs(v) / den[:, None]
            far = np.array([np.abs(v[row]).max() if row.any() else 0.0 for row in sees])
            add = (2.0 ** -11 + 2 * ds)[:, None] * spread + 2.0 ** -11 * np.abs(o) \
                + (2.0 ** -25 * sees.sum(1) * far)[:, None]
            tol[rows, h] += np.where(some[:, None], add, 0)
    return out, lse, tol
