"""Plain 64-bit restatements of the rotation with its norms, of the mixture-of-experts layer and of sampling, and the
inputs the tests give them.  numpy on the host; nothing here shares code with the library."""
import numpy as np


# ------------------------------------------------------------------ rotation

def rope_ref(x, pos, freq, interleaved=False, gain=None, eps=1e-6):
    """(out, tolerance) of x [T, H, D] at integer positions [T].

    Tolerance: one rounding to FP16 (2^-11 of the value, 2^-25 where it is subnormal), and in binary32 of a
    pair's sizes: the mean square (13 roundings, halved by the root), the root (2^-22), three products and a sum, cosine
    and sine (2^-23 each) of an angle to 2^-25 turns (2^-22.3): under 32 steps of 2^-24, twice that allowed."""
    v = x.astype(np.float64)
    if gain is not None:
        v = v / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps) * gain.astype(np.float64)
    half = len(freq)
    first = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    second = first + 1 if interleaved else first + half
    # position times frequency: the product's 55 places as an integer times the frequency's step, modulo the turn
    angle = np.empty((len(pos), half))
    for i, f in enumerate(freq):
        m, e = np.frexp(np.float64(f))
        whole = np.array([int(p) * int(m * 2 ** 24) for p in pos], dtype=object)  # exact
        angle[:, i] = [_turned(int(w), int(e) - 24) for w in whole]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = v[..., first], v[..., second]
    out = v.copy()
    size = np.abs(v)
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = np.abs(a) + np.abs(b)
    return out, 2.0 ** -11 * np.abs(out) + 2.0 ** -25 + 2.0 ** -18 * size


def _turned(whole, exponent):
    """whole * 2^exponent modulo 2 pi, with 200 bits of pi."""
    from fractions import Fraction
    two_pi = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    x = Fraction(whole) * Fraction(2) ** exponent
    return float(x - (x // two_pi) * two_pi)


# ------------------------------------------------------------------ mixture of experts

class Experts:
    def __init__(self, seed, hidden, inter, experts, bits, zp, size=1.0):
        r = self.rng = np.random.default_rng(seed)
        self.hidden, self.inter, self.experts, self.bits = hidden, inter, experts, bits

        def weight(rows, cols):
            codes = r.integers(0, 1 << bits, (experts, rows, cols), dtype=np.uint8)
            spread = (1 << bits) / 12 ** 0.5 * cols ** 0.5
            scales = (r.uniform(0.7, 1.3, (experts, rows, cols // 32)) / spread).astype(np.float16)
            mid = 1 << (bits - 1)
            z = r.integers(0, 2 * mid, (experts, rows, cols // 32)).astype(np.uint8) if zp == "any" else \
                r.integers(mid - 1, mid + 2, (experts, rows, cols // 32)).astype(np.uint8) if zp else None
            return codes, scales, z

        self.router = (r.standard_normal((experts, hidden)) * 1.5 / hidden ** 0.5 / size).astype(np.float16)
        self.up, self.down = weight(2 * inter, hidden), weight(hidden, inter)

    def dense(self, which, e):
        codes, scales, z = getattr(self, which)
        z = float(1 << (self.bits - 1)) if z is None else np.repeat(z[e].astype(np.float64), 32, 1)
        return (codes[e].astype(np.float64) - z) * np.repeat(scales[e].astype(np.float64), 32, 1)

    def layer(self, torch, mnb, top_k, normalize):
        def codes(c):
            E, rows, cols = c.shape
            if self.bits == 4:
                c = c[..., ::2] | c[..., 1::2] << 4
            return torch.from_numpy(np.ascontiguousarray(c).reshape(E, rows, cols // 32, 4 * self.bits)).cuda()

        up = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        (uc, us, uz), (dc, ds, dz) = self.up, self.down
        return mnb.MoE(up(self.router), codes(uc), up(us), codes(dc), up(ds), top_k=top_k, bits=self.bits, up_zp=up(uz),
                       down_zp=up(dz), normalize=normalize)

    def ref(self, x, top_k, normalize):
        """(ids, weights, y, tolerance).

        Tolerance.  Gate and up: products of FP16 inputs and exact codes summed in binary32, 2^-24 of the terms' sizes a
        sum of which a step of 16 products makes one (the tensor core keeps at least 23 bits), so (hidden / 16 + 8) of
        them; silu's slope is at most 1.1 and its value 2^-21 off.  FP16 of the block's products: 2^-11 of
        each, 2^-25 of twice the block's largest where that is more.  Down alike, weights 2^-21, one FP16 rounding."""
        M = len(x)
        xd = x.astype(np.float64)
        logits = xd @ self.router.astype(np.float64).T
        ids = np.stack([np.lexsort((np.arange(self.experts), -l))[:top_k] for l in logits])
        weights = np.empty((M, top_k))
        y, tol = np.zeros((M, self.hidden)), np.full((M, self.hidden), 2.0 ** -25)
        step = lambda n: (n / 16 + 8) * 2.0 ** -24  # noqa: E731
        dense = {}
        for t in range(M):
            best = logits[t, ids[t]]
            over = best if normalize else logits[t]
            weights[t] = np.exp(best - best[0]) / np.exp(over - best[0]).sum()
            for e, w in zip(ids[t], weights[t]):
                if e not in dense:
                    dense[e] = self.dense("up", e), self.dense("down", e)
                W, D = dense[e]
                g, u = np.split(W @ xd[t], 2)
                dg, du = np.split(np.abs(W) @ np.abs(xd[t]) * step(self.hidden), 2)
                silu = g / (1 + np.exp(-g))
                h = silu * u
                dh = (1.1 * dg + 2.0 ** -21 * np.abs(silu)) * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du
                block = np.repeat(np.abs(h).reshape(-1, 32).max(1), 32)
                dh += np.maximum(2.0 ** -11 * np.abs(h), 2.0 ** -24 * block)
                y[t] += w * (D @ h)
                tol[t] += w * (np.abs(D) @ dh + (step(self.inter) + 2.0 ** -20) * (np.abs(D) @ np.abs(h)))
        return ids, weights, y, tol + 2.0 ** -11 * np.abs(y)


# ------------------------------------------------------------------ sampling

def sample_ref(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log probability) of one row of FP16 logits."""
    x = row.astype(np.float64) + 0.0
    if np.isnan(x).any() or (x == np.inf).any():
        return -1, np.nan
    if (x == -np.inf).all():
        return -1, -np.inf
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    v = x[order]
    if not temperature > 0:
        temperature, top_k = 1.0, 1
    w = np.exp(np.maximum((v - v[0]) / np.float64(temperature), -745.0)) if temperature < np.inf else np.ones(len(v))
    n = len(v) if top_k <= 0 else min(int(top_k), len(v))
    cum = np.cumsum(w)
    if top_p < 1:
        n = min(n, int((cum[:n] < max(float(top_p), 0.0) * cum[n - 1]).sum()) + 1)
    if min_p > 0:
        n = min(n, max(int((w >= float(min_p)).sum()), 1))
    u = float(u) if u > 0 else 0.0
    at = min(int((cum[:n] <= u * cum[n - 1]).sum()), n - 1)
    return int(order[at]), float(np.log(w[at] / cum[n - 1]))
