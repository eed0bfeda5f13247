"""Plain 64-bit implementations that the serving operators are tested against, and the error
bounds derived from the kernels' roundings.

Bounds count, for every value: half a step of the stored type relative to it (bf16 2^-8, fp32
2^-24), the same for each bf16 operand inside (P, in attention), and 2^-24 for each fp32
operation that can round, on the sum of the magnitudes it adds up.
"""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def within(name, got, ref, bound):
    got, ref = np.asarray(got), np.asarray(ref)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN in other places"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]) and not np.isinf(got[~inf]).any(), \
        f"{name}: infinities in other places"
    ok = np.isfinite(ref)
    with np.errstate(invalid="ignore"):
        over = np.abs(got - np.where(ok, ref, 0.0)) - np.broadcast_to(bound, ref.shape)
    worst = float(np.max(np.where(ok, over, -1.0), initial=-1.0))
    assert worst <= 0, f"{name}: {worst:.3e} beyond its bound"


# ---------------------------------------------------------------------------- rotary


def rotate(x, table, pos, interleaved, back=False):
    """x [T, H, d] float64; table [L, half, 2]; returns (result, sum of magnitudes)."""
    half = table.shape[1]
    c, s = table[pos][:, None, :, 0], table[pos][:, None, :, 1]
    s = -s if back else s
    y, mag = x.copy(), np.abs(x)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
    mag[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, mag


def rotary_bound(ref, mag, dtype):
    """Two products and a sum in fp32 (three roundings), then the store."""
    e = 3 * U32 * mag
    return HALF[dtype] * (np.abs(ref) + e) + e


# ----------------------------------------------------------------------------- cache


class CacheModel:
    """The paged cache in plain Python: lists of whole numbers and a 64-bit copy of the rows."""

    def __init__(self, k, v, table, lengths, refs):
        self.k, self.v = f64(k), f64(v)
        self.table, self.lengths, self.refs = table.tolist(), lengths.tolist(), refs.tolist()
        self.ps = k.shape[3]
        self.slots, self.max_pages = len(self.table), len(self.table[0])

    def pages_of(self, n):
        return -(-n // self.ps)

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def _valid(self, slots):
        return all(0 <= s < self.slots for s in slots)

    def reserve(self, slots, counts):
        """Returns the status bits; changes nothing unless they are 0."""
        if not self._valid(slots) or len(set(slots)) < len(slots):
            return 1
        want = 0
        for s, c in zip(slots, counts):
            if c < 0 or self.lengths[s] + c > self.max_pages * self.ps:
                return 2
            if c > 0 and self.lengths[s] % self.ps and \
                    self.refs[self.table[s][self.lengths[s] // self.ps]] != 1:
                return 8
            want += self.pages_of(self.lengths[s] + c) - self.pages_of(self.lengths[s])
        free = self._free()
        if want > len(free):
            return 4
        for s, c in zip(slots, counts):
            for i in range(self.pages_of(self.lengths[s]), self.pages_of(self.lengths[s] + c)):
                self.table[s][i] = free.pop(0)
                self.refs[self.table[s][i]] = 1
            self.lengths[s] += c
        return 0

    def fork(self, parents, children):
        if not self._valid(parents + children) or len(set(children)) < len(children) or \
                set(parents) & set(children):
            return 1
        if any(self.lengths[c] for c in children):
            return 2
        free = self._free()
        if sum(self.lengths[p] % self.ps > 0 for p in parents) > len(free):
            return 4
        for p, c in zip(parents, children):
            n = self.lengths[p]
            for i in range(n // self.ps):
                self.table[c][i] = self.table[p][i]
                self.refs[self.table[p][i]] += 1
            if n % self.ps:
                i, new = n // self.ps, free.pop(0)
                for x in (self.k, self.v):
                    x[:, new, :, :n % self.ps] = x[:, self.table[p][i], :, :n % self.ps]
                self.table[c][i] = new
                self.refs[new] = 1
            self.lengths[c] = n
        return 0

    def free(self, slots):
        if not self._valid(slots):
            return 1
        for s in slots:
            self._drop(s, 0)
        return 0

    def _drop(self, s, n):
        for i in range(self.pages_of(n), self.pages_of(self.lengths[s])):
            self.refs[self.table[s][i]] -= 1
            self.table[s][i] = -1
        self.lengths[s] = n

    def accept(self, slots, base, path, accepted):
        if not self._valid(slots) or len(set(slots)) < len(slots):
            return 1
        for s, b, p, m in zip(slots, base, path, accepted):
            n = self.lengths[s]
            if b < 0 or b > n or m < 0 or m > len(p) or m > n - b:
                return 2
            if any(t < 0 or t >= n - b for t in p[:m]) or any(x >= y for x, y in zip(p[:m], p[1:m])):
                return 2
            for i in range(b // self.ps, self.pages_of(b + m)):
                if i < self.pages_of(n) and self.refs[self.table[s][i]] != 1:
                    return 8
        for s, b, p, m in zip(slots, base, path, accepted):
            for j in range(m):
                for x in (self.k, self.v):
                    x[:, self.table[s][(b + j) // self.ps], :, (b + j) % self.ps] = \
                        x[:, self.table[s][(b + p[j]) // self.ps], :, (b + p[j]) % self.ps]
            self._drop(s, b + m)
        return 0

    def place(self, slot, pos):
        return self.table[slot][pos // self.ps], pos % self.ps

    def rows(self, which, layer, slot):
        """[length, heads, d] of a slot."""
        x = self.k if which == "k" else self.v
        return np.stack([x[layer, p, :, r] for p, r in
                         (self.place(slot, t) for t in range(self.lengths[slot]))]) \
            if self.lengths[slot] else np.zeros((0,) + (x.shape[2], x.shape[4]))


# ------------------------------------------------------------------------- attention


def attend(q, k, v, visible, scale):
    """One sequence: q [n, Hq, d], k and v [L, Hkv, d], visible [n, L] bool, all 64 bits.
    Returns o, lse [Hq, n], and their bounds.  A row that sees nothing gives 0 and -inf."""
    n, Hq, d = q.shape
    Hkv = k.shape[1]
    o, bo = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse, bl = np.full((Hq, n), -np.inf), np.zeros((Hq, n))
    for h in range(Hq):
        g = h // (Hq // Hkv)
        for t in range(n):
            at = np.flatnonzero(visible[t])
            if at.size == 0:
                continue
            kk, vv = k[at, g], v[at, g]
            s = scale * (kk @ q[t, h])
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            lse[h, t] = m + np.log(l)
            with np.errstate(invalid="ignore"):
                o[t, h] = (p @ vv) / l
                mag = (p @ np.abs(vv)) / l
            # a score sums d products in fp32 (each addition may lose a step of the largest
            # partial sum); the exponential has two ulps; P enters in bf16; the sums run over
            # the keys in fp32
            ds = scale * 2 * d * U32 * float((np.abs(kk) @ np.abs(q[t, h])).max()) + 4 * U32 * abs(m)
            rel = 2 * ds + 8 * U32 + 2 * at.size * U32
            mag = np.where(np.isfinite(mag), mag, 0.0)
            bo[t, h] = HALF[torch.bfloat16] * np.abs(np.where(np.isfinite(o[t, h]), o[t, h], 0)) * 1.01 + \
                (HALF[torch.bfloat16] * (1 + rel) + rel) * mag
            bl[h, t] = rel + 4 * U32 * (1 + abs(lse[h, t]))
    return o, lse, bo, bl
