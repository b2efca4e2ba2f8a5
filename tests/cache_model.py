"""A plain model of the paged cache, for the tests: Python lists for the pages, fp64 numpy for the blocks.

Written from the interface's description (include/entmax_cache.h), one sequence after another, with no
code of the package."""
import numpy as np

PAGE = 64


def e4m3_value(byte):
    """The number an e4m3 byte stands for: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    s, e, m = byte >> 7, (byte >> 3) & 15, byte & 7
    if e == 15 and m == 7:
        return float("nan")
    v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -v if s else v


VALUES = np.array([e4m3_value(b) for b in range(256)])


def to_e4m3(x):
    """fp64 values within +-448 rounded to e4m3 values, ties to the even mantissa."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(x / step) * step  # rint: ties to even; NaN stays NaN


def block_exp(x):
    """Exponent of the smallest power of two s >= 2^-100 with max|x| / s <= 448 over the finite x."""
    a = np.abs(x[np.isfinite(x)])
    e = -100
    if a.size and a.max() > 0:
        e = max(e, int(np.ceil(np.log2(a.max() / 448.0))))
        while e > -100 and a.max() <= 448.0 * 2.0 ** (e - 1):
            e -= 1
        while a.max() > 448.0 * 2.0 ** e:
            e += 1
    return e


class Model:
    def __init__(self, n_layers, n_pages, H_kv, n_seqs, max_pages):
        shape = (n_layers, n_pages, H_kv)
        self.num = [np.zeros(shape + (PAGE, 64)) for _ in "KV"]   # e4m3 values
        self.scale = [np.zeros(shape) for _ in "KV"]
        self.refs = [0] * n_pages
        self.table = [[-1] * max_pages for _ in range(n_seqs)]
        self.lens = [0] * n_seqs

    def _pages(self, n):
        return (n + PAGE - 1) // PAGE

    def resize(self, seqs, new_lens):
        """Returns the number of missing pages."""
        grow = []
        for i, (s, n) in enumerate(zip(seqs, new_lens)):
            old = self.lens[s]
            if n <= old:
                for k in range(self._pages(n), self._pages(old)):
                    self.refs[self.table[s][k]] -= 1
                    self.table[s][k] = -1
                self.lens[s] = n
            else:
                grow.append((s, n))
        partial = {s: self.table[s][self._pages(self.lens[s]) - 1] for s, _ in grow if self.lens[s] % PAGE}
        holders = {}
        for s, p in partial.items():
            if self.refs[p] > 1:
                holders.setdefault(p, []).append(s)
        copies = []
        for s, n in grow:
            p = partial.get(s)
            if p in holders and not (len(holders[p]) == self.refs[p] and holders[p][-1] == s):
                copies.append(s)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        need = sum((s in copies) + self._pages(n) - self._pages(self.lens[s]) for s, n in grow)
        if need > len(free):
            return need - len(free)
        for s, n in grow:
            have = self._pages(self.lens[s])
            if s in copies:
                p, q = partial[s], free.pop(0)
                for x in (*self.num, *self.scale):
                    x[:, q] = x[:, p]
                self.refs[p] -= 1
                self.refs[q] = 1
                self.table[s][have - 1] = q
            for k in range(have, self._pages(n)):
                q = free.pop(0)
                self.refs[q] = 1
                self.table[s][k] = q
            self.lens[s] = n
        return 0

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            self.table[d] = list(self.table[s])
            self.lens[d] = self.lens[s]
            for p in self.table[s]:
                if p >= 0:
                    self.refs[p] += 1

    def compact(self):
        used = [p for p, r in enumerate(self.refs) if r > 0]
        U = len(used)
        to = dict(zip([p for p in used if p >= U], [p for p in range(U) if self.refs[p] == 0]))
        for p, q in to.items():
            for x in (*self.num, *self.scale):
                x[:, q] = x[:, p]
            self.refs[q], self.refs[p] = self.refs[p], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return U

    def append(self, layer, K, V, seqs, cu):
        """K, V: fp64 [T, H_kv, 64]."""
        for num, scale, x in ((self.num[0], self.scale[0], K), (self.num[1], self.scale[1], V)):
            for i, s in enumerate(seqs):
                end = self.lens[s]
                start = end - (cu[i + 1] - cu[i])
                for k in range(start // PAGE, self._pages(end)):
                    p = self.table[s][k]
                    a, b = max(start, k * PAGE), min(end, (k + 1) * PAGE)
                    if a >= b:
                        continue
                    kept = a - k * PAGE
                    for h in range(x.shape[1]):
                        new = x[cu[i] + a - start:cu[i] + b - start, h]
                        f = 2.0 ** block_exp(new)
                        if kept:
                            f = max(f, scale[layer, p, h])
                            num[layer, p, h, :kept] = to_e4m3(num[layer, p, h, :kept] * (scale[layer, p, h] / f))
                        num[layer, p, h, kept:kept + b - a] = to_e4m3(np.where(np.isfinite(new), new, np.nan) / f)
                        scale[layer, p, h] = f

    def tokens(self, layer, s):
        """(K, V) of a sequence's tokens, fp64 [len, H_kv, 64]."""
        n = self.lens[s]
        out = []
        for num, scale in zip(self.num, self.scale):
            p = self.table[s][:self._pages(n)]
            x = num[layer, p] * scale[layer, p][..., None, None]      # [pages, H_kv, 64, 64]
            out.append(x.transpose(0, 2, 1, 3).reshape(-1, x.shape[1], 64)[:n])
        return out
