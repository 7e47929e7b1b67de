"""References and tolerances of the serving tests: softmax attention from its definition in 64 bits, and the paged cache's
steps as plain Python over lists."""
import numpy as np
import torch

U32 = 2.0 ** -24      # half a step of fp32, relative
UBF = 2.0 ** -8       # half a step of bf16, relative


def attend(q, k, v, seen, scale):
    """q [t, hq, d], k, v [n, hk, d], seen [t, n]: outputs and log normalisers in 64 bits, with what the tolerances need:
    sum_j p_j |v_j| and the largest sum of |q_i k_i| scale. Rows of k and v that nothing sees take no part."""
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    t, hq, d = q.shape
    hk, n = k.shape[1], k.shape[0]
    g = hq // hk
    q, k, v, seen = q.to(dev).double(), k.to(dev).double(), v.to(dev).double(), seen.to(dev)
    used = seen.any(0)[:, None, None]
    k, v = torch.where(used, k, torch.zeros_like(k)), torch.where(used, v, torch.zeros_like(v))
    q, k, v = q.view(t, hk, g, d).permute(1, 2, 0, 3), k.permute(1, 2, 0)[:, None], v.transpose(0, 1)[:, None]
    s = (q @ k * scale).masked_fill(~seen, -float("inf"))
    big = (q.abs() @ k.abs() * scale).masked_fill(~seen, 0.0).amax(-1)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None]).masked_fill(~seen, 0.0)
    o, mag = p @ v, p @ v.abs()
    back = lambda x: x.permute(2, 0, 1, 3).reshape(t, hq, d).cpu()  # noqa: E731
    return back(o), lse.reshape(hq, t).cpu(), back(mag), big.reshape(hq, t).cpu()


def tolerances(o, lse, mag, big, n, d, *, p_bits=None, out_bf16):
    """Largest differences that roundings explain. Scores: d fp32 multiply-adds, the scale and the difference to the
    maximum (d + 4 roundings, relative to the sum of |q k|); the exponential 4 roundings more; sums over n keys at most
    n roundings each; the quotient 4. p_bits: the softmax weights are rounded once to a type of that half step before the
    product with V. The output is rounded once to its type."""
    delta = (d + 4) * U32 * big + 4 * U32
    rel = (2 * delta + (2 * n + 8) * U32).T[:, :, None]      # numerator and normaliser
    if p_bits is not None:
        rel = rel + p_bits
    tol_o = rel * mag + (UBF if out_bf16 else U32) * o.abs() * (1 + rel) + 1e-30
    # (maximum + log2 of the sum) ln 2: three roundings of numbers no larger than the maximum and the result
    tol_l = delta + (n + 8) * U32 + 4 * U32 * (lse.abs() + big)
    return tol_o, tol_l


def check(got, lse_got, want, tol, what=""):
    o, lse = want
    tol_o, tol_l = tol
    bad = ~((got.double().cpu() - o).abs() <= tol_o)
    assert not bad.any(), f"{what}: {int(bad.sum())} outputs off, worst {float(((got.double().cpu() - o).abs() / tol_o).max()):.3g} of the tolerance"
    if lse_got is not None:
        lg = lse_got.double().cpu()
        empty = torch.isinf(lse)
        assert torch.equal(torch.isinf(lg) & (lg < 0), empty), f"{what}: empty rows"
        off = (lg - lse).abs()[~empty] > tol_l[~empty]
        assert not off.any(), f"{what}: {int(off.sum())} log normalisers off"


class ListCache:
    """The cache's steps with Python lists and numpy rows: k, v [layers, pages, kv_heads, page, d] arrays."""

    def __init__(self, k, v, slots, max_pages):
        self.k, self.v = k, v
        self.page = k.shape[3]
        self.rows = [[] for _ in range(slots)]
        self.lens = [0] * slots
        self.refs = [0] * k.shape[1]
        self.max_pages = max_pages

    def free(self, slots):
        for s in slots:
            for p in self.rows[s]:
                self.refs[p] -= 1
            self.rows[s], self.lens[s] = [], 0

    def fork(self, src, dst):
        for s, t in zip(src, dst):
            n = -(-self.lens[s] // self.page)
            self.rows[t], self.lens[t] = list(self.rows[s][:n]), self.lens[s]
            for p in self.rows[t]:
                self.refs[p] += 1

    def reserve(self, slots, add):
        granted, out = [], False
        for s, a in zip(slots, add):
            rest = self.lens[s] % self.page
            at = self.lens[s] // self.page
            shared = rest and a and self.refs[self.rows[s][at]] > 1
            new = max(0, -(-(self.lens[s] + a) // self.page) - len(self.rows[s]))
            out = out or new + bool(shared) > self.refs.count(0)
            if out:
                granted.append(0)
                continue
            if shared:
                old, p = self.rows[s][at], self.refs.index(0)
                self.refs[p] = 1
                self.refs[old] -= 1
                self.rows[s][at] = p
                for x in (self.k, self.v):
                    x[:, p, :, :rest] = x[:, old, :, :rest]
            for _ in range(new):
                p = self.refs.index(0)
                self.refs[p] = 1
                self.rows[s].append(p)
            granted.append(a)
        return granted

    def append(self, slots, offsets, k, v, layer=0):
        for i, s in enumerate(slots):
            for j, t in enumerate(range(offsets[i], offsets[i + 1])):
                at = self.lens[s] + j
                p = self.rows[s][at // self.page]
                for x, new in ((self.k, k), (self.v, v)):
                    x[layer:layer + new.shape[0], p, :, at % self.page] = new[:, t]

    def commit(self, slots, counts, keep=None):
        for i, s in enumerate(slots):
            kept = list(range(counts[i])) if keep is None else list(keep[i][:counts[i]])
            for x in (self.k, self.v):
                rows = [x[:, self.rows[s][(self.lens[s] + r) // self.page], :, (self.lens[s] + r) % self.page].copy() for r in kept]
                for j, row in enumerate(rows):
                    at = self.lens[s] + j
                    x[:, self.rows[s][at // self.page], :, at % self.page] = row
            self.lens[s] += counts[i]
            n = -(-self.lens[s] // self.page)
            for p in self.rows[s][n:]:
                self.refs[p] -= 1
            self.rows[s] = self.rows[s][:n]

    def state(self):
        table = np.full((len(self.rows), self.max_pages), -1, np.int32)
        for i, r in enumerate(self.rows):
            table[i, :len(r)] = r
        return (table, np.array(self.lens, np.int32), np.array([len(r) for r in self.rows], np.int32),
                np.array(self.refs, np.int32))
