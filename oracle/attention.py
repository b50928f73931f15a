"""fp64 reference of the full-attention layers' operators: softmax attention of
packed prompts and of windows over a paged cache, rotary positions, and the
page tables as plain Python lists. Test infrastructure; shares no code with the
CUDA path.
"""
import numpy as np


def attend(q, k, v, seen, scale):
    """One head. q [n, D], k, v [m, D], seen[i]: keys query i sees (its first
    seen[i]). Returns o, lse and the mass sum_j p_ij |v_j| (what rounding errors
    of the weights scale with). Keys that a query does not see are not touched."""
    o = np.zeros((q.shape[0], v.shape[1]))
    mass = np.zeros_like(o)
    lse = np.full(q.shape[0], -np.inf)
    with np.errstate(all="ignore"):
        for i, n in enumerate(seen):
            if n > 0:
                s = scale * (k[:n] @ q[i])
                top = s.max()
                p = np.exp(s - top)
                lse[i] = top + np.log(p.sum())
                p /= p.sum()
                o[i] = p @ v[:n]
                mass[i] = p @ np.abs(v[:n])
    return o, lse, mass


def prompt(q, k, v, cu, cu_k, scale, live=None):
    """Packed causal prompts: q [N, HQ, D], k, v [M, HKV, D]."""
    N, HQ, _ = q.shape
    G = HQ // k.shape[1]
    o, mass = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.zeros((N, HQ))
    for r in range(len(cu) - 1):
        if live is not None and not live[r]:
            continue
        a, b, c, d = cu[r], cu[r + 1], cu_k[r], cu_k[r + 1]
        seen = np.clip((d - c) - (b - a) + 1 + np.arange(b - a), 0, None)
        for h in range(HQ):
            o[a:b, h], lse[a:b, h], mass[a:b, h] = attend(
                q[a:b, h], k[c:d, h // G], v[c:d, h // G], seen, scale)
    return o, lse, mass


def window(q, tokens, lengths, T, scale):
    """Windows over cached tokens: tokens[r] = (k, v) [length + T, HKV, D] of row
    r or None; q [B T, HQ, D]."""
    o, mass = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.zeros(q.shape[:2])
    for r, kv in enumerate(tokens):
        if kv is None:
            continue
        G = q.shape[1] // kv[0].shape[1]
        at = slice(r * T, r * T + T)
        for h in range(q.shape[1]):
            o[at, h], lse[at, h], mass[at, h] = attend(
                q[at, h], kv[0][:, h // G], kv[1][:, h // G], lengths[r] + 1 + np.arange(T), scale)
    return o, lse, mass


def rotate(x, pos, freq, axis):
    """x [N, H, D]; pos [axes, N]; pair i (dimensions i, i + P) turns by
    pos[axis[i]] * freq[i]."""
    P = len(freq)
    turn = np.exp(1j * pos[axis].T * freq)[:, None]
    y = x.astype(np.float64).copy()
    z = (x[..., :P] + 1j * x[..., P:2 * P]) * turn
    y[..., :P], y[..., P:2 * P] = z.real, z.imag
    return y


def pair_axes(pairs, sections, interleaved):
    if not interleaved:
        return np.repeat(np.arange(len(sections)), sections)
    n = len(sections)
    return np.array([i % n if i < n * sections[i % n] else 0 for i in range(pairs)])


class Pages:
    """Page tables: lists of page ids per slot and the number of holders of each
    page; the lowest free page goes first. `data` holds one value per page."""

    def __init__(self, n_slots, n_pages, page, max_pages):
        self.page, self.max_pages = page, max_pages
        self.table = [[] for _ in range(n_slots)]
        self.length = [0] * n_slots
        self.refs = [0] * n_pages
        self.data = list(range(n_pages))
        self.failed = False

    def _free(self):
        return [i for i, n in enumerate(self.refs) if n == 0]

    def reserve(self, slots, tokens):
        short = False
        for s, n in zip(slots, tokens):
            if s < 0:
                continue
            need = -(-(self.length[s] + n) // self.page) - len(self.table[s])
            if need <= 0:
                continue
            if len(self.table[s]) + need > self.max_pages:
                self.failed = True
                continue
            free = self._free()
            if short or len(free) < need:
                short = self.failed = True
                continue
            for p in free[:need]:
                self.refs[p] = 1
                self.table[s].append(p)

    def release(self, slots):
        for s in slots:
            if s >= 0:
                for p in self.table[s]:
                    self.refs[p] -= 1
                self.table[s], self.length[s] = [], 0

    def fork(self, src, dst, deep=False):
        rows = [(s, d) for s, d in zip(src, dst) if s >= 0 and d >= 0]
        self.release([d for _, d in rows])
        whole = {}
        for s, d in rows:
            whole[d] = 0 if deep else self.length[s] // self.page
            for p in self.table[s][:whole[d]]:
                self.refs[p] += 1
        free, at, short = self._free(), 0, False
        for s, d in rows:
            n, pages = whole[d], -(-self.length[s] // self.page)
            need = pages - n
            if need > 0 and (short or at + need > len(free)):
                short = self.failed = True
                for p in self.table[s][:n]:
                    self.refs[p] -= 1
                continue
            new = free[at:at + need]
            at += need
            for p, old in zip(new, self.table[s][n:pages]):
                self.refs[p] = 1
                self.data[p] = self.data[old]
            self.table[d] = self.table[s][:n] + new
            self.length[d] = self.length[s]

    def compact(self):
        used = sum(n > 0 for n in self.refs)
        holes = [i for i in range(used) if self.refs[i] == 0]
        movers = [i for i in range(used, len(self.refs)) if self.refs[i] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.data[b] = self.data[a]
        self.table = [[to.get(p, p) for p in row] for row in self.table]
