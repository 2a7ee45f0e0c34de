"""The 4-bit cache in plain numpy, 64 bits: format, attention and page bookkeeping.

Written from the definitions in include/wd_kv.h, one loop at a time, and sharing no code with the
library.  A cache here is a uint8 array [pages, layers, kv heads, page size / 16, group].
"""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise(x):
    """x float64 [..., D] -> codes uint8 [..., D], scale bytes uint8 [..., D / 32]."""
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    finite = np.isfinite(b).all(-1)
    a = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0)).max(-1), 1.0)
    e = np.zeros(a.shape, int)
    e[a > 0] = np.clip(np.floor(np.log2(a[a > 0])).astype(int) - 2, -127, 127)
    y = np.abs(np.where(np.isfinite(b), b, 0)) / np.exp2(e.astype(np.float64))[..., None]
    far = np.abs(y[..., None] - E2M1)
    near = far.min(-1, keepdims=True)
    tie = (far == near)
    # of two values at the same distance the one with the even code
    code = np.where(tie.sum(-1) > 1, np.argmax(tie & (np.arange(8) % 2 == 0), -1), far.argmin(-1))
    code = code + 8 * np.signbit(b)
    code = np.where(finite[..., None], code, 0).astype(np.uint8).reshape(x.shape)
    return code, np.where(finite, e + 127, 255).astype(np.uint8)


def values(code, scale):
    v = E2M1[code & 7] * np.where(code >= 8, -1.0, 1.0)
    unit = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return (v.reshape(*v.shape[:-1], -1, 32) * unit[..., None]).reshape(v.shape)


def group_bytes(D):
    return 16 * (D + 2 * (D // 32))


def _places(D):
    """Byte and shift of the K and V code of (token, channel) in a group, [16, D] each."""
    nb = min(4, D // 32)
    t, ch = np.arange(16)[:, None], np.arange(D)[None, :]
    slab, c, lane = ch // (32 * nb), ch % (32 * nb) // 32, ch % 32
    k = slab * 256 * nb + t * 16 * nb + (lane // 8) * 4 * nb + c * 4 + (lane % 8) // 2
    v = (8 * D + slab * 256 * nb + (t // 8) * 128 * nb + (lane // 4) * 16 * nb +
         (t % 8 // 2) * 4 * nb + (t % 2) * 2 * nb + c * 2 + (lane % 4) // 2)
    return k, v, np.broadcast_to(4 * (ch % 2), k.shape)


def decode(group, D):
    """Bytes [..., group] -> K and V as float64 [..., 16, D]."""
    k, v, shift = _places(D)
    at = 16 * D
    ks = group[..., at:at + D // 2].reshape(*group.shape[:-1], 16, D // 32)
    vs = group[..., at + D // 2:at + D].reshape(*group.shape[:-1], 16, D // 32)
    return (values((group[..., k] >> shift) & 15, ks), values((group[..., v] >> shift) & 15, vs))


def store(pool, page, layer, head, t, D, kcode, kscale, vcode, vscale):
    """Write one token of one head, t its place in the page."""
    k, v, shift = _places(D)
    g = pool[page, layer, head, t // 16]
    t %= 16
    for place, code in ((k, kcode), (v, vcode)):
        for ch in range(0, D, 2):
            assert place[t, ch] == place[t, ch + 1]
        g[place[t, ::2]] = code[::2] | (code[1::2] << 4)
    n, at = D // 32, 16 * D
    g[at + t * n:at + (t + 1) * n] = kscale
    g[at + 16 * n + t * n:at + 16 * n + (t + 1) * n] = vscale


def sequence(pool, row, length, layer, head, D, P):
    """K and V of the first `length` tokens of a table row, float64 [length, D]."""
    pages = row[:-(-length // P)]
    k, v = decode(pool[pages, layer, head], D)
    return k.reshape(-1, D)[:length], v.reshape(-1, D)[:length]


def attention(pool, table, lengths, layer, q, seqs, q_start, D, P, scale, window=0):
    """out, lse, and sum_j p_j |v_j| (what the rounding of p is relative to), float64."""
    T, hq, hkv = q.shape[0], q.shape[1], pool.shape[2]
    out, lse, mag = np.zeros((T, hq, D)), np.full((T, hq), -np.inf), np.zeros((T, hq, D))
    for b in range(len(q_start) - 1):
        n, s = q_start[b + 1] - q_start[b], seqs[b]
        L = int(lengths[s])
        if L == 0:
            continue
        for h in range(hkv):
            k, v = sequence(pool, table[s], L, layer, h, D, P)
            for i in range(n):
                p = L - n + i
                lo = max(0, p - window + 1) if window else 0
                if p < 0:
                    continue
                for qh in range(h * hq // hkv, (h + 1) * hq // hkv):
                    x = scale * (k[lo:p + 1] @ q[q_start[b] + i, qh])
                    top = x.max()
                    e = np.exp(x - top)
                    out[q_start[b] + i, qh] = e @ v[lo:p + 1] / e.sum()
                    mag[q_start[b] + i, qh] = e @ np.abs(v[lo:p + 1]) / e.sum()
                    lse[q_start[b] + i, qh] = top + np.log(e.sum())
    return out, lse, mag


class Pages:
    """The page operations, one request after the other, on lists."""

    def __init__(self, pages, slots, P):
        self.P, self.rows, self.lengths = P, [[] for _ in range(slots)], [0] * slots
        self.refs = [0] * pages
        self.data = [None] * pages  # what stands in a page, for the tests

    def _free(self, refs, n):
        return [p for p, r in enumerate(refs) if r == 0][:n]

    def reserve(self, seqs, counts, columns):
        ok, asked, seen = [], 0, set()
        free = [p for p, r in enumerate(self.refs) if r == 0]
        plan = []
        for s, c in zip(seqs, counts):
            good = 0 <= s < len(self.rows) and c >= 0 and s not in seen
            if 0 <= s < len(self.rows):
                seen.add(s)
            if not good or self.lengths[s] + c > columns * self.P:
                ok.append(0)
                continue
            need = -(-(self.lengths[s] + c) // self.P) - len(self.rows[s])
            good = need == 0 or asked + need <= len(free)
            ok.append(int(good))
            if good:
                plan.append((s, c, free[asked:asked + need]))
            asked += need
        for s, c, pages in plan:
            self.rows[s] = self.rows[s] + pages
            self.lengths[s] += c
            for p in pages:
                self.refs[p] = 1
        return ok

    def fork(self, src, dst):
        rows, lengths = [list(r) for r in self.rows], list(self.lengths)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        ok, asked, seen = [], 0, set()
        for s, d in zip(src, dst):
            good = 0 <= d < len(rows) and -1 <= s < len(rows) and d not in seen
            if 0 <= d < len(rows):
                seen.add(d)
            if not good:
                ok.append(0)
                continue
            if s == d:
                ok.append(1)
                continue
            new, length = ([], 0) if s < 0 else (rows[s], lengths[s])
            whole = length // self.P
            page = None
            if length % self.P:
                asked += 1
                if asked > len(free):
                    ok.append(0)
                    continue
                page = free[asked - 1]
            ok.append(1)
            for p in rows[d]:
                self.refs[p] -= 1
            for p in new[:whole]:
                self.refs[p] += 1
            self.rows[d], self.lengths[d] = new[:whole], length
            if page is not None:
                self.rows[d] = self.rows[d] + [page]
                self.refs[page] += 1
                self.data[page] = self.data[new[whole]]
        return ok

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] == 0]
        movers = [p for p in live if p >= n]
        to = {p: p for p in live}
        for m, h in zip(movers, holes):
            to[m] = h
            self.data[h] = self.data[m]
            self.refs[h], self.refs[m] = self.refs[m], 0
        self.rows = [[to[p] for p in r] for r in self.rows]
        return [to.get(p, -1) for p in range(len(self.refs))]

    def table(self, columns):
        t = np.full((len(self.rows), columns), -1, np.int32)
        for s, r in enumerate(self.rows):
            t[s, :len(r)] = r
        return t
