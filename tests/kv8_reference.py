"""Plain 64-bit implementations of the 8-bit KV cache and of the pool of pages,
and the error bounds the GPU results are held to."""
import numpy as np

EXP_LO, EXP_HI = 87, 167
E4M3_MAX = 448.0


def e4m3_table():
    b = np.arange(256)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7.0), m / 8 * 2.0 ** -6)
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b >= 128, -v, v)


_TABLE = e4m3_table()
_POS = _TABLE[:127]            # 0 .. 448, ascending with the byte


def e4m3_values(b):
    return _TABLE[np.asarray(b, np.uint8)]


def e4m3_round(x):
    """Bytes of the nearest e4m3 values (ties to the even byte), saturating."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), E4M3_MAX)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def block_exponent(amax):
    """Least e in EXP_LO..EXP_HI with amax <= 448 * 2^(e - 127); EXP_HI if none."""
    for e in range(EXP_LO, EXP_HI + 1):
        if amax <= E4M3_MAX * 2.0 ** (e - 127):
            return e
    return EXP_HI


def append(K, V, kc, vc, exp, table, lens, cu):
    """K, V [n, Hkv, D] float64; kc, vc, exp numpy uint8 arrays, changed in place."""
    P, _, Hkv, D = kc.shape
    block = 64 // exp.shape[1]
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        done = 0
        while done < n:
            pos = lens[b] - n + done
            at = pos % block
            m = min(block - at, n - done)
            page = table[b][pos // 64] if 0 <= pos // 64 < len(table[b]) else -1
            if pos >= 0 and 0 <= page < P:
                lo = pos % 64
                for i, (X, c) in enumerate(((K, kc), (V, vc))):
                    for g in range(Hkv):
                        x = X[cu[b] + done: cu[b] + done + m, g]
                        old = int(exp[page, lo // block, g, i]) if at else EXP_LO
                        e = max(old, block_exponent(np.abs(x).max()))
                        if at and e > old:
                            was = e4m3_values(c[page, lo - at:lo, g])
                            c[page, lo - at:lo, g] = e4m3_round(was * 2.0 ** (old - e))
                        c[page, lo:lo + m, g] = e4m3_round(x * 2.0 ** (127 - e))
                        exp[page, lo // block, g, i] = e
            done += m


def attention(q, kc, vc, exp, table, idx, seq, pos, sm_scale):
    """Rows q [n, Hq, D] float64 of sequences seq[r] at positions pos[r].
    Returns (out, lse, tol_out, tol_lse) in float64.

    Bounds, with u = log2 of a weight: the score is a sum of D exact products
    in fp32 over 8 or fewer matrix steps, off by at most 2^-19 of the sum of
    the products' magnitudes (32 roundings of 2^-24), plus 2^-22 |u| for the
    scaling and for adding V's exponent (|ev| <= 40 among it), plus 2^-21 for
    exp2, all relative to the weight after ln 2.  The weights that multiply V
    are rounded to fp16 (2^-11; below its normal range an absolute 2^-25 of a
    scale on which the largest weight is at least 2^7, so 2^-32 per key), sums
    over k keys are off by at most (k/16 + 64) 2^-23 of the sum of magnitudes,
    and the output is rounded to bf16 (2^-8)."""
    n, Hq, D = q.shape
    P, _, Hkv, _ = kc.shape
    G, block = Hq // Hkv, 64 // exp.shape[1]
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    tol_o, tol_l = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    k = idx.shape[1]
    for r in range(n):
        t = min(pos[r], len(table[seq[r]]) * 64 - 1)
        e = idx[r][: max(min(k, t + 1), 0)]
        e = e[(e >= 0) & (e <= t)]
        page = table[seq[r]][e // 64] if len(e) else np.zeros(0, int)
        ok = (page >= 0) & (page < P)
        e, page = e[ok], page[ok]
        if not len(e):
            continue
        s = e % 64
        sc = 2.0 ** (exp[page, s // block].astype(np.float64) - 127)      # [m, Hkv, 2]
        kk, vv = e4m3_values(kc[page, s]), e4m3_values(vc[page, s])        # [m, Hkv, D]
        for h in range(Hq):
            g = h // G
            x = (kk[:, g] @ q[r, h]) * sc[:, g, 0] * sm_scale
            mag = (np.abs(kk[:, g]) @ np.abs(q[r, h])) * sc[:, g, 0] * abs(sm_scale)
            M = x.max()
            p = np.exp(x - M)
            L = p.sum()
            v = vv[:, g] * sc[:, g, 1:2]
            out[r, h] = p @ v / L
            lse[r, h] = M + np.log(L)
            ev = np.abs(np.log2(sc[:, g, 1])).max()
            d = 2.0 ** -19 * mag.max() + np.log(2) * (2.0 ** -22 * (np.abs(x).max() * 1.45 + ev + 40) + 2.0 ** -21)
            sums = (len(e) / 16 + 64) * 2.0 ** -23
            A = p @ np.abs(v) / L
            big = (p[:, None] * sc[:, g, 1:2] * E4M3_MAX).max() / L * len(e) * 2.0 ** -32
            tol_o[r, h] = 2.0 ** -8 * np.abs(out[r, h]) + 1.01 * (2 * d + 2.0 ** -11 + 2 * sums) * A + big
            tol_l[r, h] = d + sums + 2.0 ** -22 * (abs(lse[r, h]) + 60)
    return out, lse, tol_o, tol_l


class Pool:
    """The pool of pages, one entry at a time."""

    def __init__(self, num_pages, n_slots, max_pages, bufs=()):
        self.table = np.full((n_slots, max_pages), -1, np.int32)
        self.lens = np.zeros(n_slots, np.int32)
        self.refs = np.zeros(num_pages, np.int32)
        self.bufs = list(bufs)   # numpy arrays [num_pages, ...]

    def _grant(self, entries):
        """entries: (slot or None if refused, first, need, to) in order."""
        free = np.nonzero(self.refs == 0)[0]
        used = asked = 0
        status = []
        for slot, first, need, to in entries:
            if slot is None:
                status.append(2)
                continue
            asked += need
            if need and asked > len(free):
                status.append(1)
                continue
            for j in range(need):
                self.table[slot, first + j] = free[used]
                self.refs[free[used]] = 1
                used += 1
            self.lens[slot] = to
            status.append(0)
        return np.array(status, np.int32)

    def extend(self, slots, new_lens):
        seen, entries = set(), []
        n_slots, max_pages = self.table.shape
        for s, L in zip(slots, new_lens):
            ok = 0 <= s < n_slots
            again = s in seen
            if ok:
                seen.add(s)
            if not ok or again or L < self.lens[s] or L > 64 * max_pages:
                entries.append((None, 0, 0, 0))
                continue
            a, b = -(-int(self.lens[s]) // 64), -(-int(L) // 64)
            entries.append((s, a, b - a, L))
        return self._grant(entries)

    def fork(self, parents, children):
        seen, entries = set(), []
        n_slots = len(self.lens)
        before = self.lens.copy()
        for p, c in zip(parents, children):
            ok = 0 <= c < n_slots
            again = c in seen
            if ok:
                seen.add(c)
            if not ok or again or before[c] != 0 or not 0 <= p < n_slots:
                entries.append((None, 0, 0, 0))
                continue
            entries.append((c, int(before[p]) // 64, int(before[p] % 64 != 0), before[p]))
        status = self._grant(entries)
        for p, c, st in zip(parents, children, status):
            if st:
                continue
            full = int(before[p]) // 64
            self.table[c, :full] = self.table[p, :full]
            np.add.at(self.refs, self.table[p, :full], 1)
            if before[p] % 64:
                for b in self.bufs:
                    b[self.table[c, full]] = b[self.table[p, full]]
        return status

    def free(self, slots):
        for s in slots:
            if not 0 <= s < len(self.lens):
                continue
            n = -(-int(self.lens[s]) // 64)
            for p in self.table[s, :n]:
                self.refs[p] -= 1
            self.table[s, :n] = -1
            self.lens[s] = 0

    def compact(self):
        used = self.refs != 0
        n = int(used.sum())
        ids = np.arange(len(used))
        high, low = ids[n:][used[n:]], ids[:n][~used[:n]]
        to = np.where(used, ids, -1)
        to[high] = low
        for b in self.bufs:
            b[low] = b[high]
        self.refs[low] = self.refs[high]
        self.refs[n:] = 0
        for s in range(len(self.lens)):
            m = -(-int(self.lens[s]) // 64)
            self.table[s, :m] = to[self.table[s, :m]]
            self.table[s, m:] = -1
        return to.astype(np.int32), n
