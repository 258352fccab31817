"""Plain restatements of the serving operators in 64 bits (or whole numbers),
one token, row or entry at a time.  Used by the tests only; shares no code with
the GPU path.
"""

import numpy as np

PAGE = 64


def e4m3_value(codes):
    """Values of E4M3 codes (uint8), from the bits: S EEEE MMM, bias 7."""
    c = np.asarray(codes, dtype=np.int64)
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(s == 1, -v, v)


# ------------------------------------------------------------------ append


def append_targets(cu, lens, table, num_pages, max_pos=None, refcount=None):
    """For each token: (page, row, position), or None where it is not written;
    and whether a bad one was met.  Tokens outside the sequences are None."""
    out, bad = {}, False
    table = np.asarray(table)
    for b in range(len(lens)):
        for t in range(cu[b], cu[b + 1]):
            pos = lens[b] - (cu[b + 1] - t)
            if pos < 0 or pos >= table.shape[1] * PAGE or (max_pos is not None and pos >= max_pos):
                bad = True
                continue
            page = int(table[b, pos // PAGE])
            if page < 0 or page >= num_pages or (refcount is not None and refcount[page] != 1):
                bad = True
                continue
            out[t] = (page, pos % PAGE, pos)
    return out, bad


def latent_row(c, r, pos, weight=None, eps=1e-6, cos_sin=None, interleaved=False):
    """(c', r') in float64 of one token's c [512] and r [64]."""
    c = np.asarray(c, dtype=np.float64)
    r = np.array(r, dtype=np.float64)
    if weight is not None:
        c = c / np.sqrt(np.mean(c * c) + eps) * np.asarray(weight, dtype=np.float64)
    if cos_sin is not None:
        cos, sin = np.asarray(cos_sin[pos][:32], np.float64), np.asarray(cos_sin[pos][32:], np.float64)
        at = (np.arange(0, 64, 2), np.arange(1, 64, 2)) if interleaved else (np.arange(32), np.arange(32, 64))
        x, y = r[at[0]], r[at[1]]
        r[at[0]], r[at[1]] = x * cos - y * sin, y * cos + x * sin
    return c, r


# ------------------------------------------------------------------ pages


def _pages(n):
    return -(-n // PAGE)


class Pool:
    """The bookkeeping of a page pool as plain lists."""

    def __init__(self, refcount, table, seqlens):
        self.ref = [int(v) for v in refcount]
        self.table = [[int(v) for v in row] for row in table]
        self.lens = [int(v) for v in seqlens]
        self.bad = self.empty = False

    def _free(self):
        return [p for p, c in enumerate(self.ref) if c == 0]

    def grow(self, rows, new):
        free, at, width = self._free(), 0, len(self.table[0])
        for r, a in zip(rows, new):
            if not 0 <= r < len(self.table) or list(rows).count(r) > 1 or a < 0 or self.lens[r] < 0 or \
                    self.lens[r] + a > width * PAGE:
                self.bad = True
                continue
            have, want = _pages(self.lens[r]), _pages(self.lens[r] + a)
            first, at = at, at + want - have
            if want > have and at > len(free):
                self.empty = True
                continue
            for j in range(have, want):
                self.table[r][j] = free[first + j - have]
                self.ref[free[first + j - have]] = 1
            self.lens[r] += a

    def fork(self, parents, children):
        free, at, width = self._free(), 0, len(self.table[0])
        pairs, lens0, ref0 = [], list(self.lens), list(self.ref)
        for p, c in zip(parents, children):
            ok = 0 <= p < len(self.table) and 0 <= c < len(self.table) and list(children).count(c) == 1 and \
                p not in list(children) and lens0[c] == 0 and 0 <= lens0[p] <= width * PAGE and \
                all(0 <= q < len(ref0) and ref0[q] > 0 for q in self.table[p][:_pages(lens0[p])])
            pairs.append((-1, -1))
            if not ok:
                self.bad = True
                continue
            full, tail = lens0[p] // PAGE, lens0[p] % PAGE > 0
            at += tail
            if tail and at > len(free):
                self.empty = True
                continue
            row = [-1] * width
            for j in range(full):
                row[j] = self.table[p][j]
                self.ref[row[j]] += 1
            if tail:
                row[full] = free[at - 1]
                self.ref[free[at - 1]] = 1
                pairs[-1] = (self.table[p][full], free[at - 1])
            self.table[c] = row
            self.lens[c] = lens0[p]
        return pairs

    def free(self, rows):
        for r in rows:
            if not 0 <= r < len(self.table) or not 0 <= self.lens[r] <= len(self.table[r]) * PAGE:
                self.bad = True
                continue
            for j in range(_pages(self.lens[r])):
                p, self.table[r][j] = self.table[r][j], -1
                if not 0 <= p < len(self.ref) or self.ref[p] <= 0:
                    self.bad = True
                else:
                    self.ref[p] -= 1
            self.lens[r] = 0

    def compact(self):
        n = sum(c != 0 for c in self.ref)
        src = [p for p, c in enumerate(self.ref) if c != 0 and p >= n]
        dst = [p for p, c in enumerate(self.ref) if c == 0 and p < n]
        live = [c != 0 for c in self.ref]
        to = dict(zip(src, dst))
        for r, row in enumerate(self.table):
            if not 0 <= self.lens[r] <= len(row) * PAGE:
                self.bad = True
            for j in range(min(_pages(max(self.lens[r], 0)), len(row))):
                if not 0 <= row[j] < len(self.ref) or not live[row[j]]:
                    self.bad = True
                else:
                    row[j] = to.get(row[j], row[j])
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
        return list(to.items())


def copy_pairs(pairs, num_pages):
    """The pairs that copy_pages carries out, and whether it refuses any."""
    done, bad = [], False
    for i, (a, b) in enumerate(pairs):
        if (a < 0 and b < 0) or a == b:
            continue
        clash = any(j != i and ((y == b and j < i) or (x == b and x != y)) for j, (x, y) in enumerate(pairs))
        if not (0 <= a < num_pages and 0 <= b < num_pages) or clash:
            bad = True
        else:
            done.append((a, b))
    return done, bad


# ------------------------------------------------------------------ prompt


def prompt_attention(q, k, v, cu_q, cu_k, causal, scale):
    """(out, lse, mix, reach) in float64: mix = sum_j w_j |v_j| (what a rounding
    of the weights can move the output by) and reach = max_j scale |q|.|k_j|
    (what the rounding of a score scales with).  Rows outside every sequence
    are NaN."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    out = np.full((q.shape[0], q.shape[1], v.shape[2]), np.nan)
    mix, lse, reach = out.copy(), np.full(q.shape[:2], np.nan), np.full(q.shape[:2], np.nan)
    group = q.shape[1] // k.shape[1]
    for b in range(len(cu_q) - 1):
        lq, lk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        rows = slice(cu_q[b], cu_q[b + 1])
        for h in range(q.shape[1]):
            kk, vv = k[cu_k[b]:cu_k[b + 1], h // group], v[cu_k[b]:cu_k[b + 1], h // group]
            s = scale * q[rows, h] @ kk.T
            if causal:
                hide = np.arange(lk)[None] > np.arange(lq)[:, None] + lk - lq
                s[hide] = -np.inf
            top = s.max(1, initial=-np.inf)
            e = np.exp(s - np.where(np.isfinite(top), top, 0.0)[:, None])
            z = e.sum(1)
            w = e / np.where(z > 0, z, 1.0)[:, None]
            out[rows, h], mix[rows, h] = w @ vv, w @ np.abs(vv)
            with np.errstate(divide="ignore"):
                lse[rows, h] = top + np.log(z)
            reach[rows, h] = (scale * np.abs(q[rows, h]) @ np.abs(kk).T).max(1, initial=0.0)
    return out, lse, mix, reach


# ------------------------------------------------------------------ chunks of new tokens


def record_rows(rec):
    """[n, 576] float64 values of FP8 records uint8 [n, 656]."""
    rec = np.ascontiguousarray(rec)
    scale = rec[:, 512:528].copy().view(np.float32).astype(np.float64)
    rope = (rec[:, 528:].copy().view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return np.concatenate([e4m3_value(rec[:, :512]) * np.repeat(scale, 128, axis=1), rope], 1)


def request_keys(cache, table_row, length):
    """Rows 0 .. length - 1 of a request in a pool [pages, 64, width], and whether each is on a page of the pool (else
    page 0 stands in)."""
    rows, seen = [], []
    for p in range(length):
        j = p // PAGE
        page = int(table_row[j]) if j < len(table_row) else -1
        good = 0 <= page < cache.shape[0]
        seen.append(good)
        rows.append(cache[page if good else 0, p % PAGE])
    return np.array(rows).reshape(length, cache.shape[2]), np.array(seen, dtype=bool)


def chunk_attention(q, keys, seen, cu, lens, causal, scale):
    """As prompt_attention, for chunks over their requests' keys: keys[b] [len, 576] float64 (the first 512 dims the value)
    and seen[b] [len] (a key on a page outside the pool is masked)."""
    q = np.asarray(q, dtype=np.float64)
    out = np.full((*q.shape[:2], 512), np.nan)
    mix, lse, reach = out.copy(), np.full(q.shape[:2], np.nan), np.full(q.shape[:2], np.nan)
    for b in range(len(lens)):
        n, total = cu[b + 1] - cu[b], max(lens[b], 0)
        for i in range(n):
            see = np.array(seen[b][:total])
            if causal:
                see = see & (np.arange(total) <= total - n + i)
            k = keys[b][:total][see]
            v = k[:, :512]
            t = cu[b] + i
            s = scale * q[t] @ k.T
            top = s.max(1, initial=-np.inf)
            e = np.exp(s - np.where(np.isfinite(top), top, 0.0)[:, None])
            z = e.sum(1)
            w = e / np.where(z > 0, z, 1.0)[:, None]
            out[t], mix[t] = w @ v, w @ np.abs(v)
            with np.errstate(divide="ignore"):
                lse[t] = top + np.log(z)
            reach[t] = (scale * np.abs(q[t]) @ np.abs(k).T).max(1, initial=0.0)
    return out, lse, mix, reach


def rope_frequencies(dim, base, scaling, factor, original, low, high):
    """(frequencies, magnitude) of rotary positions, from their definitions."""
    freq, magnitude = [], 1.0
    for i in range(dim // 2):
        f = base ** (-2.0 * i / dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "ntk":
            f = (base * factor ** (dim / (dim - 2.0))) ** (-2.0 * i / dim)
        elif scaling == "yarn":
            place = [dim * np.log(original / (2 * np.pi * t)) / (2 * np.log(base)) for t in (high, low)]
            a, b = max(np.floor(place[0]), 0), min(np.ceil(place[1]), dim - 1)
            w = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
            f = w * f / factor + (1 - w) * f
            magnitude = 0.1 * np.log(factor) + 1.0
        elif scaling == "wavelength":
            w = min(max((original * f / (2 * np.pi) - low) / (high - low), 0.0), 1.0)
            f = (1 - w) * f / factor + w * f
        freq.append(f)
    return np.array(freq), float(magnitude)


def rope_head(x, cos_sin_row, offset, interleaved, weight=None, eps=1e-6):
    """One head [dim] in float64: norm (with weights), then dims offset .. offset + len(cos_sin_row) turned."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y) + eps) * np.asarray(weight, dtype=np.float64)
    if cos_sin_row is not None:
        n = len(cos_sin_row) // 2
        cos, sin = (np.asarray(v, dtype=np.float64) for v in (cos_sin_row[:n], cos_sin_row[n:]))
        lo, hi = (slice(offset, offset + 2 * n, 2), slice(offset + 1, offset + 2 * n, 2)) if interleaved else \
            (slice(offset, offset + n), slice(offset + n, offset + 2 * n))
        a, b = y[lo].copy(), y[hi].copy()
        y[lo], y[hi] = a * cos - b * sin, b * cos + a * sin
    return y
