"""A plain form of the paged 4-bit key/value cache in 64 bits on the CPU (numpy), for the tests of
the tq_kv_* calls: layout, rounding, plan, rotary positions and attention, each written element by
element from its definition in tq.h."""
import numpy as np

PLACE = np.array([0, 2, 1, 3])


class Layout:
    """Byte offsets of the cache's elements."""

    def __init__(self, kv_heads, head_dim, page_tokens):
        self.kv, self.dim, self.page = kv_heads, head_dim, page_tokens
        self.nb = head_dim // 32
        self.words = min(self.nb, 4)
        self.quants, self.scales = 256 * self.nb, 32 * self.nb
        self.half = self.quants + self.scales
        self.page_bytes = kv_heads * (page_tokens // 16) * 2 * self.half

    def offsets(self, slot, which):
        """(byte of each element, its shift, low byte of its scale), each [kv, dim], of one slot's
        keys (which 0) or values (1)."""
        page, tok = slot // self.page, slot % self.page
        tile, t = tok // 16, tok % 16
        h, e = np.arange(self.kv)[:, None], np.arange(self.dim)[None]
        base = page * self.page_bytes + ((h * (self.page // 16) + tile) * 2 + which) * self.half
        b, i = e // 32, e % 16
        chunk, word = b // self.words, b % self.words
        four, sixteen, place = (i // 4, t, PLACE[i % 4]) if which == 0 else (t // 4, i, PLACE[t % 4])
        at = (((chunk * 4 + four) * 16 + sixteen) * self.words + word) * 4 + place
        scale = self.quants + ((t // 4 * self.nb + b) * 4 + t % 4) * 2
        return base + at, (e % 32 // 16 * 4) + 0 * h, base + scale


def read(data, lay, slots):
    """Keys and values [rows, kv, dim] in fp64 of a flat uint8 cache; zeros for slots outside."""
    n_slots = data.size // lay.page_bytes * lay.page
    out = np.zeros((2, len(slots), lay.kv, lay.dim))
    for r, s in enumerate(np.asarray(slots, np.int64)):
        if not 0 <= s < n_slots:
            continue
        for w in (0, 1):
            at, shift, sc = lay.offsets(s, w)
            n = (data[at].astype(np.int64) >> shift) & 15
            d = (data[sc].astype(np.uint16) | data[sc + 1].astype(np.uint16) << 8).view(np.float16)
            with np.errstate(invalid="ignore"):
                out[w, r] = d.astype(np.float64) * (n - 8)
    return out[0], out[1]


def round_block(x):
    """(d fp16, n 0..15) of one block of 32 fp32 values."""
    x = np.asarray(x, np.float32)
    if not np.isfinite(x).all():
        return np.float16(np.nan), np.full(32, 8)
    m = x[np.argmax(np.abs(x))]  # the first of the largest
    d = np.float16(np.clip(np.float64(m) / -8, -65504, 65504))
    if d == 0:
        return d, np.full(32, 8)
    n = np.clip(np.rint(x.astype(np.float64) / np.float64(d)), -8, 7).astype(np.int64) + 8
    return d, n


def write(data, lay, slots, k, v):
    """Rounds fp32 rows k, v [rows, kv, dim] into a flat uint8 cache, in place."""
    n_slots = data.size // lay.page_bytes * lay.page
    for r, s in enumerate(np.asarray(slots, np.int64)):
        if not 0 <= s < n_slots:
            continue
        for w, x in ((0, k[r]), (1, v[r])):
            at, shift, sc = lay.offsets(s, w)
            for h in range(lay.kv):
                for b in range(lay.nb):
                    e = slice(32 * b, 32 * b + 32)
                    d, n = round_block(x[h, e])
                    for a, sh, q in zip(at[h, e], shift[h, e], n):
                        data[a] = (int(data[a]) & (0xF0 if sh == 0 else 0x0F)) | (int(q) << int(sh))
                    bits = int(np.array(d).view(np.uint16))
                    data[sc[h, 32 * b]] = bits & 255
                    data[sc[h, 32 * b] + 1] = bits >> 8


def turn(x, positions, inv_freq, sections, interleaved):
    """Rows x [rows, heads, dim] turned in fp64; positions [axes, rows]."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    pairs = len(inv_freq)
    axis = np.repeat(np.arange(len(sections)), sections)
    for p in range(pairs):
        th = positions[axis[p]].astype(np.float64) * np.float64(inv_freq[p])
        c, s = np.cos(th)[:, None], np.sin(th)[:, None]
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)
        y[..., i] = x[..., i] * c - x[..., j] * s
        y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def plan(kv_len, new_len, table, rows, page, pages, free=None, count=None):
    """The step plan, request by request with an explicit stack. Returns a dict of numpy arrays."""
    R, mb = table.shape
    kv, new = [int(a) for a in kv_len], [int(a) for a in new_len]
    table = table.copy()
    managed = free is not None
    status = 0
    ceil = lambda n: -(-n // page)  # noqa: E731
    for a, b in zip(kv, new):
        if a < 0 or b < -1:
            status |= 8
        elif ceil(a + max(b, 0)) > mb:
            status |= 4
    ok = [a >= 0 and b >= -1 for a, b in zip(kv, new)]
    back = sum(ceil(a) for a, b, g in zip(kv, new, ok) if g and b < 0) if managed else 0
    need = sum(ceil(a + b) - ceil(a) for a, b, g in zip(kv, new, ok) if g and b >= 0) if managed else 0
    if managed and not (0 <= count <= pages and count + back <= pages):
        status |= 8
    elif managed and need > count + back:
        status |= 1
    if sum(b for b, g in zip(new, ok) if g and b > 0) > rows:
        status |= 2
    res = {"block_table": table, "cu_new": np.zeros(R + 1, np.int64), "seq_len": np.maximum(kv, 0),
           "slots": np.full(rows, -1), "positions": np.full(rows, -1), "requests": np.full(rows, -1),
           "status": np.array([status])}
    if managed:
        res["free_pages"], res["free_count"] = free.copy(), np.array([count])
    if status:
        return res
    stack = list(free[:count]) if managed else []
    if managed:
        for r in range(R):
            if new[r] < 0:
                stack += list(table[r, :ceil(kv[r])])
        res["free_pages"][:len(stack)] = stack
    t = 0
    for r in range(R):
        if new[r] < 0:
            res["seq_len"][r] = 0
        else:
            if managed:
                for col in range(ceil(kv[r]), ceil(kv[r] + new[r])):
                    table[r, col] = stack.pop()
            for i in range(new[r]):
                pos = kv[r] + i
                pg = int(table[r, pos // page])
                res["slots"][t] = pg * page + pos % page if 0 <= pg < pages else -1
                res["positions"][t], res["requests"][t] = pos, r
                t += 1
            res["seq_len"][r] = kv[r] + new[r]
        res["cu_new"][r + 1] = t
    if managed:
        res["free_count"] = np.array([len(stack)])
    return res


def attention(q, k_of, v_of, seq_len, cu_new, kv_heads, scale, window, hidden=None):
    """(out, lse, bound of out, bound of lse) in fp64 for q [rows, heads, dim]; k_of(r), v_of(r):
    keys and values [len, kv, dim] of request r; hidden(r): tokens that no row sees (bad pages).

    The bounds are per unit of the kernel's own roundings, without the output's and the weights'
    (which the caller knows): with S = scale * sum|q||k| the largest over a row's tokens, a logit is
    off by at most dl = 2^-18 S (32 fp32 products a block, the blocks' sum, the query to 2^-22 of its
    row's largest) + 2^-22 (|logit| + 40) (the exponent's fp32 argument and its reference); the
    weights then by e^dl - 1 each, the sums over n tokens by (n / 16 + 64) 2^-23 of the sum of
    magnitudes (32 tokens a product, steps one after another, waves and parts joined).

    Weights times a value's scale enter the second product as fp16 numbers x = p d, exact to 2^-25
    (or lost whole) below fp16's normal range, and a nibble is at most 8: out is off by
    8 min(2^-25, x) / l a token, with l = sum p. The kernel takes p = 2^(s - m), m <= max s + T - 28,
    so l = max p / max w >= 2^(28 - T) / max w, w the softmax weights. T bounds the scales,
    max d < 2^(T - 15); it is a power of two up to 16 with max d >= 2^(T/2 - 15) (subnormal d: T = 1,
    max d >= 2^-24), or above 16 exact, max d >= 2^(T - 16). So 8 * 2^-25 / l <= 2^(T - 50) max w is at
    most 2^-27 max w max d (at T = 16; 2^-25 at T = 1), and max d <= max |v| of the row's tokens."""
    q = np.asarray(q, np.float64)
    rows, heads, dim = q.shape
    G = heads // kv_heads
    out, lse = np.full(q.shape, np.nan), np.full((rows, heads), np.nan)
    tol, ltol, mag = np.zeros(q.shape), np.zeros((rows, heads)), np.zeros(q.shape)
    for r, n in enumerate(seq_len):
        new = int(cu_new[r + 1] - cu_new[r])
        if new == 0:
            continue
        k, v = k_of(r), v_of(r)
        t = np.arange(n)
        for i in range(new):
            row, pos = int(cu_new[r]) + i, n - new + i
            see = t <= pos
            if window:
                see &= t > pos - window
            if hidden is not None:
                see &= ~hidden(r)
            for h in range(heads):
                if not see.any():
                    out[row, h], lse[row, h] = 0.0, -np.inf
                    continue
                kk, vv = k[see, h // G], v[see, h // G]
                x = scale * (kk @ q[row, h])
                top = x.max()
                p = np.exp(x - top)
                tot = p.sum()
                out[row, h] = (p @ vv) / tot
                lse[row, h] = top + np.log(tot)
                mag[row, h] = (p @ np.abs(vv)) / tot
                s = scale * (np.abs(kk) @ np.abs(q[row, h])).max()
                dl = 2.0**-18 * s + 2.0**-22 * (np.abs(x).max() + 40)
                many = (see.sum() / 16 + 64) * 2.0**-23
                tol[row, h] = mag[row, h] * (2 * np.expm1(dl) + 2 * many)
                far = np.abs(vv).max()  # max w = 1 / tot; x / l = w d, d <= far
                tol[row, h] += np.minimum((2.0**-27 if far >= 2.0**-14 else 2.0**-25) * far / tot, 8 * far * p / tot).sum()
                ltol[row, h] = dl + many + 2.0**-22 * (abs(lse[row, h]) + 40)
    return out, lse, tol, ltol, mag
