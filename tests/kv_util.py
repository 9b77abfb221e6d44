"""Plain 64-bit references of the paged 8-bit cache, the attention over it
and the residual norm (numpy, float64), and seeded inputs for their tests."""
import math

import numpy as np

PAGE = 64


def rotate(x, pos, rope, rot, pairs):
    """x [heads][D] float64 at one position -> float64 (one exact product each)."""
    y = x.copy()
    if rot == 0:
        return y
    c, s = rope[pos, 0].astype(np.float64), rope[pos, 1].astype(np.float64)
    h = rot // 2
    if pairs:
        a, b = x[:, 0:rot:2], x[:, 1:rot:2]
        y[:, 0:rot:2], y[:, 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[:, :h], x[:, h:rot]
        y[:, :h], y[:, h:rot] = a * c - b * s, b * c + a * s
    return y


def scale_for(m):
    """The smallest power of two (2^-126 .. 2^121) with m < 128 * scale; 0 for m = 0."""
    if m == 0:
        return 0.0
    e = -126
    while not m < 128 * 2.0 ** e and e < 121:
        e += 1
    return 2.0 ** e


class Cache:
    """The cache and its append, token by token: every token is quantised with
    the final scale of its page, from its own values (no codes are shifted)."""

    def __init__(self, pages, heads, dim):
        self.k, self.v = {}, {}
        self.heads, self.dim = heads, dim

    def put(self, page, slot, k, v):
        for store, x in ((self.k, k), (self.v, v)):
            if slot == 0:
                store[page] = {}
            store.setdefault(page, {})[slot] = np.asarray(x, dtype=np.float32).astype(np.float64)

    def codes(self, store, page):
        """(scale [heads], codes {slot: [heads][dim]}) of a page."""
        rows = store[page]
        scale = np.array([scale_for(max(np.abs(r[h]).max() for r in rows.values())) for h in range(self.heads)])
        out = {}
        for slot, r in rows.items():
            c = np.zeros_like(r)
            for h in range(self.heads):
                if scale[h]:
                    c[h] = np.floor(r[h] / scale[h])
            out[slot] = (np.clip(c, -128, 127) + 128).astype(np.uint8)
        return scale, out


def append_rows(cache, qkv, hq, hkv, dim, rope, rot, pairs, cu, kv_len, table, num_pages):
    """Appends to `cache` and returns the rotated queries as float16 (None
    rows: padding)."""
    q_out = {}
    limit = rope.shape[0] if rot else 1 << 60
    for s in range(len(kv_len)):
        n = cu[s + 1] - cu[s]
        for i in range(n):
            r, pos = cu[s] + i, kv_len[s] - n + i
            x = qkv[r].astype(np.float64).reshape(hq + 2 * hkv, dim)
            if pos < 0 or pos >= limit:
                q_out[r] = np.zeros((hq, dim), np.float16)
                continue
            qk = rotate(x[:hq + hkv], pos, rope, rot, pairs).astype(np.float32)
            q_out[r] = qk[:hq].astype(np.float16)
            if pos // PAGE < table.shape[1] and 0 <= table[s, pos // PAGE] < num_pages:
                cache.put(int(table[s, pos // PAGE]), pos % PAGE, qk[hq:], x[hq + hkv:])
    return q_out


def attention(q, cu, kv_len, table, k, v, ks, vs, scale, window, sinks):
    """float64 reference: (out, sum w |v| / sum w, largest sum |q||k| * scale of a row).
    q [rows][hq][D]; k uint8 [P][hkv][64][D], v uint8 [P][hkv][D][64].  Rows that
    belong to no sequence stay NaN."""
    rows, hq, dim = q.shape
    P, hkv = ks.shape
    group = hq // hkv
    out = np.full((rows, hq, dim), np.nan)
    mag = np.zeros((rows, hq, dim))
    dot = np.zeros((rows, hq))
    for s in range(len(kv_len)):
        n = cu[s + 1] - cu[s]
        if n <= 0:
            continue
        t = max(0, min(int(kv_len[s]), table.shape[1] * PAGE))
        ids = table[s, :(t + PAGE - 1) // PAGE].astype(np.int64)
        there = np.repeat((ids >= 0) & (ids < P), PAGE)[:t]
        safe = np.where((ids >= 0) & (ids < P), ids, 0)
        pos = kv_len[s] - n + np.arange(n)
        j = np.arange(t)
        see = (j[None] <= pos[:, None]) & there[None]
        if window:
            see &= (j[None] > pos[:, None] - window) | (j[None] < sinks)
        for h in range(hkv):
            kk = ((k[safe, h].astype(np.float64) - 127.5) * ks[safe, h].astype(np.float64)[:, None, None]).reshape(-1, dim)[:t]
            vv = (v[safe, h].astype(np.float64) - 127.5) * vs[safe, h].astype(np.float64)[:, None, None]
            vv = vv.transpose(0, 2, 1).reshape(-1, dim)[:t]
            qq = q[cu[s]:cu[s] + n, h * group:(h + 1) * group].astype(np.float64)
            z = np.einsum("ngd,td->ngt", qq, kk) * scale
            a = np.einsum("ngd,td->ngt", np.abs(qq), np.abs(kk)) * scale
            z = np.where(see[:, None], z, -np.inf)
            m = z.max(-1, keepdims=True, initial=-1e300)
            w = np.exp(z - m)
            total = w.sum(-1, keepdims=True)
            w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
            out[cu[s]:cu[s] + n, h * group:(h + 1) * group] = w @ vv
            mag[cu[s]:cu[s] + n, h * group:(h + 1) * group] = w @ np.abs(vv)
            dot[cu[s]:cu[s] + n, h * group:(h + 1) * group] = np.where(see[:, None], a, 0).max(-1, initial=0)
    return out, mag, dot


def attention_tolerance(ref, mag, dot, keys, dim):
    """How far an fp16 output may be from the reference, element by element.
    With u = 2^-24 (half an fp32 step) and e the relative error of a weight:
      - a score in units of log2 e is a sum of dim products of fp16 by an
        exact code plus the half-code term: at most (dim + 8) u of
        sum |q||k| * scale (the 8: the half-code sum's own dim additions are of
        fp16 values, bounded by the same sum; the scale's product and the
        maximum's subtraction, one rounding each), and exp2's instruction is
        within one fp32 step (2 u);
      - a weight is rounded to fp16 once: 2^-11;
      - a weight's rescalings, one per tile of 64 keys, and the sums over the
        keys: (keys / 64 + keys) roundings of u, on both sums.
    The quotient takes the numerator's and the denominator's error.  The
    output is rounded to fp16: 2^-11 of it, or half a subnormal step (2^-25)."""
    u = 2.0 ** -24
    e = 2 * (2 * dim + 16) * u * np.asarray(dot)[..., None] + 2 * 2 * u + 2.0 ** -11 + 2 * (keys + keys / 64 + 8) * u
    return 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + e * mag


def norm(y, res, res_type, post, gate, scale, pre, eps):
    """(r' as stored, x float64) in float64."""
    r = res.astype(np.float64)
    if y is not None:
        u = y.astype(np.float64)
        if post is not None:
            u = u / np.sqrt((u * u).mean(1, keepdims=True) + eps) * post.astype(np.float64)
        if gate is not None:
            u = u * gate.astype(np.float64)
        r = (r + scale * u).astype(np.float32).astype(res_type)
    else:
        r = res
    w = r.astype(np.float64)
    x = w / np.sqrt((w * w).mean(1, keepdims=True) + eps)
    if pre is not None:
        x = x * pre.astype(np.float64)
    return r, x


def lay_out(rng, kv_len, num_extra=2, width_extra=1, unused=-1):
    """(page table, number of pages): every sequence's pages scattered over the pool."""
    used = [max(0, math.ceil(t / PAGE)) for t in kv_len]
    pages = sum(used) + num_extra
    order = rng.permutation(pages)
    table = np.full((len(kv_len), max(used + [1]) + width_extra), unused, dtype=np.int32)
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u
    return table, pages
