"""Plain 64-bit forms of the 8-bit paged cache and its attention, and inputs
for them.  Source: the format and the formulas of include/dflash.h, written
here with numpy and sharing no code with the library."""
import numpy as np

EMIN, EMAX, BIAS = -100, 119, 127


def code_values():
    """The value of each e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = np.nan if (b & 127) == 127 else (-x if b >> 7 else x)
    return v


VALUES = code_values()
STEPS = VALUES[:127]


def quantise(x):
    """Codes and exponent bytes of the vectors in the last dimension of x (float64)."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    top = np.abs(x).max(-1)
    e = np.full(top.shape, EMIN)
    for i in range(EMIN, EMAX):
        e = np.where(top > 448.0 * 2.0 ** i, i + 1, e)
    y = np.abs(x) / 2.0 ** e[..., None].astype(np.float64)
    hi = np.searchsorted(STEPS, np.minimum(y, 448.0)).clip(0, 126)  # first step at or above
    lo = np.maximum(hi - 1, 0)
    up, down = STEPS[hi] - np.minimum(y, 448.0), np.minimum(y, 448.0) - STEPS[lo]
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(x), 128, 0)
    code = np.where(bad[..., None], 0, code)
    return code.astype(np.uint8), np.where(bad, 255, e + BIAS).astype(np.uint8)


def dequantise(codes, exps):
    sc = np.where(exps == 255, np.nan, 2.0 ** (exps.astype(np.float64) - BIAS))
    return VALUES[codes] * sc[..., None]


class Case:
    """Sequences given as (rows, positions before them); a negative second
    number leaves the first rows at negative positions (padding)."""

    def __init__(self, seqs, heads, hd, page, seed=0, first_row=0, extra_rows=0, n_pages=None, q_heads=None, spare=2):
        g = np.random.default_rng(seed)
        self.g, self.seqs, self.heads, self.hd, self.page = g, seqs, heads, hd, page
        self.q_heads = q_heads or heads
        self.n = np.array([r for r, _ in seqs])
        self.kv_len = np.array([r + c for r, c in seqs], np.int32)
        assert (self.kv_len >= 0).all()
        self.row_start = (first_row + np.concatenate([[0], np.cumsum(self.n)])).astype(np.int32)
        self.rows = int(self.row_start[-1]) + extra_rows
        need = -(-self.kv_len // page)
        n_pages = n_pages or int(need.sum()) + spare
        ids = g.permutation(n_pages)[:int(need.sum())] if n_pages < 10000 else n_pages - 1 - np.arange(need.sum())
        self.n_pages = n_pages
        self.table = np.full((len(seqs), int(need.max()) + 1), -1, np.int32)
        at = 0
        for s, k in enumerate(need):
            self.table[s, :k] = ids[at:at + k]
            at += k

    def positions(self, s):
        return int(self.kv_len[s]) - int(self.n[s]) + np.arange(self.n[s])

    def vectors(self, n):
        """n tokens of keys or values: tokens and channels differ in size."""
        g = self.g
        x = g.standard_normal((n, self.heads, self.hd))
        return x * np.exp(0.5 * g.standard_normal((n, self.heads, 1))) * np.exp(0.5 * g.standard_normal((1, 1, self.hd)))


class Cache:
    """codes and exps as numpy arrays in the library's layout."""

    def __init__(self, c, fill=None):
        shape = (c.n_pages, 2, c.heads, c.page, c.hd)
        self.c = c
        self.codes = np.zeros(shape, np.uint8) if fill is None else fill.integers(0, 256, shape, dtype=np.uint8)
        eshape = (c.n_pages, c.heads, c.page, 2)
        self.exps = np.full(eshape, 127, np.uint8) if fill is None else fill.integers(0, 256, eshape, dtype=np.uint8)

    def put(self, s, pos, k, v):
        """Vectors k, v [heads, hd] at position pos of sequence s."""
        c = self.c
        page, slot = c.table[s, pos // c.page], pos % c.page
        for kv, x in ((0, k), (1, v)):
            codes, e = quantise(x)
            self.exps[page, :, slot, kv] = e
            if kv == 0:
                self.codes[page, 0, :, slot] = codes
            else:
                self.codes[page, 1].reshape(c.heads, c.page // 16, c.hd, 16)[:, slot // 16, :, slot % 16] = codes

    def put_many(self, s, p0, k, v):
        c = self.c
        pos = p0 + np.arange(len(k))
        page, slot = c.table[s, pos // c.page], pos % c.page
        kc, ke = quantise(k)
        vc, ve = quantise(v)
        self.exps[page, :, slot] = np.stack([ke, ve], -1)
        self.codes[page, 0, :, slot] = kc
        plane = self.codes.reshape(c.n_pages, 2, c.heads, c.page // 16, c.hd, 16)
        plane[page, 1, :, slot // 16, :, slot % 16] = vc

    def get(self, s, n):
        """Keys and values (float64 [n, heads, hd]) of sequence s's first n positions."""
        c = self.c
        pos = np.arange(n)
        page, slot = c.table[s, pos // c.page], pos % c.page
        k = dequantise(self.codes[page, 0, :, slot], self.exps[page, :, slot, 0])
        plane = self.codes.reshape(c.n_pages, 2, c.heads, c.page // 16, c.hd, 16)
        v = dequantise(plane[page, 1, :, slot // 16, :, slot % 16], self.exps[page, :, slot, 1])
        return k, v


def attention(c, cache, q, causal=True, window=0, scale=None, hidden=None):
    """(out, lse, bound on out's error, bound on lse's error) for q [rows,
    Hq, hd] in float64; rows of no sequence are NaN.  hidden(s, t): positions
    of unusable pages.

    Bounds, with A = sum p|v| / sum p, n keys, D = scale * max_t sum |q k|:
    scores accumulate hd products in fp32 (hd 2^-24 D, twice that for the two
    roundings of scaling), p is a 2^-22 exponential of them, rounded to f16 at
    worst (2^-11), or below 2^-14 of the format's range to 2^-31 of the row's
    largest term; the sums of n terms add n 2^-24 each; out rounds to bf16 (2^-8)."""
    scale = c.hd ** -0.5 if scale is None else scale
    group = c.q_heads // c.heads
    out = np.full((c.rows, c.q_heads, c.hd), np.nan)
    lse = np.full((c.rows, c.q_heads), np.nan)
    dout, dlse = np.zeros_like(out), np.zeros_like(lse)
    for s in range(len(c.seqs)):
        n = int(c.kv_len[s])
        k, v = cache.get(s, n)
        t = np.arange(n)
        r0 = c.row_start[s]
        for j, p in enumerate(c.positions(s)):
            see = (t <= p) if causal else np.full(n, p >= 0)
            if window:
                see &= t > p - window
            if p < 0:
                see &= False
            if hidden is not None:
                see &= ~hidden(s, t)
            for h in range(c.q_heads):
                if not see.any():
                    out[r0 + j, h], lse[r0 + j, h] = 0.0, -np.inf
                    continue
                kk, vv, qq = k[see, h // group], v[see, h // group], q[r0 + j, h]
                x = scale * (kk @ qq)
                m = x.max()
                e = np.exp(x - m)
                out[r0 + j, h], lse[r0 + j, h] = e @ vv / e.sum(), m + np.log(e.sum())
                D = abs(scale) * (np.abs(kk) @ np.abs(qq)).max()
                ds = 2 * c.hd * 2.0 ** -24 * D + 2.0 ** -24 * np.abs(x).max()
                A = e @ np.abs(vv) / e.sum()
                count = see.sum()
                dout[r0 + j, h] = (2.0 ** -8 * (np.abs(out[r0 + j, h]) + A * 2.0 ** -7) +
                                   A * (2.0 ** -11 + 2 * ds + 2.0 ** -20 + 2 * count * 2.0 ** -24) +
                                   count * 2.0 ** -30 * np.abs(vv).max())
                dlse[r0 + j, h] = ds + 2.0 ** -20 + count * 2.0 ** -24 + 2.0 ** -22 * abs(lse[r0 + j, h])
    return out, lse, dout, dlse
