"""Plain float64 restatement (numpy, loops) of the block-scaled 8-bit cache and of the norm + rotation, for the tests.
It shares no code with the library. A cache is, for each (b, h), the list of its positions, expire values and, page by
page, integer-valued codes and the two scales."""
import math

import numpy as np

E4M3, INT8 = 0, 1
LARGEST = {E4M3: 448.0, INT8: 127.0}
NEVER = 2**31 - 1
PAGE = 16


def widen(bits):
    """bf16 bit patterns (uint16) as float64."""
    return (np.asarray(bits, np.uint32) << 16).view(np.float32).astype(np.float64)


def _e4m3_table():
    """The numbers of the 256 E4M3 bytes (NaN at 0x7F, 0xFF)."""
    out = np.empty(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v = math.ldexp(1 + f / 8, e - 7) if e else math.ldexp(f / 8, -6)
        out[b] = math.nan if (b & 127) == 127 else (-v if b & 128 else v)
    return out


TABLE = {E4M3: _e4m3_table(), INT8: np.array([b if b < 128 else b - 256 for b in range(256)], float)}


def scale_of(x, fmt):
    """Scale of a set of values: from the largest finite magnitude."""
    x = np.abs(np.asarray(x, float)).ravel()
    x = x[np.isfinite(x)]
    a = x.max() if x.size else 0.0
    if a == 0:
        return 0.0
    e = -126
    while a > LARGEST[fmt] * math.ldexp(1.0, e):
        e += 1
    return math.ldexp(1.0, e)


def encode(x, scale, fmt):
    """Bytes of x / scale, to nearest even, saturating; NaN -> 0x7F or 0xFF of E4M3, 0 of int8."""
    x = np.asarray(x, float)
    y = x / scale if scale else x     # scale 0: the finite values are all zeros
    if fmt == INT8:
        return np.rint(np.clip(np.nan_to_num(y, nan=0.0, posinf=127, neginf=-127), -127, 127)).astype(np.int8).view(np.uint8)
    mag = TABLE[E4M3][:127]                                  # 0 .. 448, ascending, index = code
    a = np.minimum(np.abs(np.nan_to_num(y, nan=0.0, posinf=448, neginf=-448)), 448.0)
    hi = np.clip(np.searchsorted(mag, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - mag[lo], mag[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = np.where(mag[hi] == a, hi, code).astype(np.uint8)
    code |= np.where(np.signbit(y), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(y), 0x7F, code).astype(np.uint8)


def decode(codes, fmt):
    return TABLE[fmt][np.asarray(codes, np.uint8)]


class Head:
    """One (b, h)'s rows."""

    def __init__(self, d, fmt):
        self.d, self.fmt = d, fmt
        self.codes = [np.zeros((0, d), np.uint8), np.zeros((0, d), np.uint8)]   # K, V
        self.scales = [[], []]                                                  # per page
        self.expire, self.pos = [], []

    @property
    def count(self):
        return len(self.pos)

    def fill(self, k, v, expire, pos):
        """All rows at once, quantised page by page."""
        for w, x in ((0, k), (1, v)):
            out = []
            for p in range(0, len(x), PAGE):
                s = scale_of(x[p:p + PAGE], self.fmt)
                self.scales[w].append(s)
                out.append(encode(x[p:p + PAGE], s, self.fmt))
            self.codes[w] = np.concatenate(out) if out else self.codes[w]
        self.expire, self.pos = list(expire), list(pos)

    def append(self, k, v, expire, pos):
        r = self.count % PAGE
        for w, x in ((0, k), (1, v)):
            if r == 0:
                self.scales[w].append(0.0)
            old = self.scales[w][-1]
            new = max(old, scale_of(x, self.fmt))
            if r and new > old:
                rows = decode(self.codes[w][-r:], self.fmt) * (old / new)
                self.codes[w][-r:] = encode(rows, 1.0, self.fmt)
            self.scales[w][-1] = new
            self.codes[w] = np.concatenate([self.codes[w], encode(x, new, self.fmt)[None]])
        self.expire.append(expire)
        self.pos.append(pos)

    def values(self, w):
        s = np.repeat(np.array(self.scales[w]), PAGE)[:self.count, None]
        return decode(self.codes[w], self.fmt) * s

    def attend(self, q, now, scale):
        """(out, lse, (sum of p |v|, sum of |v|), largest sum of |q k|) for the rows of q [G, d]."""
        on = np.array([e > now for e in self.expire], bool)
        g, d = q.shape
        if not on.any():
            return np.zeros((g, d)), np.full(g, -np.inf), (np.zeros((g, d)), np.zeros((g, d))), np.zeros(g)
        k, v = self.values(0)[on], self.values(1)[on]
        x = scale * (q @ k.T)
        top = x.max(1, keepdims=True)
        p = np.exp(x - top)
        l = p.sum(1, keepdims=True)
        size = scale * (np.abs(q) @ np.abs(k).T).max(1)
        return (p / l) @ v, (top + np.log(l))[:, 0], ((p / l) @ np.abs(v), np.broadcast_to(np.abs(v).sum(0), (g, d))), size


def expire_of(mode, t, window, delay, score=None, tau=None, flag=None):
    """mode 0: KVzap, 1: DMS; float32 comparison as given."""
    if mode == 0:
        return NEVER if score >= tau else t + window
    return NEVER if flag < 0 else max(int(flag) + delay, t + window)


def compact(fmt, mode, k, v, now, window, delay, scores=None, tau=None, flag=None):
    """k, v float64 [B, T, H, d] -> Head[b][h]."""
    B, T, H, d = k.shape
    out = []
    for b in range(B):
        row = []
        for h in range(H):
            e = [expire_of(mode, t, window, delay, None if scores is None else scores[b, t, h],
                           None if tau is None else tau[b, h], None if flag is None else flag[b, h, t]) for t in range(T)]
            at = [t for t in range(T) if e[t] > now]
            head = Head(d, fmt)
            head.fill(k[b, at, h], v[b, at, h], [e[t] for t in at], at)
            row.append(head)
        out.append(row)
    return out


def attention_bounds(d, n, out_abs, size):
    """How far an fp32 computation of the attention may be off, element by element.

    A logit in base 2 is a sum of d products, accumulated in fp32 by at most 2^-23 (a step of truncation) of the sum
    of magnitudes S at each addition, times factors that round once each: at most (d + 8) 2^-23 S. Its difference
    from the reference and 2^x (ex2: 2 steps) add 2^-22 each relative to |x|, |x| <= 2 S log2 e. So a weight is off by a
    factor 1 + eps with eps <= (d + 16) 2^-22 S + 2^-20 (with the fp16 pair's 2^-22). The normalised output is off by
    at most 2 eps sum(p |v|), and the sums over n tokens add at most (n / 16 + 200) 2^-23 of sum(p |v|): one addition
    a page, the page's own, the merges'. The fp16 pair of a small weight ends at fp16's smallest step, 2^-24, so it is off
    by up to 2^-25 where a row's largest weight is at least 2^12: 2^-37 of |v| for each token. The log-sum-exp is off by eps (absolute) plus its fp32 steps."""
    eps = (d + 16) * 2.0**-22 * size + 2.0**-20
    weighted, plain = out_abs
    return (2 * eps[:, None] + (n / 16 + 200) * 2.0**-23) * weighted + 2.0**-37 * plain + 1e-37, eps + 2.0**-20


def rotate(x, weight, eps, pos, inv_freq, interleaved):
    """x [n, H, d] float64, inv_freq (exact radians) of length rot / 2."""
    y = np.array(x, float)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    half = len(inv_freq)
    if half:
        turn = np.array([[math.fmod(float(f) / (2 * math.pi) * int(p), 1.0) for f in inv_freq] for p in pos])
        c, s = np.cos(2 * math.pi * turn)[:, None], np.sin(2 * math.pi * turn)[:, None]
        first = np.arange(half) * 2 if interleaved else np.arange(half)
        second = first + (1 if interleaved else half)
        a, b = y[..., first].copy(), y[..., second].copy()
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y
