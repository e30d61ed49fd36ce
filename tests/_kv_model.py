"""The 8-bit cache, attention over it and gradient clipping in NumPy doubles,
written from the definitions of include/mlora_kv.h and include/mlora.h: one
sequence, one head, one page at a time.  Test infrastructure only."""
import numpy as np

PAGE = 64
MIN_EXP = -100


def byte_k(j, c, hd):
    s = 4 * (j % 2) if hd == 128 else 0
    return j * hd + ((c // 16) ^ s) * 16 + c % 16


def byte_v(j, c, hd):
    return (j // 4) * 4 * hd + ((c // 4) ^ (2 * (j // 4 % 4))) * 16 + 4 * (c % 4) + j % 4


_MAPS = {}


def maps(hd):
    """byte offset of (token, dim): [64, hd] for keys and for values"""
    if hd not in _MAPS:
        j, c = np.meshgrid(np.arange(PAGE), np.arange(hd), indexing="ij")
        _MAPS[hd] = (byte_k(j, c, hd), byte_v(j, c, hd))
    return _MAPS[hd]


def e4m3_value(b):
    b = np.asarray(b, dtype=np.uint8)
    s = np.where(b & 0x80, -1.0, 1.0)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7))
    return np.where((b & 0x7f) == 0x7f, np.nan, s * v)


_TABLE = e4m3_value(np.arange(127, dtype=np.uint8))       # 0 .. 448, ascending


def e4m3_byte(x):
    """Magnitudes <= 448 (or not finite -> NaN) to the nearest byte, ties to the even one."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    a = np.where(ok, np.abs(x), 0.0)
    assert (a <= 448).all()
    hi = np.clip(np.searchsorted(_TABLE, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _TABLE[lo], _TABLE[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    out = pick.astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(ok, out, 0x7f).astype(np.uint8)


def need_exp(x):
    a = np.abs(x[np.isfinite(x)]).max() if np.isfinite(x).any() else 0.0
    if a == 0:
        return MIN_EXP
    e = int(np.floor(np.log2(a / 448))) - 1
    while a > 448 * 2.0 ** e:
        e += 1
    return max(e, MIN_EXP)


class Cache:
    """Logical state: bytes [n_pages, n_kv, 64, hd] in (token, dim) order and exponents."""

    def __init__(self, n_pages, n_kv, hd):
        self.hd = hd
        self.b = {x: np.zeros((n_pages, n_kv, PAGE, hd), np.uint8) for x in "kv"}
        self.e = {x: np.zeros((n_pages, n_kv), np.int64) for x in "kv"}

    def append(self, table, start, rows):
        """rows: {"k": [n, n_kv, hd], "v": ..} at positions start.. of the sequence with these pages"""
        for x, r in rows.items():
            n = len(r)
            for p in range(start // PAGE, -(-(start + n) // PAGE)):
                a, b = max(start - p * PAGE, 0), min(start + n - p * PAGE, PAGE)
                new = np.asarray(r[p * PAGE + a - start:p * PAGE + b - start], dtype=np.float64)
                page = table[p]
                for h in range(r.shape[1]):
                    e = need_exp(new[:, h])
                    if a > 0:
                        old = self.e[x][page, h]
                        e = max(e, old)
                        if e > old:
                            v = e4m3_value(self.b[x][page, h, :a]) * 2.0 ** (old - e)
                            self.b[x][page, h, :a] = np.where(np.isnan(v), 0x7f, e4m3_byte(v))
                    self.e[x][page, h] = e
                    self.b[x][page, h, a:b] = e4m3_byte(new[:, h] * 2.0 ** -e)

    def values(self, x, table, n):
        """[n, n_kv, hd] doubles of positions 0 .. n-1"""
        out = [e4m3_value(self.b[x][p]) * 2.0 ** self.e[x][p][:, None, None].astype(np.float64)
               for p in table[:-(-n // PAGE)]]
        if not out:
            return np.zeros((0, self.b[x].shape[1], self.hd))
        return np.concatenate([o.transpose(1, 0, 2) for o in out])[:n]

    def pages(self, x):
        """the bytes in page order, as the library holds them"""
        n, kv = self.b[x].shape[:2]
        out = np.zeros((n, kv, PAGE * self.hd), np.uint8)
        out[:, :, maps(self.hd)[0 if x == "k" else 1].reshape(-1)] = self.b[x].reshape(n, kv, -1)
        return out.reshape(n, kv, PAGE, self.hd)


def attention(q, k, v, first, scale):
    """q [n, heads, hd] at positions first.. over k, v [len, n_kv, hd].  Returns
    (out, lse, sum_i p_i |v_i|, the largest sum_d |q_d k_d| of a row)."""
    n, heads, hd = q.shape
    group = heads // k.shape[1]
    out, lse = np.zeros(q.shape), np.full((n, heads), -np.inf)
    mass, big = np.zeros(q.shape), np.zeros((n, heads))
    for i in range(n):
        for h in range(heads):
            kk, vv = k[:first + i + 1, h // group], v[:first + i + 1, h // group]
            if not len(kk):
                continue
            s = kk @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            lse[i, h] = m + np.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ vv
            mass[i, h] = p @ np.abs(vv)
            big[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, mass, big
