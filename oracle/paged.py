"""Plain fp64 forms of the operators around a paged key/value cache: E4M3 rows
with power-of-two scales, pages, attention of new tokens over them, rotary
positions.  Numpy only; shares no code with the library."""

import numpy as np

E4M3_MAX = 448.0
E_MIN, E_MAX = -110, 119


def e4m3_grid():
    """The non-negative finite E4M3 values, by code 0 .. 126."""
    v = []
    for code in range(127):
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


_GRID = e4m3_grid()


def e4m3_codes(y):
    """Codes (uint8) of values y, |y| <= 448: nearest, ties to the even code."""
    a = np.abs(y)
    hi = np.clip(np.searchsorted(_GRID, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = _GRID[hi] - a
    down = a - _GRID[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def e4m3_values(codes):
    """Values of codes; the two NaN codes give NaN."""
    full = np.concatenate([_GRID, [np.nan]])
    c = codes.astype(np.int64)
    return np.where(c >= 128, -1.0, 1.0) * full[c & 127]


def quantise(x):
    """(codes, scale bytes) of rows x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    amax = np.max(np.abs(x), axis=-1)
    bad = ~np.isfinite(amax)
    e = np.full(amax.shape, E_MIN, dtype=np.int64)
    it = np.nditer(np.where(bad, 0.0, amax), flags=["multi_index"])
    for a in it:
        k = E_MIN
        if a > 0:
            k = max(E_MIN, int(np.frexp(float(a))[1]) - 12)
            while k < E_MAX and float(a) > E4M3_MAX * 2.0 ** k:
                k += 1
        e[it.multi_index] = k
    y = np.clip(np.where(bad[..., None], 0.0, x) * 2.0 ** -e[..., None].astype(np.float64), -E4M3_MAX, E4M3_MAX)
    codes = np.where(bad[..., None], 0, e4m3_codes(y)).astype(np.uint8)
    return codes, np.where(bad, 255, e + 127).astype(np.uint8)


def dequantise(codes, scale):
    f = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127.0))
    return e4m3_values(codes) * f[..., None]


def slot_of(block_table, page_size, b, pos):
    return int(block_table[b, pos // page_size]), pos % page_size


def gather(pages, block_table, b, length):
    """Rows [length, Hkv, D] (or [length, Hkv] for scales) of sequence b."""
    P = pages.shape[2]
    if length == 0:
        return np.zeros((0, pages.shape[1]) + pages.shape[3:], dtype=pages.dtype)
    return np.stack([pages[int(block_table[b, t // P]), :, t % P] for t in range(length)])


def attention(q, k, v, causal, scale):
    """One sequence: q [n, Hq, D], k and v [L, Hkv, D].  Returns (o, lse [Hq, n],
    a), a = sum of |weight| |value| / sum of weights, for tolerances."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    o, a = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse = np.full((Hq, n), -np.inf)
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // Hkv)], v[:, h // (Hq // Hkv)]
        for i in range(n):
            end = min(L, max(0, L - n + i + 1)) if causal else L
            if end == 0:
                continue
            s = kh[:end] @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            o[i, h] = p @ vh[:end] / p.sum()
            a[i, h] = p @ np.abs(vh[:end]) / p.sum()
            lse[h, i] = m + np.log(p.sum())
    return o, lse, a


def rope(x, positions, sections, base, restart=False, interleaved=False, inverse=False):
    """x [T, H, D], positions [axes, T]."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    R = int(sum(sections))
    i = 0
    for a, m in enumerate(sections):
        for j in range(m):
            f = float(base) ** (-(j / m if restart else i / R))
            ang = positions[a].astype(np.float64) * f * (-1.0 if inverse else 1.0)
            c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
            p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + R)
            y[..., p] = x[..., p] * c - x[..., q] * s
            y[..., q] = x[..., q] * c + x[..., p] * s
            i += 1
    return y


# ------------------------------------------- drafted trees, sums, eviction --

def tree_ancestors(parents):
    """[n, n] truth values, token i's own and its ancestors', and the depths."""
    n = len(parents)
    sees = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            sees[i, j] = True
            j = int(parents[j])
    return sees, sees.sum(1) - 1


def pack_bits(sees, words):
    """Rows of truth values as int32 words of 32."""
    n, m = sees.shape
    out = np.zeros((n, words), dtype=np.uint32)
    for j in range(m):
        out[:, j // 32] |= sees[:, j].astype(np.uint32) << np.uint32(j % 32)
    return out.view(np.int32)


def tree_sees(bits, L):
    """[n, L]: which keys a sequence's n drafted tokens see, by their masks' truth values [n, >= n]."""
    n = bits.shape[0]
    sees = np.zeros((n, L), dtype=bool)
    past = L - n
    for i in range(n):
        if past + i < 0:                # padded
            continue
        sees[i, :max(0, past)] = True
        for j in range(n):
            if past + j >= 0:
                sees[i, past + j] = bits[i, j]
    return sees


def causal_sees(n, L, causal):
    """[n, L]: which keys the last n tokens of a sequence of L see."""
    i, j = np.arange(n)[:, None], np.arange(L)[None, :]
    return (j <= L - n + i) if causal else np.ones((n, L), dtype=bool)


def attention_of(q, k, v, sees, scale):
    """attention() with a mask [n, L] of truth values."""
    n, Hq, D = q.shape
    o, a = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse = np.full((Hq, n), -np.inf)
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // k.shape[1])], v[:, h // (Hq // v.shape[1])]
        for i in range(n):
            if not sees[i].any():
                continue
            s = kh[sees[i]] @ q[i, h] * scale
            p = np.exp(s - s.max())
            o[i, h] = p @ vh[sees[i]] / p.sum()
            a[i, h] = p @ np.abs(vh[sees[i]]) / p.sum()
            lse[h, i] = s.max() + np.log(p.sum())
    return o, lse, a


def select(sums, keep, first, recent):
    """Ascending tokens that stay of one head's sums [L]."""
    L = len(sums)
    if L <= keep:
        return np.arange(L)
    x = np.where(np.isnan(sums), np.inf, sums.astype(np.float64))
    above = np.isnan(sums).astype(int)                  # a NaN is above an infinity
    at = np.arange(L)
    above[(at < first) | (at >= L - recent)] = 2
    order = np.lexsort((at, -x, -above))                # by class, then by size, then the lowest token
    return np.sort(order[:keep])


def weights(q, lse, k, sees, scale):
    """What one sequence's keys get: q [n, Hq, D], lse [Hq, n], k [L, Hkv, D], mask
    [n, L].  Returns ([Hkv, L], the same with each weight times its |score - lse|)."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    out, slack = np.zeros((Hkv, L)), np.zeros((Hkv, L))
    for h in range(Hq):
        x = q[:, h] @ k[:, h // (Hq // Hkv)].T * scale
        for i in range(n):
            if np.isneginf(lse[h, i]):
                continue
            d = np.where(sees[i], x[i] - lse[h, i], -np.inf)
            w = np.exp(d)
            out[h // (Hq // Hkv)] += w
            slack[h // (Hq // Hkv)] += np.where(w > 0, w * np.abs(np.where(sees[i], d, 0.0)), 0.0)
    return out, slack
