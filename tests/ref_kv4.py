"""The 4-bit key/value cache in NumPy float64, from its definition (no code shared with the library)."""
import numpy as np

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """Value of each E4M3 byte (bias 7, subnormals, no infinities, 0x7F and 0xFF are NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


E4M3 = e4m3_values()


def nearest(x, table):
    """Index of the entry of an ascending table nearest to each x >= 0, ties to the even index, saturating."""
    up = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo, hi = x - table[up - 1], table[up] - x
    return np.where((lo < hi) | ((lo == hi) & (up % 2 == 1)), up - 1, up)


def quantise(x, t):
    """codes [..., d / 2] and scales [..., d / 16] (uint8) of x [..., d] (float32 or float64 values of bf16)."""
    f32 = np.float32
    y = np.asarray(x, f32) / f32(t)
    g = y.reshape(y.shape[:-1] + (-1, 16))
    a = np.abs(g).max(-1)
    s8 = nearest(np.minimum((a / f32(6)).astype(np.float64), 448.0), E4M3[:127]).astype(np.uint8)
    s = E4M3[s8].astype(f32)[..., None]
    q = np.abs(g) / np.where(s > 0, s, f32(1))
    c = np.where(s > 0, nearest(q.astype(np.float64), MAGS) + 8 * np.signbit(g), 0).astype(np.uint8)
    c = c.reshape(y.shape)
    return c[..., 0::2] | (c[..., 1::2] << 4), s8


def values(codes, scales, t):
    """float64 values [..., d]."""
    lut = np.concatenate([MAGS, -MAGS])
    c = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],))
    c[..., 0::2] = lut[codes & 15]
    c[..., 1::2] = lut[codes >> 4]
    return c * np.repeat(E4M3[scales], 16, -1) * float(np.float32(t))


def attend(q, K, V):
    """q [G, d], K, V [n, d] -> out [G, d], lse [G], p [G, n], and sum_j p_j |V_j| and the largest
    sum_d |q_d K_d| / sqrt(d) that the tolerances are made of. n = 0: zeros, -inf."""
    G, d = q.shape
    if K.shape[0] == 0:
        z = np.zeros((G, d))
        return z, np.full(G, -np.inf), np.zeros((G, 0)), z, 0.0
    x = q @ K.T / np.sqrt(d)
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m)
    p = e / e.sum(-1, keepdims=True)
    size = float((np.abs(q) @ np.abs(K).T).max() / np.sqrt(d))
    return p @ V, (np.log(e.sum(-1, keepdims=True)) + m)[:, 0], p, p @ np.abs(V), size


def keep_positions(w, n, keep, recent, first):
    """Ascending positions of n tokens that stay (w [>= n] float32)."""
    j = np.arange(n)
    if n <= keep:
        return j
    mid = j[first:n - recent]
    best = mid[np.lexsort((mid, -w[mid].astype(np.float64)))][:keep - recent - first]
    return np.sort(np.concatenate([j[:first], best, j[n - recent:]]))
