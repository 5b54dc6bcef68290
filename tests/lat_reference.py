"""Plain 64-bit implementations, in numpy, of the norm and rotation ahead of the
append and of the latent cache's operators, written from their definitions, with
the bounds that their tests hold the kernels to."""
import numpy as np

BS, LAT, ROPE, ROW = 16, 512, 64, 576
NOPE, VAL = 128, 128


def cdiv(a, b):
    return -(-a // b)


def table(n, rot, base=10000.0):
    """cos | sin of n positions, fp32."""
    a = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def norm(x, w, eps):
    """x [..., n] over its last dim."""
    with np.errstate(over="ignore", invalid="ignore"):
        return w * x / np.sqrt(np.square(x).mean(-1, keepdims=True) + eps)


def rotate(x, cs, inter):
    """x [tokens, heads, d], cs [tokens, rot].  Returns (y, size): the rotated
    vectors and, dim by dim, the sum of the magnitudes that were added."""
    cs = cs.astype(np.float64)
    half = cs.shape[1] // 2
    y, size = x.copy(), np.abs(x)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
    c, s = cs[:, None, :half], cs[:, None, half:]
    with np.errstate(invalid="ignore"):
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        size[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        size[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, size


def turned_bound(y, size):
    """fp32 arithmetic of a norm (a sum of up to 512 squares by a tree, a square
    root, a division: well within 2^-19) and of a rotation (2^-22), relative to the
    magnitudes added, then the rounding to bf16, half a step: 2^-8."""
    return 2.0 ** -8 * np.abs(y) + 2.0 ** -18 * size + 1e-38


def softmax_rows(s):
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.exp(s - s.max(1, keepdims=True))
        return w / w.sum(1, keepdims=True)


def _attend(x, k, v, scale, sees):
    """One head: rows x over keys k and values v; and the bound of a computation
    whose scores and sums are fp32 and whose weights are bf16."""
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.where(sees, scale * (x @ k.T), -np.inf)
        w = softmax_rows(s)
        o = w @ v
        # Scores: fp32 sums of up to 576 products, 2^-20 of the sum of
        # magnitudes (as the other attention tests take it), and exp2 of an
        # argument of that size carries 2^-23 of it; the weight and the
        # normaliser are off by as much, relative.
        mag = np.where(sees, abs(scale) * (np.abs(x) @ np.abs(k).T), 0).max(1, keepdims=True)
        ds = 2 * mag * (2.0 ** -20 + 2.0 ** -22)
        mean = w @ np.abs(v)
        # Weights rounded by at most 2^-8 each, in the product and in the sum:
        # first order sum w d (v - o); fp32 sums 2^-16; and the output's own
        # rounding, 2^-8.
        return o, 2.0 ** -8 * np.abs(o) + (2.0 ** -8 * (mean + np.abs(o)) + (ds + 2.0 ** -16) * mean) * \
            (1 + 2.0 ** -6) + 1e-37


def absorbed(q, pool, tab, lens, qsl, scale):
    """q float64 [T, H, 576], pool float64 [blocks, 16, 576]: (out, bound) [T, H, 512].
    A key that a row does not see is no part of its sum, whatever it holds."""
    T, H = q.shape[:2]
    out, bound = np.zeros((T, H, LAT)), np.zeros((T, H, LAT))
    for r, n in enumerate(lens):
        m = qsl[r + 1] - qsl[r]
        c = pool[tab[r, :cdiv(n, BS)]].reshape(-1, ROW)
        for i in range(m):
            t, p = qsl[r] + i, n - m + i + 1
            o, b = _attend(q[t], c[:p], c[:p, :LAT], scale, np.ones((H, p), bool))
            out[t], bound[t] = o, b
    return out, bound


def expand(pool, w, tab, lens):
    """pool float64, w float64 [H, 256, 512]: (kv, k_rope, bound of kv)."""
    c = np.concatenate([pool[tab[r, :cdiv(n, BS)]].reshape(-1, ROW)[:n] for r, n in enumerate(lens)])
    kv = np.einsum("jc,hoc->jho", c[:, :LAT], w, optimize=True)
    size = np.einsum("jc,hoc->jho", np.abs(c[:, :LAT]), np.abs(w), optimize=True)
    # fp32 sums of 512 products, 2^-20 of the magnitudes, and the rounding
    return kv, c[:, LAT:], 2.0 ** -8 * np.abs(kv) + 2.0 ** -19 * size


def expanded(q, kv, k_rope, lens, qsl, scale):
    """q float64 [T, H, 192], kv [rows, H, 256], k_rope [rows, 64]: (out, bound) [T, H, 128]."""
    T, H = q.shape[:2]
    out, bound = np.zeros((T, H, VAL)), np.zeros((T, H, VAL))
    k0 = 0
    for r, n in enumerate(lens):
        m = qsl[r + 1] - qsl[r]
        for h in range(H if m > 0 else 0):
            x = q[qsl[r]:qsl[r + 1], h]
            k = np.concatenate([kv[k0:k0 + n, h, :NOPE], k_rope[k0:k0 + n]], 1)
            v = kv[k0:k0 + n, h, NOPE:]
            if np.isfinite(k).all() and np.isfinite(v).all():
                sees = np.arange(n)[None, :] <= np.arange(n - m, n)[:, None]
                out[qsl[r]:qsl[r + 1], h], bound[qsl[r]:qsl[r + 1], h] = _attend(x, k, v, scale, sees)
            else:  # row by row, over the keys that it sees
                for i in range(m):
                    p = n - m + i + 1
                    o, b = _attend(x[i:i + 1], k[:p], v[:p], scale, np.ones((1, p), bool))
                    out[qsl[r] + i, h], bound[qsl[r] + i, h] = o[0], b[0]
        k0 += n
    return out, bound
