"""Plain 64-bit implementations of the block-scaled e4m3 cache's operators, in
numpy, written from their definitions: the step's buffers from request
lengths, blocks given back, the quantising append, attention.  Shared by the
CPU tests that pin them and the GPU tests that compare with them."""
import numpy as np

import oracle

BS, D = 16, 128
TOP = 448.0
E4M3 = np.array([oracle.e4m3_decode(c) for c in range(256)], np.float64)  # NaN at 0x7f, 0xff
_ORDER = np.argsort(E4M3[:127])
_GRID = E4M3[:127][_ORDER]  # 0 .. 448, ascending


def cdiv(a, b):
    return -(-a // b)


def encode(x):
    """e4m3 codes of x (float64): nearest, ties to the even code, magnitudes
    past 448 saturated, NaN 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), TOP)
    hi = np.clip(np.searchsorted(_GRID, np.where(np.isnan(a), 0, a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = _GRID[hi] - a < a - _GRID[lo]
    tie = _GRID[hi] - a == a - _GRID[lo]
    pick = np.where(tie, np.where(hi % 2 == 0, hi, lo), np.where(up, hi, lo))
    code = pick.astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def need_scale(top):
    """The smallest power of two s >= 2^-126 with top / s <= 448."""
    s = -126
    while top > TOP * 2.0 ** s:
        s += 1
    return 2.0 ** s


def append(k_new, v_new, table, lens, qsl, pools, scales):
    """k_new, v_new float64 [T, Hkv, 128]; pools = (K, V) uint8 codes, scales
    float32, updated copies returned."""
    pools, scales = [p.copy() for p in pools], [s.copy() for s in scales]
    for r, n in enumerate(lens):
        old = n - (qsl[r + 1] - qsl[r])
        if old == n:
            continue
        for b in range(old // BS, cdiv(n, BS)):
            i, a, z = table[r, b], max(old, b * BS), min(n, b * BS + BS)
            for new, pool, sc in zip((k_new, v_new), pools, scales):
                for h in range(new.shape[1]):
                    x = new[qsl[r] + a - old:qsl[r] + z - old, h]
                    fin = np.abs(x[np.isfinite(x)])
                    s = need_scale(fin.max(initial=0.0))
                    keep = a - b * BS
                    if keep > 0:
                        was = sc[i, h]
                        s = max(float(was), s)
                        # the old scale over the new one, as one fp32 number
                        ratio = np.float32(was) / np.float32(s)
                        if ratio != 1:
                            v = (E4M3[pool[i, h, :keep]].astype(np.float32) * ratio).astype(np.float64)
                            pool[i, h, :keep] = encode(v)
                    with np.errstate(over="ignore", invalid="ignore"):
                        y = (x.astype(np.float32) / np.float32(s)).astype(np.float64)
                    pool[i, h, keep:keep + z - a] = encode(y)
                    sc[i, h] = s
    return pools, scales


def attention(q, pools, scales, table, lens, qsl, scale, min_q=16):
    """q float64 [T, Hq, 128].  Returns (out, bound): the outputs and, element
    by element, how far a computation may be off that rounds what the kernels
    round (see bound's terms below).  Requests with at least min_q query rows
    are taken by the prefill kernel, whose weights are f16."""
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    hq, hkv = q.shape[1], pools[0].shape[1]
    g = hq // hkv
    for r, n in enumerate(lens):
        m = qsl[r + 1] - qsl[r]
        if m == 0:
            continue
        ids = table[r, :cdiv(n, BS)]
        sees = np.arange(n)[None, :] <= np.arange(n - m, n)[:, None]
        for k in range(hkv):
            codes = [E4M3[p[ids, k]].reshape(-1, D)[:n] for p in pools]
            sc = [np.repeat(s[ids, k].astype(np.float64), BS)[:n] for s in scales]
            K, V = codes[0] * sc[0][:, None], codes[1] * sc[1][:, None]
            for h in range(k * g, k * g + g):
                x = q[qsl[r]:qsl[r + 1], h]
                s = np.where(sees, scale * (x @ K.T), -np.inf)
                w = np.exp(s - s.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                o = w @ V
                # Scores: fp32 sums of 128 products and a few fp32 factors,
                # 2^-20 of the sum of magnitudes; a probability is off by as
                # much, relative, and so is the normaliser.  exp2 of an
                # argument of size |s| carries |s| 2^-23.
                mag = np.where(sees, abs(scale) * (np.abs(x) @ np.abs(K).T), 0).max(1, keepdims=True)
                ds = 2 * mag * (2.0 ** -20 + 2.0 ** -22)
                # q, scaled so that its largest element lies in [128, 256), is
                # a pair of e4m3 numbers: exact where the lowest of its eight
                # bits is at least e4m3's smallest, 2^-9 (elements from 2^-2
                # on, scaled), and off by at most half of that below.
                top = np.abs(x).max(1, keepdims=True)
                unit = 2.0 ** (np.floor(np.log2(np.where(top > 0, top, 1))) - 7)
                small = (np.abs(x) < unit / 4) * (x != 0) * unit * 2.0 ** -10
                ds = ds + 2 * np.where(sees, abs(scale) * (small @ np.abs(K).T), 0).max(1, keepdims=True)
                # A weight is a pair of e4m3 numbers: rounded by at most 2^-9,
                # or by at most 2^-18 of the largest weight times value scale.
                # The prefill kernel rounds it to f16: 2^-11.
                rounded = 2.0 ** -11 if m >= min_q else 2.0 ** -9
                floor = 2.0 ** -18 * (w * sc[1][None]).max(1, keepdims=True) * \
                    (np.where(sees, 1.0, 0.0) @ np.abs(codes[1]))
                mean = w @ np.abs(V)
                out[qsl[r]:qsl[r + 1], h] = o
                # and the output is bf16, half a step 2^-8
                bound[qsl[r]:qsl[r + 1], h] = 2.0 ** -8 * np.abs(o) + \
                    (rounded + ds + 2.0 ** -16) * (1 + 2.0 ** -7) * mean + floor + 1e-37
    return out, bound


def build(prev, new, free_list, num_free, table, cap):
    """(table, lens, qsl, slots, free left, refused)."""
    table = table.copy()
    lens, qsl, slots, refused = [], [0], [], 0
    limit, stop = table.shape[1] * BS, False
    blocks = tokens = 0  # of the valid requests so far, served or not
    left = num_free
    for r, (p, n) in enumerate(zip(prev, new)):
        if p < 0 or n < 0 or p + n > limit:
            lens.append(0)
            refused += 1
        else:
            blocks += cdiv(p + n, BS) - cdiv(p, BS)
            tokens += n
            stop = stop or (n > 0 and (blocks > num_free or tokens > cap))
            if n > 0 and stop:
                lens.append(p)
                refused += 1
            else:
                lens.append(p + n)
                for b in range(cdiv(p, BS), cdiv(p + n, BS)):
                    left -= 1
                    table[r, b] = free_list[left]
                slots += [int(table[r, x // BS]) * BS + x % BS for x in range(p, p + n)]
        qsl.append(len(slots))
    slots += [-1] * (cap - len(slots))
    return table, np.array(lens), np.array(qsl), np.array(slots, np.int64), left, refused


def release(table, lens, keep, free_list, num_free):
    """(free list, number of free blocks)."""
    free_list, n = free_list.copy(), num_free
    for r, (a, b) in enumerate(zip(keep, lens)):
        if 0 <= a <= b <= table.shape[1] * BS:
            for i in table[r, cdiv(a, BS):cdiv(b, BS)]:
                if 0 <= i < len(free_list) and n < len(free_list):
                    free_list[n] = i
                    n += 1
    return free_list, n
