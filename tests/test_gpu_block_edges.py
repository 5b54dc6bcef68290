"""Attention over the block-scaled e4m3 cache on the rows that a number format
or a mask can spoil: one heavy key beside a long tail of light ones, NaN in
keys that a row must not see."""
import numpy as np
import pytest
import torch

import paged_kv_cache_195_gb300 as pkv

import blk_reference as ref
from test_gpu_block import Cache, _attend, _built, _rows  # noqa: F401  (_built: the module's fixture)

pytestmark = pytest.mark.gpu
BS = 16


def _plain(c, q, rows, scale, exp2_off=2.0 ** -16, ends=2.0 ** -33):
    """Outputs in 64 bits and, element by element, how far a computation may
    be off that holds scores and sums in 32 bits and a weight in f16's eleven
    bits: half a bf16 step of the output (2^-8), of the weighted mean of |V|
    the f16 half step (2^-11) and the scores' error (an fp32 sum of 128
    products, 2^-20 of their magnitudes, twice: in the weight and in the
    normaliser; as much for q's elements below 2^-13 of the largest's
    binade, which the two 8-bit numbers hold to 2^-20 of that; exp2_off for
    exp2 of the scores, 2^-16 where they are below 2^7), and for each weight
    `ends` of the largest (times value scale), where its format does: 2^-33 in
    the decode, 2^-31 in the prefill.  Third, the norm of a row's offsets that
    these ends alone give when they are independent of each other."""
    out, bound, tail = np.zeros(rows.shape), np.zeros(rows.shape), np.zeros(rows.shape[:2])
    hkv = c.pools[0].shape[1]
    g, t = rows.shape[1] // hkv, 0
    for r, (n, m) in enumerate(zip(c.lens, q)):
        if m == 0:
            continue
        ids = c.table[r, :-(-n // BS)]
        sees = np.arange(n)[None] <= np.arange(n - m, n)[:, None]
        for k in range(hkv):
            K, V = (ref.E4M3[p[ids, k]].reshape(-1, 128)[:n] for p in c.pools)
            ks, vs = (np.repeat(s[ids, k].astype(np.float64), BS)[:n] for s in c.scales)
            for h in range(k * g, k * g + g):
                x = rows[t:t + m, h]
                s = np.where(sees, scale * (x @ (K * ks[:, None]).T), -np.inf)
                w = np.exp(s - s.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                o = np.where(w > 0, w, 0) @ (V * vs[:, None])
                mag = np.where(sees, abs(scale) * (np.abs(x) @ np.abs(K * ks[:, None]).T), 0).max(1, keepdims=True)
                unit = 2.0 ** np.floor(np.log2(np.maximum(np.abs(x).max(1, keepdims=True), 2.0 ** -100)))
                fine = np.where(np.abs(x) < unit * 2.0 ** -13, unit, 0) @ np.abs(K * ks[:, None]).T
                ds = mag * 2.0 ** -20 + abs(scale) * np.where(sees, fine, 0).max(1, keepdims=True) * 2.0 ** -20
                floor = ends * (w * vs).max(1, keepdims=True) * (sees @ np.abs(V))
                tail[t:t + m, h] = ends * (w * vs).max(1) * np.sqrt(sees @ (V * V).sum(1))
                out[t:t + m, h] = o
                bound[t:t + m, h] = 2.0 ** -8 * np.abs(o) + floor + \
                    (2.0 ** -11 + 2 * ds + exp2_off) * (1 + 2.0 ** -7) * (w @ np.abs(V * vs[:, None]))
        t += m
    return out, bound, tail


def _sinks(rng, n, m, g, hkv, at, shares):
    """One request of n keys whose last m tokens attend: the key at position
    `at` has value 0 and takes the head's share of the weight, the other keys'
    scores are normal.  (Dim 0 of K is the heavy key's alone, so q's dim 0
    sets its score.)"""
    c = Cache(rng, [n], hkv, spread=0.0)
    ids = c.table[0]
    K = c.pools[0][ids].transpose(1, 0, 2, 3).reshape(hkv, -1, 128)
    K[:, :, 0], K[:, at] = 0, 0
    K[:, at, 0] = ref.encode(np.array([448.0]))[0]
    c.pools[0][ids] = K.reshape(hkv, -1, BS, 128).transpose(1, 0, 2, 3)
    c.pools[1][ids[at // BS], :, at % BS] = 0
    scale = 0.09
    rows = _rows(rng, m, g * hkv).double().numpy()
    rows[:, :, 0] = 0
    for h in range(g * hkv):
        s = scale * rows[:, h] @ (ref.E4M3[K[h // g, :n - m + 1]] * 2.0 ** -7).T
        share = shares[h % len(shares)]
        rows[:, h, 0] = np.log(share / (1 - share) * np.exp(s).sum(1)) / (scale * 448 * 2.0 ** -7)
    return c, torch.tensor(rows).bfloat16(), scale


def _check_tight(c, q, rows, scale, norm=True, **kw):
    got = _attend(c, q, rows, scale)
    torch.cuda.synchronize()
    assert pkv.pkv_get_device_error() == 0, pkv.pkv_last_error()
    want, bound, tail = _plain(c, q, rows.double().numpy(), scale, **kw)
    got = got.double().cpu().numpy()
    off = np.abs(got - want)
    assert (off <= bound).all(), ((off / bound).max(), np.unravel_index((off / bound).argmax(), off.shape))
    if norm:  # independent roundings: the output's 2^-8, the weights' below it
        rel = (np.linalg.norm(got - want, axis=2) - tail) / np.linalg.norm(want, axis=2)
        assert rel.max() <= 2.0 ** -8 + 2.0 ** -9, rel


@pytest.mark.parametrize("g", [1, 4, 5, 6, 8])
@pytest.mark.parametrize("n,at", [(512, 0), (4096, 0), (4096, 4000), (32768, 0), (32768, 20000), (131072, 5)])
def test_attention_one_heavy_key_beside_a_long_tail(n, at, g, pkv_opts):
    # On one CTA, so that the heavy key and the tail share their references.
    rng = np.random.default_rng(n + at + g)
    c, rows, scale = _sinks(rng, n, 1, g, 1, at, [0.9, 0.97, 0.5, 0.8, 0.999])
    pkv_opts(decode_grid=1)
    _check_tight(c, [1], rows, scale)


@pytest.mark.parametrize("n,m,g", [(131072, 8, 4), (131072, 9, 1), (32768, 20, 6)])
def test_attention_chunks_with_one_heavy_key_beside_a_long_tail(n, m, g):
    rng = np.random.default_rng(n + m)
    c, rows, scale = _sinks(rng, n, m, g, 1, 7, [0.999, 0.97, 0.9, 0.5])
    _check_tight(c, [m], rows, scale, ends=2.0 ** -31)


@pytest.mark.parametrize("m", [1, 5, 7, 8, 40])
def test_attention_heavy_keys_whatever_kernel_serves_the_row(m):
    # one token, drafts, chunks; split over the grid as the step's plan has it
    rng = np.random.default_rng(m)
    c, rows, scale = _sinks(rng, 6000, m, 6, 2, 3, [0.97, 0.9, 0.5])
    _check_tight(c, [m], rows, scale)


def test_attention_heavy_keys_of_more_rows_than_ctas():
    rng = np.random.default_rng(77)
    parts = [_sinks(rng, n, 1, 4, 2, 0, [0.97, 0.9, 0.5, 0.999]) for n in rng.integers(500, 3000, 12)]
    c = parts[0][0]
    lens, tables, base = [], [], 0
    cols = max(p[0].table.shape[1] for p in parts)
    for p, _, _ in parts:
        t = np.full((1, cols), -9, np.int32)
        t[:, :p.table.shape[1]] = np.where(p.table >= 0, p.table + base, -9)
        tables.append(t)
        lens += p.lens
        base += len(p.pools[0])
    c.pools = [np.concatenate([p[0].pools[i] for p in parts]) for i in range(2)]
    c.scales = [np.concatenate([p[0].scales[i] for p in parts]) for i in range(2)]
    pick = rng.permutation(np.repeat(np.arange(12), 30))  # 360 requests, 720 rows and KV heads
    c.table, c.lens = np.concatenate(tables)[pick], [lens[i] for i in pick]
    rows = torch.cat([parts[i][1] for i in pick])
    _check_tight(c, [1] * len(pick), rows, parts[0][2])


def _check_nan_stays_behind(n, m, g, hkv, bad):
    """NaN codes stored for tokens `bad` (counted from the first of the m that
    attend) of the middle one of three requests: every row that comes before
    the first of them is bit for bit what it was, a value's NaN reaches the
    rows that see it in its own dim alone, a key's in every dim."""
    rng = np.random.default_rng(n + 31 * m + g)
    c = Cache(rng, [40, n, 300], hkv)
    q = [1, m, 1]
    rows = _rows(rng, m + 2, g * hkv)
    clean = _attend(c, q, rows, 0.09).cpu()
    assert clean.isfinite().all()
    at = [(c.table[1, (n - m + i) // BS], hkv - 1, (n - m + i) % BS) for i in bad]
    mine = slice((hkv - 1) * g, hkv * g)
    for tensor in (1, 0):
        keep = c.pools[tensor].copy()
        for j, a in enumerate(at):
            c.pools[tensor][a][(j * 50 + 7) % 128] = 0x7F if j % 2 else 0xFF
        got = _attend(c, q, rows, 0.09).cpu()
        c.pools[tensor] = keep
        nan = torch.zeros(clean.shape, dtype=torch.bool)
        for j, i in enumerate(bad):
            nan[1 + i:1 + m, mine, (j * 50 + 7) % 128 if tensor else slice(None)] = True
        assert (got.isnan() == nan).all(), (tensor, (got.isnan() != nan).nonzero()[:5])
        assert torch.equal(got[~nan].view(torch.int16), clean[~nan].view(torch.int16))
    assert pkv.pkv_get_device_error() == 0


@pytest.mark.parametrize("g,hkv", [(1, 1), (4, 2), (7, 1)])
@pytest.mark.parametrize("n,m,bad", [(2, 2, [1]), (40, 3, [1, 2]), (33, 7, [0, 3, 6]), (130, 5, [2]), (129, 7, [6]),
                                     (3000, 6, [1, 4])])
def test_attention_nan_of_a_later_draft_token_stays_behind(n, m, bad, g, hkv):
    _check_nan_stays_behind(n, m, g, hkv, bad)


@pytest.mark.parametrize("g,hkv", [(1, 1), (4, 2), (7, 1), (8, 1)])
@pytest.mark.parametrize("n,m,bad", [(8, 8, [7]), (40, 20, [1, 2, 19]), (33, 33, [0, 16, 32]), (130, 30, [2, 28, 29]),
                                     (400, 300, [0, 15, 16, 17, 127, 128, 129, 200, 299]), (900, 17, [5]),
                                     (9000, 40, [1, 33])])
def test_attention_nan_of_a_later_chunk_token_stays_behind(n, m, bad, g, hkv):
    # items of one tile and of several, whole and split over their keys
    _check_nan_stays_behind(n, m, g, hkv, bad)


@pytest.mark.parametrize("split", [False, True])
def test_attention_nan_in_some_of_many_chunks(split):
    # Several items per SM, in a row on the same notes; every fourth request
    # holds NaN values at two of its tokens.
    rng = np.random.default_rng(5)
    R, g, hkv = (12, 4, 2) if split else (150, 2, 3)
    q = [int(x) for x in rng.integers(9, 200, R)]
    lens = [n + int(x) for n, x in zip(q, rng.integers(0, 2000 if split else 150, R))]
    c = Cache(rng, lens, hkv)
    rows = _rows(rng, sum(q), g * hkv)
    clean = _attend(c, q, rows, 0.09).cpu()
    nan = torch.zeros(clean.shape, dtype=torch.bool)
    start = np.concatenate([[0], np.cumsum(q)])
    for r in range(0, R, 4):
        for d in (3, 90):
            i, k = int(rng.integers(0, q[r])), int(rng.integers(0, hkv))
            pos = lens[r] - q[r] + i
            c.pools[1][c.table[r, pos // BS], k, pos % BS, d + k] = 0x7F
            nan[start[r] + i:start[r + 1], k * g:k * g + g, d + k] = True
    for _ in range(3):
        got = _attend(c, q, rows, 0.09).cpu()
        assert (got.isnan() == nan).all(), (got.isnan() != nan).nonzero()[:5]
        assert torch.equal(got[~nan].view(torch.int16), clean[~nan].view(torch.int16))
    assert pkv.pkv_get_device_error() == 0


@pytest.mark.parametrize("q", [[1], [5], [8], [30], [300], [64, 1, 40]])
@pytest.mark.parametrize("apart", [80, 100, 110, 124])
def test_attention_value_scales_as_far_apart_as_the_weights(apart, q):
    # Blocks whose keys weigh 2^-apart of the heaviest ones' and whose value
    # scales are 2^apart times theirs, so that both carry the output.
    rng = np.random.default_rng(apart + len(q))
    c = Cache(rng, [n + 600 for n in q], 2, spread=0.0)
    for i, n in enumerate(c.lens):
        for b, x in enumerate(c.table[i, :-(-n // BS)]):
            heavy = b % 3 == 0
            c.scales[1][x] = (1 + rng.random(2)) * 2.0 ** (-65 if heavy else apart - 65 + int(rng.integers(-2, 3)))
            c.pools[0][x, :, :, 0] = ref.encode(np.array([384.0 if heavy else -384.0]))[0]
    rows = _rows(rng, sum(q), 8, 0.25).double()
    # scores of -s and s, 2 s = apart in log2 units
    scale = 0.25
    rows[:, :, 0] = apart / 2 * np.log(2) / (scale * 3)
    # Scores, shifts and their sums stay below 2^8 in log2 units: four
    # roundings of them, 2^-24 relative each, are 2^-14 of a weight.
    _check_tight(c, q, rows.bfloat16(), scale, norm=False, exp2_off=2.0 ** -14)


@pytest.mark.parametrize("R,q,n,hkv", [(9, 8, 60, 2), (300, 256, 300, 2), (1000, 400, 2000, 2), (65, 64, 70, 8)])
def test_attention_chunk_among_idle_requests(R, q, n, hkv):
    # Fewer rows than requests.  From 512 rows times KV heads on the chunk runs
    # as one: its outputs are bit for bit those of a step that holds nothing else.
    rng = np.random.default_rng(R)
    lens = [0] * R
    lens[R // 2] = n
    c = Cache(rng, lens, hkv)
    rows = _rows(rng, q, 3 * hkv)
    m = [0] * R
    m[R // 2] = q
    _check_tight(c, m, rows, 0.09)
    idle = _attend(c, m, rows, 0.09)
    c.table, c.lens = c.table[R // 2:R // 2 + 1], [n]
    alone = _attend(c, [q], rows, 0.09)
    if q * hkv >= 512:
        assert torch.equal(idle.view(torch.int16), alone.view(torch.int16))


@pytest.mark.parametrize("m", [1, 7, 8, 40])
@pytest.mark.parametrize("binades", [6, 9, 12])
def test_attention_one_large_dim_of_q_beside_the_rest(binades, m):
    # q's dim 0 is 2^binades times the others and meets nothing in K: the
    # scores are the other dims' alone, none of them below 2^-13 of its binade.
    rng = np.random.default_rng(binades)
    c = Cache(rng, [500, 130], 2)
    c.pools[0][..., 0] = np.where(c.pools[0][..., 0] & 0x7F == 0x7F, c.pools[0][..., 0], 0)
    rows = _rows(rng, 2 * m, 8)
    rows = torch.where(rows.abs() < 0.5, 0.5, rows)
    rows[:, :, 0] = 1.5 * 2.0 ** binades
    _check_tight(c, [m, m], rows, 0.09, norm=False)


@pytest.mark.parametrize("m", [1, 3, 20])
def test_append_and_attention_past_32_bits(m):
    # the request's blocks lie beyond 2^32 bytes of either pool
    rng = np.random.default_rng(m)
    nb, n, hkv = 2_200_000, 70, 1
    small = Cache(rng, [n], hkv)
    ids = torch.tensor(nb - 1 - np.arange(5) * 3).cuda()
    pools = [torch.zeros((nb, hkv, BS, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((nb, hkv), device="cuda") for _ in range(2)]
    for big, x in zip(pools + scales, small.pools + small.scales):
        big[ids] = torch.tensor(x[small.table[0, :5]]).cuda()
    table = ids.int()[None].contiguous()
    lens, qsl = torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([0, m], dtype=torch.int32).cuda()
    k, v = _rows(rng, m, hkv), _rows(rng, m, hkv)
    pkv.pkv_append_fp8_block(k.cuda(), v.cuda(), table, lens, qsl, *pools, *scales)
    rows = _rows(rng, m, 4)
    got = pkv.pkv_attention_fp8_block(rows.cuda(), *pools, *scales, table, lens, qsl, 0.09)
    torch.cuda.synchronize()
    assert pkv.pkv_get_device_error() == 0, pkv.pkv_last_error()
    codes, sc = ref.append(k.double().numpy(), v.double().numpy(), small.table, [n], [0, m], small.pools, small.scales)
    for big, x in zip(pools + scales, codes + sc):
        assert np.array_equal(big[ids].cpu().numpy(), x[small.table[0, :5]])
        assert int((big != 0).flatten(1).any(1).sum()) == 5
    small.pools, small.scales = codes, sc
    want, bound, _ = _plain(small, [m], rows.double().numpy(), 0.09)
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
