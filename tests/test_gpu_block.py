"""The block-scaled e4m3 cache on the GPU: step buffers built and blocks given
back on the device, the quantising append, attention over it, each against a
plain 64-bit implementation, and a run of them together.

Append and the integer operators are compared exactly.  Attention is compared
element by element with the bound that blk_reference.attention derives beside
its formula (half a bf16 step of the output, 2^-9 of the probability-weighted
mean of |V| for the rounded probabilities -- 2^-11 for prefill chunks -- and the
fp32 sums), and, on random inputs, as a whole: independent roundings of the
output (2^-8) and of the weights give at most their sum of the outputs' norm."""
import numpy as np
import pytest
import torch

import paged_kv_cache_195_gb300 as pkv
from paged_kv_cache_195_gb300 import build as pkv_build

import blk_reference as ref

pytestmark = pytest.mark.gpu
BS = 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    pkv.load_library()
    yield
    assert pkv.pkv_get_device_error() == 0, pkv.pkv_last_error()


def dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(a):
    return dev(np.asarray(a, np.int32))


# ------------------------------------------------------------ build, release
def _build(prev, new, free_list, num_free, table, cap, in_place=False, **kw):
    R = len(prev)
    t, pl = i32(table), i32(prev)
    lens = pl if in_place else torch.full((R,), -7, dtype=torch.int32, device="cuda")
    qsl = torch.full((R + 1,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((cap,), -7, dtype=torch.int64, device="cuda")
    nf, ref_ = i32([num_free]), i32([-7])
    out = nf if in_place else i32([-7])
    pkv.pkv_build_step(pl, i32(new), i32(free_list), nf, t, lens, qsl, slots, num_free_out=out,
                       num_refused=ref_, **kw)
    torch.cuda.synchronize()
    return t.cpu().numpy(), lens.cpu().numpy(), qsl.cpu().numpy(), slots.cpu().numpy(), int(out), int(ref_)


def _same(got, want):
    for a, b, what in zip(got, want, ("table", "lens", "qsl", "slots", "free", "refused")):
        assert np.array_equal(a, b), what


def _step(rng, R, cols, most, blocks=None):
    prev = rng.integers(0, cols * BS // 2, R)
    new = np.where(rng.random(R) < 0.3, rng.integers(0, most + 1, R), 1)
    new = np.minimum(new, cols * BS - prev)
    held = -(-prev // BS)
    nb = blocks or int(held.sum() + (-(-(prev + new) // BS) - held).sum() + 5)
    order = rng.permutation(max(nb, int(held.sum()))).astype(np.int32)
    table = np.full((R, cols), -1, np.int32)
    mine = np.arange(cols)[None] < held[:, None]
    table[mine] = order[:held.sum()]
    fl = np.zeros(len(order), np.int32)
    free = order[held.sum():]
    fl[:len(free)] = free
    return prev, new, fl, len(free), table


@pytest.mark.parametrize("R,cols,most", [(1, 4, 60), (2, 3, 17), (33, 9, 40), (64, 130, 3), (257, 12, 90),
                                         (1024, 8, 2), (1025, 8, 50), (4096, 6, 30), (9001, 5, 1), (20000, 3, 4)])
def test_build_matches_the_plain_form(R, cols, most):
    rng = np.random.default_rng(R)
    s = _step(rng, R, cols, most)
    cap = int(s[1].sum()) + 11
    for in_place in (False, True):
        _same(_build(*s, cap, in_place), ref.build(*s, cap))


@pytest.mark.parametrize("R", [5, 300, 2000])
def test_build_refuses_in_order(R):
    rng = np.random.default_rng(R + 1)
    prev, new, fl, nf, table = _step(rng, R, 10, 60)
    total = int(new.sum())
    for free, cap in ((nf // 2, total), (nf, total // 2), (0, total), (nf, 0), (nf // 3, total // 3), (3, 7)):
        _same(_build(prev, new, fl, free, table, cap), ref.build(prev, new, fl, free, table, cap))


def test_build_first_step_of_an_empty_cache_and_idle_requests():
    fl = np.arange(40, dtype=np.int32)[::-1].copy()
    table = np.full((4, 8), -1, np.int32)
    for new in ([0, 0, 0, 0], [128, 0, 1, 16], [0, 128, 128, 128]):
        _same(_build([0] * 4, new, fl, 40, table, 400), ref.build([0] * 4, new, fl, 40, table, 400))


def test_build_reports_invalid_requests_and_ids():
    fl = np.arange(16, dtype=np.int32)
    table = np.full((5, 4), -1, np.int32)
    prev, new = [0, -1, 60, 0, 2 ** 31 - 1], [5, 3, 5, -2, 2 ** 31 - 1]
    _same(_build(prev, new, fl, 16, table, 32), ref.build(prev, new, fl, 16, table, 32))
    assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS
    fl[15] = 99  # popped first
    t, lens, qsl, slots, left, refused = _build([0, 0], [17, 2], fl, 16, table[:2], 19)
    assert t[0, 0] == 99 and (slots[:16] == -1).all() and slots[16] == 14 * 16 and slots[17] == 13 * 16
    assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS
    _same(_build([0], [3], fl[:15], 99, table[:1], 4), ref.build([0], [3], fl[:15], 15, table[:1], 4))
    assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS


def test_build_and_release_without_requests():
    got = _build([], [], np.arange(4, dtype=np.int32), 4, np.zeros((0, 3), np.int32), 3)
    _same(got, (np.zeros((0, 3)), np.zeros(0), [0], [-1] * 3, 4, 0))
    nf = i32([3])
    pkv.pkv_release_blocks(i32(np.zeros((0, 3))), i32([]), i32([]), i32([1, 2, 3, 0]), nf)
    assert int(nf) == 3


def test_build_largest_request_count():
    R = 65536
    prev, new = np.full(R, 15), np.full(R, 2)
    table = np.stack([np.arange(R), np.full(R, -1)], 1).astype(np.int32)
    fl = np.concatenate([np.arange(R, 2 * R), np.zeros(R)]).astype(np.int32)
    for free in (R, R // 2):
        _same(_build(prev, new, fl, free, table, 2 * R), ref.build(prev, new, fl, free, table, 2 * R))


def _release(table, lens, keep, fl, nf, in_place=False):
    f, n = i32(fl), i32([nf])
    out = n if in_place else i32([-7])
    pkv.pkv_release_blocks(i32(table), i32(lens), i32(keep), f, n, num_free_out=out)
    torch.cuda.synchronize()
    return f.cpu().numpy(), int(out)


@pytest.mark.parametrize("R,cols", [(1, 5), (64, 130), (1024, 9), (1025, 9), (5000, 7), (20000, 2), (3, 2048)])
def test_release_matches_the_plain_form(R, cols):
    rng = np.random.default_rng(R)
    lens = rng.integers(0, cols * BS + 1, R)
    keep = np.where(rng.random(R) < 0.5, 0, np.maximum(lens - rng.integers(0, 40, R), 0))
    order = rng.permutation(int((-(-lens // BS)).sum()) + 9).astype(np.int32)
    table = np.full((R, cols), -5, np.int32)
    mine = np.arange(cols)[None] < (-(-lens // BS))[:, None]
    table[mine] = order[:mine.sum()]
    fl = np.zeros(len(order), np.int32)
    fl[:9] = order[mine.sum():]
    want = ref.release(table, lens, keep, fl, 9)
    for in_place in (False, True):
        f, n = _release(table, lens, keep, fl, 9, in_place)
        assert n == want[1] and np.array_equal(f[:n], want[0][:n])


@pytest.mark.parametrize("R", [4, 1500])
def test_release_drops_what_is_invalid(R):
    rng = np.random.default_rng(7)
    table = rng.integers(-3, 4 * R + 6, (R, 4)).astype(np.int32)
    lens, keep = np.full(R, 64), np.zeros(R, np.int64)
    lens[0], keep[1], keep[2] = 65, -1, 70
    fl = np.zeros(4 * R, np.int32)
    want = ref.release(table, lens, keep, fl, 0)
    f, n = _release(table, lens, keep, fl, 0)
    assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS
    assert n == want[1] and np.array_equal(f[:n], want[0][:n])
    # a list with no room for all of them
    small = np.arange(10, dtype=np.int32)
    f, n = _release(np.arange(8).reshape(2, 4), [64, 64], [0, 0], small, 5)
    assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS
    assert n == 10 and f.tolist() == [0, 1, 2, 3, 4, 0, 1, 2, 3, 4]


# ------------------------------------------------------------ a cache in use
class Cache:
    """A block-scaled cache of random contents: unowned blocks and the rows
    past each request's end hold the NaN code, unowned scales NaN."""

    def __init__(self, rng, lens, hkv, spread=1.0, pow2=True, zero=0.0):
        self.lens = list(lens)
        cols = max(1, max(-(-n // BS) for n in lens))
        need = sum(-(-n // BS) for n in lens)
        nb = need + 7
        order = rng.permutation(nb)
        self.table = np.full((len(lens), cols), -9, np.int32)
        mine = np.arange(cols)[None] < np.array([-(-n // BS) for n in lens])[:, None]
        self.table[mine] = order[:need]
        self.pools, self.scales = [], []
        for _ in range(2):
            codes = ref.encode(rng.normal(0, 1, (nb, hkv, BS, 128)) * 100)
            sc = 2.0 ** (rng.normal(0, spread, (nb, hkv)) - 7)
            sc = 2.0 ** np.round(np.log2(sc)) if pow2 else sc
            sc = np.where(rng.random((nb, hkv)) < zero, 0, sc)
            own = np.zeros(nb, bool)
            own[order[:need]] = True
            codes[~own], sc[~own] = 0x7F, np.nan
            for r, n in enumerate(lens):
                if n % BS:
                    codes[self.table[r, n // BS], :, n % BS:] = 0xFF
            self.pools.append(codes)
            self.scales.append(sc.astype(np.float32))

    def gpu(self):
        return [dev(p) for p in self.pools] + [dev(s) for s in self.scales]


def _qsl(q):
    return np.concatenate([[0], np.cumsum(q)]).astype(np.int32)


def _rows(rng, T, hq, size=1.0):
    return (torch.tensor(rng.normal(0, 1, (T, hq, 128))) * size).bfloat16()


# ------------------------------------------------------------ append
def _append(c, k, v, q, opts=None):
    kp, vp, ks, vs = c.gpu()
    pkv.pkv_append_fp8_block(k.cuda(), v.cuda(), i32(c.table), i32(c.lens), i32(_qsl(q)), kp, vp, ks, vs)
    torch.cuda.synchronize()
    return [kp.cpu().numpy(), vp.cpu().numpy()], [ks.cpu().numpy(), vs.cpu().numpy()]


def _check_append(c, k, v, q):
    got = _append(c, k, v, q)
    T = sum(q)
    want = ref.append(k[:T].double().numpy(), v[:T].double().numpy(), c.table, c.lens, _qsl(q), c.pools, c.scales)
    for a, b, what in zip(got[1] + got[0], want[1] + want[0], ("k scales", "v scales", "k codes", "v codes")):
        assert np.array_equal(a, b, equal_nan=a.dtype != np.uint8), what


@pytest.mark.parametrize("hkv", [1, 2, 3, 8])
@pytest.mark.parametrize("pow2", [True, False])
def test_append_matches_the_plain_form(hkv, pow2):
    rng = np.random.default_rng(hkv)
    lens = [1, 2, 15, 16, 17, 33, 100, 64, 5, 300]
    q = [1, 1, 1, 1, 1, 18, 100, 16, 0, 77]
    c = Cache(rng, lens, hkv, pow2=pow2)
    size = 2.0 ** torch.tensor(rng.integers(-6, 7, (sum(q), hkv, 1)))
    k, v = _rows(rng, sum(q), hkv) * size, _rows(rng, sum(q), hkv) / size
    _check_append(c, k.bfloat16(), v.bfloat16(), q)


def test_append_every_offset_and_length_of_one_block():
    rng = np.random.default_rng(3)
    pairs = [(n, m) for n in range(1, 33) for m in range(1, n + 1)]
    c = Cache(rng, [n for n, _ in pairs], 2)
    q = [m for _, m in pairs]
    _check_append(c, _rows(rng, sum(q), 2, 3.0), _rows(rng, sum(q), 2, 0.2), q)


def test_append_special_values():
    rng = np.random.default_rng(4)
    lens = [16, 17, 20, 40, 18, 19, 21]
    q = [16, 1, 4, 24, 2, 3, 5]
    c = Cache(rng, lens, 2)
    k, v = _rows(rng, sum(q), 2), _rows(rng, sum(q), 2)
    k[0, 0, 5], k[3, 1, 7], k[17] = np.inf, -np.inf, np.nan  # a block of nothing finite among them
    v[0], v[16:18], v[40] = 0, 0, 3.3e38
    k[21:30] = 448 * 2.0 ** -3  # exactly 448 of a power of two
    k[30:45] *= 1e-39  # subnormals
    v[50:, :, ::2] = 2.0 ** -133
    _check_append(c, k, v, q)


def test_append_padding_and_many_requests():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 60, 3000)] + [0] * 100
    q = [min(n, int(x)) for n, x in zip(lens, rng.choice([0, 1, 1, 1, 2, 40], 3100))]
    c = Cache(rng, lens, 1)
    T = sum(q) + 37
    _check_append(c, _rows(rng, T, 1), _rows(rng, T, 1), q)


def test_append_skips_and_reports_bad_ids_and_lengths():
    rng = np.random.default_rng(6)
    c = Cache(rng, [20, 30, 40], 2)
    q = [3, 30, 2]
    good = [p.copy() for p in c.pools]
    k, v = _rows(rng, 35, 2), _rows(rng, 35, 2)
    c.table[1, 1] = 10 ** 6
    c.lens[2] = 1  # shorter than its new tokens
    got, _ = _append(c, k, v, q)
    assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS
    touched = {c.table[0, 1], c.table[1, 0]}
    for a, b in zip(got, good):
        changed = {int(x) for x in np.nonzero((a != b).any((1, 2, 3)))[0]}
        assert changed == touched


# ------------------------------------------------------------ attention
def _attend(c, q, rows, scale, workspace=None, out=None, **kw):
    kp, vp, ks, vs = c.gpu()
    return pkv.pkv_attention_fp8_block(rows.cuda(), kp, vp, ks, vs, i32(c.table), i32(c.lens), i32(_qsl(q)),
                                       scale, workspace=workspace, out=out, **kw)


def _check(c, q, rows, scale=0.09, norm=True, min_q=16, **kw):
    got = _attend(c, q, rows, scale, **kw)
    torch.cuda.synchronize()
    assert pkv.pkv_get_device_error() == 0, pkv.pkv_last_error()
    T = sum(q)
    want, bound = ref.attention(rows[:T].double().numpy(), c.pools, c.scales, c.table, c.lens, _qsl(q), scale,
                               min_q)
    g = got[:T].double().cpu().numpy()
    assert np.isfinite(g).all()
    off = np.abs(g - want)
    worst = (off / bound).max(initial=0)
    assert worst <= 1, (worst, np.unravel_index((off / bound).argmax(), off.shape))
    if norm:
        rel = np.linalg.norm(g - want) / np.linalg.norm(want)
        assert rel <= 2.0 ** -8 + 2.0 ** -9, rel
    return got


@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 6, 7, 8])
def test_attention_every_group_size(g):
    rng = np.random.default_rng(100 + g)
    lens = [1, 15, 16, 17, 31, 127, 128, 129, 300, 2000]
    c = Cache(rng, lens, 2)
    _check(c, [1] * 10, _rows(rng, 10, 2 * g))


@pytest.mark.parametrize("hkv", [1, 3, 5])
def test_attention_several_rows_a_request(hkv):
    rng = np.random.default_rng(200 + hkv)
    lens = [1, 5, 16, 40, 130, 257, 900, 0, 33]
    q = [1, 5, 3, 15, 2, 7, 4, 0, 0]
    c = Cache(rng, lens, hkv, pow2=False)
    _check(c, q, _rows(rng, sum(q) + 3, 4 * hkv))


@pytest.mark.parametrize("q", range(2, 17))
def test_attention_every_draft_length(q):
    # around the number of query tokens from which a request is a chunk
    rng = np.random.default_rng(250 + q)
    c = Cache(rng, [q, 40, 513, 127 + q, 1000, 16], 2)
    n = [q, q, q, 1, q, 1]
    _check(c, n, _rows(rng, sum(n), 12), min_q=8)


@pytest.mark.parametrize("g,hkv", [(1, 2), (3, 1), (4, 2), (6, 1), (7, 1), (8, 2)])
def test_attention_chunks(g, hkv):
    # query chunks around every tile edge, ragged ends, beside decode rows
    rng = np.random.default_rng(300 + g)
    lens = [16, 200, 64, 129, 300, 77, 513, 16]
    q = [16, 17, 64, 128, 40, 1, 33, 0]
    c = Cache(rng, lens, hkv, pow2=False)
    _check(c, q, _rows(rng, sum(q), g * hkv))


@pytest.mark.parametrize("R", [300, 1500])
def test_attention_chunks_among_many_requests(R):
    # batches of requests with no chunk, with one, with several
    rng = np.random.default_rng(260 + R)
    lens = [int(x) for x in rng.integers(1, 70, R)]
    q = [1] * R
    for r in [0, 1, 33, R // 2, R // 2 + 1, R - 1] + [int(x) for x in rng.integers(0, R, 5)]:
        q[r] = lens[r]
    c = Cache(rng, lens, 2)
    _check(c, q, _rows(rng, sum(q), 8), min_q=8)


def test_attention_long_rows_split_over_the_grid():
    rng = np.random.default_rng(8)
    c = Cache(rng, [9000, 20001, 3], 2)
    _check(c, [1, 1, 1], _rows(rng, 3, 12))
    _check(c, [2, 5, 3], _rows(rng, 10, 2))


def test_attention_long_chunk_after_a_long_prefix():
    rng = np.random.default_rng(18)
    c = Cache(rng, [5000, 1100], 1)
    _check(c, [90, 200], _rows(rng, 290, 5))


@pytest.mark.parametrize("g,hkv,lens,q", [(6, 2, [4000], [64]), (4, 1, [3000, 2100, 40], [40, 33, 1]),
                                          (8, 1, [2500], [17]), (1, 1, [6000], [130]), (7, 3, [1500], [19]),
                                          (3, 2, [700, 5000, 129], [45, 16, 129]), (2, 8, [2000, 1999], [65, 16]),
                                          (5, 1, [9000], [26]),
                                          (7, 3, [100, 3000, 160, 250, 4000, 400, 90, 640, 1000] * 3, [9] * 27),
                                          (8, 2, [300, 2500, 64, 900], [60, 33, 64, 1])])
def test_attention_few_chunks_split_over_the_keys(g, hkv, lens, q):
    # Work items cut into parts; q-tiles of one token, quads of rows without a
    # query, parts behind a row's last key; the same sums every time.
    rng = np.random.default_rng(1000 + g)
    c = Cache(rng, lens, hkv, pow2=False)
    rows = _rows(rng, sum(q) + 2, g * hkv)
    kp = c.gpu()[0]
    ws = pkv.Workspace(pkv.make_dims(tuple(rows.shape), tuple(kp.shape), len(q), c.table.shape[1]))
    first = _check(c, q, rows, workspace=ws)
    again = _check(c, q, rows)
    for _ in range(3):
        again = _attend(c, q, rows, 0.09, workspace=ws)
    T = sum(q)
    assert torch.equal(again[:T].view(torch.int16), first[:T].view(torch.int16))
    ws.nbytes -= 1  # no room for the parts: the calls split nothing
    whole = _check(c, q, rows, workspace=ws)
    d = (whole[:T].double() - first[:T].double()).abs().max() / first[:T].double().abs().max()
    assert d <= 2.0 ** -7  # two roundings to bf16, and the sums' order


@pytest.mark.parametrize("g,hkv", [(4, 4), (5, 8)])
def test_attention_many_chunks_whose_scores_rise_to_the_end(g, hkv):
    # Several work items per SM, and the running maxima raised at every tile,
    # an item's last one too.
    rng = np.random.default_rng(22)
    lens = [int(x) for x in rng.integers(100, 900, 40)]
    q = [min(n, 100) for n in lens]
    c = Cache(rng, lens, hkv)
    for r, n in enumerate(lens):
        for b in range(-(-n // BS)):
            c.scales[0][c.table[r, b]] = 2.0 ** (b // 4 % 8 - 8)
            c.scales[1][c.table[r, b]] = 2.0 ** (b // 8 * 3 % 16 - 12)
    rows = _rows(rng, sum(q), g * hkv).cuda()
    kp, vp, ks, vs = c.gpu()
    args = (rows, kp, vp, ks, vs, i32(c.table), i32(c.lens), i32(_qsl(q)), 0.09)
    got = pkv.pkv_attention_fp8_block(*args)
    torch.cuda.synchronize()
    assert pkv.pkv_get_device_error() == 0, pkv.pkv_last_error()
    for r in (0, 7, 39):  # compared request by request
        one = Cache.__new__(Cache)
        one.pools, one.scales, one.table, one.lens = c.pools, c.scales, c.table[r:r + 1], lens[r:r + 1]
        s = _qsl(q)
        want, bound = ref.attention(rows[s[r]:s[r + 1]].double().cpu().numpy(), one.pools, one.scales, one.table,
                                    one.lens, [0, q[r]], 0.09)
        assert (np.abs(got[s[r]:s[r + 1]].double().cpu().numpy() - want) <= bound).all(), r
    again = pkv.pkv_attention_fp8_block(*args)
    assert torch.equal(again.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("q", [[1, 1, 1], [30, 90, 20]])
@pytest.mark.parametrize("spread", [6.0, 12.0])
def test_attention_scales_far_apart(q, spread):
    # Scales from block to block a factor of thousands apart, zeros among them.
    rng = np.random.default_rng(int(spread))
    c = Cache(rng, [700, 129, 40], 2, spread=spread, pow2=False, zero=0.1)
    c.scales[0] = np.minimum(c.scales[0], np.float32(0.02))  # scores stay below a few hundred
    _check(c, q, _rows(rng, sum(q), 8), norm=False)


@pytest.mark.parametrize("q", [1, 30])
def test_attention_weight_on_a_block_of_small_values(q):
    # The keys that hold the probability sit in blocks whose V scale is 2^-24
    # of an unattended block's.
    rng = np.random.default_rng(9)
    c = Cache(rng, [400], 1)
    ids = c.table[0]
    c.scales[0][ids], c.scales[1][ids] = 2.0 ** -7, 2.0 ** -20
    c.scales[1][ids[3]] = 2.0 ** 4
    rows = torch.full((q, 4, 128), 0.5).bfloat16()
    c.pools[0][ids[3]] = ref.encode(np.full((1, 16, 128), -440.0))
    got = _check(c, [q], rows, scale=2.0)
    assert got.abs().max() < 1


@pytest.mark.parametrize("q", [1, 20])
def test_attention_negative_scale_and_wide_rows(q):
    # rows whose elements span forty binades, under scales of either sign
    rng = np.random.default_rng(19)
    c = Cache(rng, [200, 150], 1)
    rows = (_rows(rng, 2 * q, 4).double() * 2.0 ** torch.tensor(rng.integers(-40, 1, (2 * q, 4, 128)))).bfloat16()
    for scale in (0.5, -0.5):
        _check(c, [q, q], rows, scale=scale)


@pytest.mark.parametrize("q", [1, 20])
@pytest.mark.parametrize("size", [0.0, 1e-38, 2.0 ** -100, 30.0, 1e30])
def test_attention_sizes_of_q(size, q):
    rng = np.random.default_rng(10)
    c = Cache(rng, [200, 50], 2)
    rows = _rows(rng, 2 * q, 6, size)
    _check(c, [q, q], rows, scale=0.09 if size <= 30 else 0.09 / size)


@pytest.mark.parametrize("q", [1, 20])
def test_attention_nan_and_infinity_stay_in_their_rows(q):
    rng = np.random.default_rng(11)
    c = Cache(rng, [200, 50, 300], 1)
    rows = _rows(rng, 3 * q, 4)
    clean = _attend(c, [q] * 3, rows, 0.09).cpu()
    bad = rows.clone()
    bad[0, 1, 3], bad[2 * q, 2, 100] = float("nan"), float("inf")
    got = _attend(c, [q] * 3, bad, 0.09).cpu()
    assert got[0, 1].isnan().all() and got[2 * q, 2].isnan().all()
    keep = torch.ones(3 * q, 4, dtype=torch.bool)
    keep[0, 1] = keep[2 * q, 2] = False
    assert torch.equal(got[keep].view(torch.int16), clean[keep].view(torch.int16))
    # a NaN value in the cache reaches the rows that see it
    c.pools[1][c.table[1, 1], 0, 4, 7] = 0x7F
    got = _attend(c, [q] * 3, rows, 0.09).cpu()
    sees = torch.tensor([i >= q - (50 - 20) for i in range(q)])
    assert got[q:2 * q][sees][:, :, 7].isnan().all()
    assert torch.equal(got[:q].view(torch.int16), clean[:q].view(torch.int16))


def test_attention_padding_rows_are_left_alone():
    rng = np.random.default_rng(12)
    c = Cache(rng, [40, 0, 300, 0, 0], 2)
    rows = _rows(rng, 50, 8)
    out = torch.full((50, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    for q in ([1, 0, 1, 0, 0], [2, 0, 33, 0, 0]):
        out.fill_(7.0)
        _check(c, q, rows, out=out)
        assert (out[sum(q):] == 7).all()


def test_attention_reports_bad_ids_and_lengths():
    rng = np.random.default_rng(13)
    for q in ([1, 1, 1], [20, 20, 1]):
        c = Cache(rng, [300, 60, 40], 1)
        rows = _rows(rng, sum(q), 4)
        want = _attend(c, q, rows, 0.09).cpu()
        c.table[0, 2] = 10 ** 6
        got = _attend(c, q, rows, 0.09).cpu()
        assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS
        assert torch.equal(got[q[0]:].view(torch.int16), want[q[0]:].view(torch.int16))
        c.table[0, 2], c.lens[1] = c.table[2, 0], 10 ** 6
        got = _attend(c, q, rows, 0.09).cpu()
        assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS
        assert torch.equal(got[q[0] + q[1]:].view(torch.int16), want[q[0] + q[1]:].view(torch.int16))


@pytest.mark.parametrize("q", [[1] * 40, [1] * 30 + [25] * 10])
def test_attention_is_deterministic_on_any_stream_and_workspace(q):
    rng = np.random.default_rng(14)
    lens = [int(x) for x in rng.integers(25, 1500, 40)]
    c = Cache(rng, lens, 2)
    rows = _rows(rng, sum(q), 12).cuda()
    kp, vp, ks, vs = c.gpu()
    t, l, s = i32(c.table), i32(c.lens), i32(_qsl(q))
    args = (rows, kp, vp, ks, vs, t, l, s, 0.09)
    want = pkv.pkv_attention_fp8_block(*args)
    dims = pkv.make_dims(tuple(rows.shape), tuple(kp.shape), 40, t.shape[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [pkv.Workspace(dims) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(12):  # two streams at once, each with its own workspace
        with torch.cuda.stream(streams[i % 2]):
            outs.append(pkv.pkv_attention_fp8_block(*args, workspace=spaces[i % 2]))
    outs.append(pkv.pkv_attention_fp8_block(*args, stream=streams[0], workspace=spaces[0]))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("R,hkv,lo,hi", [(3, 2, 300, 5000), (40, 2, 1, 2500), (75, 2, 500, 540), (76, 2, 250, 300),
                                         (77, 2, 1, 300), (101, 3, 100, 140), (152, 2, 1, 600), (153, 2, 1, 200),
                                         (256, 1, 1, 700), (257, 1, 1, 700), (20, 8, 1, 900)])
def test_attention_ragged_rows_on_every_side_of_the_grid(R, hkv, lo, hi):
    # Fewer, as many and more rows (times KV heads) than SMs and than CTAs;
    # one row a request, then several, on one workspace.
    rng = np.random.default_rng(R)
    lens = [int(x) for x in rng.integers(lo, hi + 1, R)]
    c = Cache(rng, lens, hkv)
    q = [1] * R
    few = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 4, R))]
    T = max(R, sum(few))
    rows = _rows(rng, T, 3 * hkv)
    kp = c.gpu()[0]
    ws = pkv.Workspace(pkv.make_dims(tuple(rows.shape), tuple(kp.shape), R, c.table.shape[1]))
    got = [_check(c, q, rows, workspace=ws) for _ in range(2)]
    _check(c, few, rows, workspace=ws)
    got.append(_check(c, q, rows, workspace=ws))
    for o in got[1:]:
        assert torch.equal(o[:R].view(torch.int16), got[0][:R].view(torch.int16))


def test_attention_shares_a_workspace_with_the_other_caches():
    # The same lengths through two kernels that cut them differently.
    rng = np.random.default_rng(23)
    lens = [int(x) for x in rng.integers(200, 900, 50)]
    c = Cache(rng, lens, 2, zero=0.0)
    c.pools = [np.where((p & 0x7F) == 0x7F, 0, p).astype(np.uint8) for p in c.pools]
    rows = _rows(rng, 50, 8)
    kp, vp = c.gpu()[:2]
    ws = pkv.Workspace(pkv.make_dims(tuple(rows.shape), tuple(kp.shape), 50, c.table.shape[1]))
    t, l, s, one = i32(c.table), i32(c.lens), i32(_qsl([1] * 50)), torch.full((2,), 0.01, device="cuda")
    fp8 = lambda: pkv.pkv_attention_fp8kv(rows.cuda(), kp, vp, one, one, t, l, s, 0.09, workspace=ws)  # noqa: E731
    first = fp8()
    for _ in range(2):
        _check(c, [1] * 50, rows, workspace=ws)
        assert torch.equal(fp8().view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("changes", [dict(pdl=0), dict(early_plan=0), dict(plan_cache=0), dict(decode_grid=7),
                                     dict(min_chunk=1, align=0), dict(rowgroup_cost=0),
                                     dict(min_chunk=2 ** 31 - 1), dict(align_slack=2 ** 31 - 1), dict(align_slack=0), dict(prefill_min_q=0),
                                     dict(prefill_min_q=1)])
def test_attention_under_every_option(changes, pkv_opts):
    rng = np.random.default_rng(15)
    lens = [int(x) for x in rng.integers(40, 700, 20)]
    q = [1] * 12 + [3] * 4 + [31] * 4
    c = Cache(rng, lens, 2)
    pkv_opts(**changes)
    _check(c, q, _rows(rng, sum(q), 8), min_q=changes.get("prefill_min_q", 16) or 10 ** 9)


def test_attention_withheld_q_times_out(pkv_opts):
    rng = np.random.default_rng(16)
    c = Cache(rng, [300, 40, 129, 700, 2048], 2)
    rows = _rows(rng, 5, 8)
    kp, vp, ks, vs = c.gpu()
    t, l, s = i32(c.table), i32(c.lens), i32(_qsl([1] * 5))
    dims = pkv.make_dims(tuple(rows.shape), tuple(kp.shape), 5, t.shape[1])
    ws = pkv.Workspace(dims)
    out = torch.full((5, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv_opts(wait_limit_us=1000, debug_withhold_q=1)
    pkv.pkv_attention_fp8_block(rows.cuda(), kp, vp, ks, vs, t, l, s, 0.09, out=out, workspace=ws)
    assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_TIMEOUT
    assert out.isnan().all()
    pkv_opts(wait_limit_us=2_000_000, debug_withhold_q=0)
    pkv.pkv_workspace_init(ws, dims)
    _check(c, [1] * 5, rows, workspace=ws)


def test_binding_refusals():
    rng = np.random.default_rng(17)
    c = Cache(rng, [20, 30], 2)
    kp, vp, ks, vs = c.gpu()
    rows = _rows(rng, 2, 8).cuda()
    t, l, s = i32(c.table), i32(c.lens), i32([0, 1, 2])
    ok = dict(q=rows, k_pool=kp, v_pool=vp, k_scales=ks, v_scales=vs, block_tables=t, seq_lens=l, query_start_loc=s)
    for name, bad in [("q", rows.transpose(0, 1)), ("q", rows.half()), ("k_pool", kp.view(torch.int8)),
                      ("v_pool", vp[:-1]), ("k_scales", ks[:, :1].contiguous()), ("v_scales", vs.double()),
                      ("k_scales", ks.t()), ("block_tables", t[:1]), ("seq_lens", l.long()),
                      ("query_start_loc", s[:2]), ("q", rows[..., :64].contiguous()), ("seq_lens", l.cpu())]:
        with pytest.raises(ValueError):
            pkv.pkv_attention_fp8_block(**dict(ok, **{name: bad}), scale=0.1)
    for scale in (0.0, float("nan")):
        with pytest.raises(pkv.PagedKVError):
            pkv.pkv_attention_fp8_block(**ok, scale=scale)
    kv = _rows(rng, 2, 2).cuda()
    ok = dict(k_new=kv, v_new=kv, block_tables=t, seq_lens=l, query_start_loc=s, k_pool=kp, v_pool=vp, k_scales=ks,
              v_scales=vs)
    for name, bad in [("k_new", kv.float()), ("v_new", kv[:1]), ("k_new", kv[:, :1].contiguous()),
                      ("v_scales", vs[:3]), ("k_pool", kp[:3]), ("query_start_loc", s[1:])]:
        with pytest.raises(ValueError):
            pkv.pkv_append_fp8_block(**dict(ok, **{name: bad}))
    one = i32([0])
    ok = dict(prev_lens=l, new_tokens=l, free_list=l, num_free=one, block_tables=t, seq_lens=l, query_start_loc=s,
              slot_mapping=torch.zeros(4, dtype=torch.int64, device="cuda"))
    for name, bad in [("new_tokens", one), ("num_free", l), ("slot_mapping", l), ("query_start_loc", l),
                      ("num_refused", l), ("block_tables", t[:, ::2])]:
        with pytest.raises(ValueError):
            pkv.pkv_build_step(**dict(ok, **{name: bad}))
    ok = dict(block_tables=t, seq_lens=l, keep_lens=l, free_list=l, num_free=one)
    for name, bad in [("keep_lens", one), ("num_free_out", l), ("free_list", l.float())]:
        with pytest.raises(ValueError):
            pkv.pkv_release_blocks(**dict(ok, **{name: bad}))


# ------------------------------------------------------------ together
class Loop:
    """A serving loop whose step buffers live on the device, and the same loop
    in the plain implementations."""

    def __init__(self, R, cols, nb, cap, hq, hkv):
        self.R, self.cap, self.hq, self.hkv = R, cap, hq, hkv
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.lens, self.new, self.qsl, self.keep = z(R), z(R), z(R + 1), z(R)
        self.table = torch.full((R, cols), -1, dtype=torch.int32, device="cuda")
        self.free, self.nfree, self.refused = torch.arange(nb, dtype=torch.int32, device="cuda"), i32([nb]), i32([0])
        self.slots = torch.zeros(cap, dtype=torch.int64, device="cuda")
        self.pools = [torch.full((nb, hkv, BS, 128), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.full((nb, hkv), float("nan"), device="cuda") for _ in range(2)]
        self.k, self.v = (torch.zeros(cap, hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.q, self.out = (torch.zeros(cap, hq, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.ws = pkv.Workspace(pkv.make_dims(tuple(self.q.shape), tuple(self.pools[0].shape), R, cols))
        self.p = dict(lens=np.zeros(R, np.int64), table=np.full((R, cols), -1, np.int32), free=np.arange(nb, dtype=np.int32),
                      nfree=nb, pools=[p.cpu().numpy() for p in self.pools], scales=[s.cpu().numpy() for s in self.scales])

    def step(self):
        pkv.pkv_build_step(self.lens, self.new, self.free, self.nfree, self.table, self.lens, self.qsl, self.slots,
                           num_refused=self.refused)
        pkv.pkv_append_fp8_block(self.k, self.v, self.table, self.lens, self.qsl, *self.pools, *self.scales)
        pkv.pkv_attention_fp8_block(self.q, *self.pools, *self.scales, self.table, self.lens, self.qsl, 0.09,
                                    out=self.out, workspace=self.ws)

    def release(self):
        pkv.pkv_release_blocks(self.table, self.lens, self.keep, self.free, self.nfree)
        self.lens.copy_(self.keep)

    def inputs(self, rng, new):
        self.new.copy_(i32(new))
        for t, h in ((self.k, self.hkv), (self.v, self.hkv), (self.q, self.hq)):
            t.copy_(_rows(rng, self.cap, h) * 2.0 ** torch.tensor(rng.integers(-3, 4, (self.cap, 1, 1))).float())
        self.out.fill_(7.0)

    def check(self, new):
        p = self.p
        p["table"], p["lens"], qsl, slots, p["nfree"], refused = ref.build(
            p["lens"], new, p["free"], p["nfree"], p["table"], self.cap)
        _same([x.cpu().numpy() for x in (self.table, self.lens, self.qsl, self.slots)] + [int(self.nfree), int(self.refused)],
              (p["table"], p["lens"], qsl, slots, p["nfree"], refused))
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        p["pools"], p["scales"] = ref.append(f(self.k), f(self.v), p["table"], p["lens"], qsl, p["pools"], p["scales"])
        for a, b in zip(self.pools + self.scales, p["pools"] + p["scales"]):
            assert np.array_equal(a.cpu().numpy(), b, equal_nan=b.dtype != np.uint8)
        want, bound = ref.attention(f(self.q), p["pools"], p["scales"], p["table"], p["lens"], qsl, 0.09)
        T = qsl[-1]
        assert (np.abs(f(self.out) - want)[:T] <= bound[:T]).all()
        assert (self.out[T:] == 7).all()

    def check_release(self, keep):
        p = self.p
        p["free"], p["nfree"] = ref.release(p["table"], p["lens"], keep, p["free"], p["nfree"])
        p["lens"] = np.asarray(keep, np.int64)
        assert int(self.nfree) == p["nfree"]
        assert np.array_equal(self.free.cpu().numpy()[:p["nfree"]], p["free"][:p["nfree"]])


def _news(rng, lens, cols, most):
    new = rng.choice([0, 1, 1, 1, 2, most], len(lens))
    return np.minimum(new, cols * BS - lens)


@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(graph):
    rng = np.random.default_rng(20)
    loop = Loop(R=9, cols=8, nb=40, cap=100, hq=8, hkv=2)  # blocks and rows run out now and then
    g = None
    refused = 0
    for i in range(14):
        new = _news(rng, loop.p["lens"], 8, 45)
        loop.inputs(rng, new)
        if graph and g is None:
            loop.step()  # a first eager step, then the capture
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                loop.step()
        elif graph:
            g.replay()
        else:
            loop.step()
        torch.cuda.synchronize()
        loop.check(new)
        refused += int(loop.refused)
        keep = np.where(rng.random(9) < 0.25, 0, np.maximum(loop.p["lens"] - rng.integers(0, 4, 9), 0))
        loop.keep.copy_(i32(keep))
        loop.release()
        torch.cuda.synchronize()
        loop.check_release(keep)
    assert refused > 0
    assert pkv.pkv_get_device_error() == 0


@pytest.mark.parametrize("new,steps", [(1, 60), (20, 8)])
def test_attention_right_after_build_reads_the_new_tables(new, steps):
    # No append between: the lengths and tables come from the kernel issued
    # just before the attention (decode rows; prefill chunks), step after step
    # on the same buffers.
    rng = np.random.default_rng(21)
    R, cols = 30, -(-new * steps // BS)
    loop = Loop(R=R, cols=cols, nb=R * cols, cap=R * new, hq=12, hkv=2)
    for p in loop.pools:
        p.copy_(dev(ref.encode(rng.normal(0, 100, tuple(p.shape)))))
    for s in loop.scales:
        s.fill_(2.0 ** -7)
    loop.q.copy_(_rows(rng, R * new, 12))
    loop.new.fill_(new)
    outs = []
    for i in range(steps):
        pkv.pkv_build_step(loop.lens, loop.new, loop.free, loop.nfree, loop.table, loop.lens, loop.qsl, loop.slots)
        outs.append(pkv.pkv_attention_fp8_block(loop.q, *loop.pools, *loop.scales, loop.table, loop.lens, loop.qsl,
                                                0.09, workspace=loop.ws))
    torch.cuda.synchronize()
    table = loop.table.cpu().numpy()
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    pools, scales = [p.cpu().numpy() for p in loop.pools], [s.cpu().numpy() for s in loop.scales]
    for i in sorted({0, 1, steps // 4, steps // 2, steps - 1}):
        want, bound = ref.attention(f(loop.q), pools, scales, table, [new * (i + 1)] * R, _qsl([new] * R), 0.09)
        assert (np.abs(f(outs[i]) - want) <= bound).all(), i
    assert pkv.pkv_get_device_error() == 0
