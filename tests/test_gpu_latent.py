"""The latent cache's operators and the norm and rotation ahead of the append,
on a GPU, against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import paged_kv_cache_195_gb300 as pkv
from paged_kv_cache_195_gb300 import build as pkv_build

import lat_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    pkv.load_library()


@pytest.fixture(autouse=True)
def _clean():
    yield
    torch.cuda.synchronize()
    assert pkv.pkv_get_device_error() == 0


def f64(t):
    return t.detach().double().cpu().numpy()


def dev(x, dtype):
    return torch.as_tensor(np.ascontiguousarray(x)).to(dtype).cuda()


def close(got, want, bound, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    nan = np.isnan(want)
    assert (np.isnan(got) == nan).all(), f"{what}: NaN in other places ({np.isnan(got).sum()} for {nan.sum()})"
    inf = np.isinf(want)
    assert (got[inf] == want[inf]).all(), what
    fin = ~nan & ~inf
    off = np.abs(got[fin] - want[fin]) - bound[fin]
    assert (off <= 0).all(), f"{what}: off by {off.max():.3g} more than the bound, " \
        f"at {np.argwhere(fin)[off.argmax()]}, {np.abs(got[fin] - want[fin])[off.argmax()]:.3g}"


# ------------------------------------------------------------ norm, rotation, append
def rope_case(T, hq, hkv, rot, inter, wq, wk, seed=0, eps=1e-6, max_pos=5000):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, hq + 2 * hkv, 128, generator=g) * 2).to(BF).cuda()
    w = [(1 + 0.3 * torch.randn(128, generator=g)).to(BF).cuda() if on else None for on in (wq, wk)]
    nb = T // 16 + 3
    slots = torch.randperm(nb * 16, generator=g)[:T].cuda()
    pos = torch.randint(0, max_pos, (T,), generator=g).cuda()
    pools = [torch.randn(nb, hkv, 16, 128, generator=g).to(BF).cuda() for _ in range(2)]
    return qkv, w, slots, pos, pools, torch.from_numpy(ref.table(max_pos, rot)).cuda()


def rope_check(qkv, before, w, slots, pos, pools, cs, inter, out, hq, hkv, eps, old_out):
    T = qkv.shape[0]
    live = (slots >= 0).cpu().numpy()
    x = f64(before)
    rows = cs.cpu().numpy()[np.where(live, pos.cpu().numpy(), 0)]
    want, size = [], []
    for a, ww in ((x[:, :hq], w[0]), (x[:, hq:hq + hkv], w[1])):
        y, s = ref.rotate(a if ww is None else ref.norm(a, f64(ww), eps), rows, inter)
        want.append(y)
        size.append(s)
    close(f64(out)[live], want[0][live], ref.turned_bound(want[0], size[0])[live], "q")
    assert torch.equal(out[~torch.from_numpy(live).cuda()], old_out[~torch.from_numpy(live).cuda()])
    k, v = (f64(p) for p in pools[1])
    k0, v0 = (f64(p) for p in pools[0])
    bound = np.zeros_like(k0)
    s = slots.cpu().numpy()[live]
    k0[s // 16, :, s % 16] = want[1][live]
    bound[s // 16, :, s % 16] = ref.turned_bound(want[1], size[1])[live]
    v0[s // 16, :, s % 16] = x[:, hq + hkv:][live]
    close(k, k0, bound, "k pool")
    assert np.array_equal(v, v0), "v pool"


@pytest.mark.parametrize("T,hq,hkv,rot,inter,wq,wk", [
    (1, 1, 1, 128, False, True, True), (1, 12, 2, 128, True, True, True), (3, 5, 5, 64, False, True, False),
    (7, 21, 3, 96, False, False, True), (64, 12, 2, 128, False, True, True), (33, 8, 8, 16, True, False, False),
    (130, 32, 8, 112, False, True, True), (701, 32, 8, 48, True, True, True), (2000, 4, 1, 128, False, True, True),
    (5, 0, 2, 128, False, True, True), (300, 70, 7, 80, True, True, True)])
@pytest.mark.parametrize("place", ["split", "in place", "apart"])
def test_norm_rope_append(T, hq, hkv, rot, inter, wq, wk, place):
    eps = 1e-5
    qkv, w, slots, pos, pools, cs = rope_case(T, hq, hkv, rot, inter, wq, wk, seed=T + hq)
    if T > 4:
        slots[T // 2] = -1
        pos[T // 2] = 1 << 40  # not looked at
    before, old = qkv.clone(), [p.clone() for p in pools]
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    if place == "split":
        kw, old_out = dict(q_out=torch.full((T, hq, 128), 7.0, dtype=BF, device="cuda")), None
        old_out = kw["q_out"].clone()
    elif place == "in place":
        kw, old_out = dict(q_out=q), before[:, :hq].clone()
    else:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        wide = torch.full((T, hq + 3, 128), 7.0, dtype=BF, device="cuda")
        kw, old_out = dict(q_out=wide[:, 2:2 + hq]), wide[:, 2:2 + hq].clone()
    out = pkv.pkv_norm_rope_append(q, k, v, pos, cs, slots, *pools, q_weight=w[0], k_weight=w[1], eps=eps,
                                   interleaved=inter, **kw)
    rope_check(qkv, before, w, slots, pos, (old, pools), cs, inter, out, hq, hkv, eps, old_out)
    if place == "apart":
        assert (wide[:, :2] == 7).all() and (wide[:, 2 + hq:] == 7).all()


def test_norm_rope_extremes():
    """Rows of zeros, of one huge and of tiny values, infinities and NaN."""
    qkv, w, slots, pos, pools, cs = rope_case(8, 2, 1, 128, False, True, True)
    qkv[0] = 0
    qkv[1] = 3e38
    qkv[2, :, 5] = 2e38
    qkv[3] = 1e-20
    qkv[4, 0, 3] = float("inf")
    qkv[5, 1, 4] = float("nan")
    qkv[6] *= 1e19
    before, old = qkv.clone(), [p.clone() for p in pools]
    q, k, v = qkv.split([2, 1, 1], 1)
    out = pkv.pkv_norm_rope_append(q, k, v, pos, cs, slots, *pools, q_weight=w[0], k_weight=w[1], eps=1e-6)
    x = f64(before)
    rows = cs.cpu().numpy()[pos.cpu().numpy()]
    y, s = ref.rotate(ref.norm(x[:, :2], f64(w[0]), 1e-6), rows, False)
    ok = np.isfinite(x[:, :2]).all(2)
    close(f64(out)[ok], y[ok], ref.turned_bound(y, s)[ok])
    assert np.isnan(f64(out)[5, 1]).all()
    got = f64(out)[4, 0]  # x / inf: zeros but for inf / inf, which its pair gets too
    assert np.isnan(got[[3, 67]]).all() and (np.delete(got, [3, 67]) == 0).all()


def test_norm_rope_errors_skip_the_token():
    qkv, w, slots, pos, pools, cs = rope_case(6, 4, 2, 128, False, True, True)
    old = [p.clone() for p in pools]
    bad_slots, bad_pos = slots.clone(), pos.clone()
    bad_slots[1] = pools[0].shape[0] * 16
    bad_pos[2], bad_pos[4] = cs.shape[0], -1
    q, k, v = qkv.split([4, 2, 2], 1)
    out = torch.full((6, 4, 128), 7.0, dtype=BF, device="cuda")
    pkv.pkv_norm_rope_append(q, k, v, bad_pos, cs, bad_slots, *pools, q_weight=w[0], k_weight=w[1], q_out=out)
    assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS
    bad_slots[[1, 2, 4]] = -1
    rope_check(qkv, qkv, w, bad_slots, bad_pos, (old, pools), cs, False, out, 4, 2, 1e-6,
               torch.full((6, 4, 128), 7.0, dtype=BF, device="cuda"))


@pytest.mark.parametrize("T,heads,inter,weight,place", [
    (1, 1, False, True, "out"), (1, 16, True, True, "in"), (5, 128, True, False, "out"), (64, 16, True, True, "out"),
    (7, 0, False, True, "none"), (130, 33, False, True, "in"), (1500, 40, True, True, "out"), (300, 128, False, True, "turned")])
def test_append_latent(T, heads, inter, weight, place):
    g = torch.Generator().manual_seed(T + heads)
    wide = (torch.randn(T, 1600, generator=g) * 2).to(BF).cuda()
    kv = wide[:, 1024:]
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(BF).cuda() if weight else None
    nb = T // 16 + 3
    slots = torch.randperm(nb * 16, generator=g)[:T].cuda()
    pos = torch.randint(0, 3000, (T,), generator=g).cuda()
    if T > 4:
        slots[3] = -1
        pos[3] = -5
    live = (slots >= 0).cpu().numpy()
    pool = torch.randn(nb, 16, 576, generator=g).to(BF).cuda()
    cs = torch.from_numpy(ref.table(3000, 64)).cuda()
    want_pool, bound = f64(pool), np.zeros((nb, 16, 576))
    rows = cs.cpu().numpy()[np.where(live, pos.cpu().numpy(), 0)]
    x = f64(kv)
    c = x[:, None, :512] if w is None else ref.norm(x[:, None, :512], f64(w), 1e-6)
    r, size = ref.rotate(x[:, None, 512:], rows, inter)
    s = slots.cpu().numpy()[live]
    y, z = np.concatenate([c, r], 2)[:, 0], np.concatenate([np.abs(c), size], 2)[:, 0]
    want_pool.reshape(-1, 576)[s] = y[live]
    bound.reshape(-1, 576)[s] = ref.turned_bound(y, z)[live]
    kw, out = {}, None
    if place != "none":
        full = torch.randn(T, heads, 192, generator=g).to(BF).cuda()
        qr = full[:, :, 128:]
        if place == "turned":  # heads outermost
            qr = torch.randn(heads, T, 192, generator=g).to(BF).cuda()[:, :, 128:].transpose(0, 1)
        q0 = qr.clone()
        out = qr if place == "in" else torch.full((T, heads, 576), 7.0, dtype=BF, device="cuda")[:, :, 512:]
        old = out.clone()
        kw = dict(q_rope=qr) if place == "in" else dict(q_rope=qr, q_rope_out=out)
    pkv.pkv_append_latent(kv, pos, cs, slots, pool, weight=w, interleaved=inter, **kw)
    close(pool, want_pool, bound, "pool")
    if out is not None:
        y, z = ref.rotate(f64(q0), rows, inter)
        close(f64(out)[live], y[live], ref.turned_bound(y, z)[live], "q")
        assert np.array_equal(f64(out)[~live], f64(old)[~live])


def test_append_latent_errors_skip_the_token():
    T = 5
    kv = torch.randn(T, 576, device="cuda").to(BF)
    pool = torch.zeros(2, 16, 576, dtype=BF, device="cuda")
    cs = torch.from_numpy(ref.table(100, 64)).cuda()
    slots = torch.tensor([0, 32, 2, 3, 4], device="cuda")
    pos = torch.tensor([1, 1, 100, -1, 99], device="cuda")
    qr = torch.ones(T, 3, 64, device="cuda", dtype=BF)
    pkv.pkv_append_latent(kv, pos, cs, slots, pool, q_rope=qr)
    assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS
    rows = pool.view(32, 576).any(1).cpu().tolist()
    assert [i for i, on in enumerate(rows) if on] == [0, 4]
    assert (qr[[1, 2, 3]] == 1).all() and (qr[0] != 1).any()


# --------------------------------------------------------------- absorbed attention
def lat_case(lens, qs, heads, seed=0, pad=0, poison=True):
    """A step over a latent cache, every slot that no request owns NaN."""
    g = torch.Generator().manual_seed(seed)
    cols = max([ref.cdiv(n, 16) for n in lens] + [1]) + 1
    need = sum(ref.cdiv(n, 16) for n in lens)
    nb = need + 3
    perm = torch.randperm(nb, generator=g).tolist()
    tab = np.full((len(lens), cols), 10 ** 8, np.int32)
    pool = torch.full((nb, 16, 576), float("nan") if poison else 0.0)
    for r, n in enumerate(lens):
        for b in range(ref.cdiv(n, 16)):
            tab[r, b] = perm.pop()
            k = min(16, n - 16 * b)
            pool[tab[r, b], :k] = torch.randn(k, 576, generator=g)
    qsl = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
    q = torch.randn(int(qsl[-1]) + pad, heads, 576, generator=g)
    return dict(q=q.to(BF).cuda(), pool=pool.to(BF).cuda(), tab=tab, lens=np.array(lens, np.int32), qsl=qsl,
                scale=192 ** -0.5)


def lat_run(c, **kw):
    return pkv.pkv_attention_latent(c["q"], c["pool"], dev(c["tab"], torch.int32), dev(c["lens"], torch.int32),
                                    dev(c["qsl"], torch.int32), c["scale"], **kw)


def lat_check(c, out):
    n = int(c["qsl"][-1])
    want, bound = ref.absorbed(f64(c["q"]), f64(c["pool"]), c["tab"], c["lens"], c["qsl"], c["scale"])
    close(f64(out)[:n], want[:n], bound[:n])


@pytest.mark.parametrize("heads", [1, 5, 16, 17, 32, 33, 48, 64, 65, 100, 128])
@pytest.mark.parametrize("lens", [[1], [64], [65], [17, 64, 100, 128], [1, 2, 15, 16, 63, 130, 700]])
def test_absorbed_decode(heads, lens):
    c = lat_case(lens, [1] * len(lens), heads, seed=heads + len(lens))
    lat_check(c, lat_run(c))


@pytest.mark.parametrize("heads", [1, 3, 16, 20, 64, 128])
@pytest.mark.parametrize("lens,qs", [([4], [4]), ([70, 9, 300], [5, 9, 1]), ([200, 130, 64, 1], [130, 1, 64, 1]),
                                     ([1000, 67], [3, 66])])
def test_absorbed_chunks(heads, lens, qs):
    c = lat_case(lens, qs, heads, seed=heads)
    lat_check(c, lat_run(c))


@pytest.mark.parametrize("heads,lens,qs", [(16, [5000], [1]), (128, [5000, 300], [1, 1]), (16, [3000, 50, 2000], [4, 1, 70]),
                                           (40, [20000], [2]), (8, [900] * 40, [1] * 40)])
def test_absorbed_split_rows(heads, lens, qs):
    c = lat_case(lens, qs, heads, seed=1)
    lat_check(c, lat_run(c))


def test_absorbed_many_requests():
    rng = np.random.default_rng(5)
    lens = rng.integers(1, 90, 1500).tolist()
    qs = [min(n, int(q)) for n, q in zip(lens, rng.integers(0, 3, 1500))]
    c = lat_case(lens, qs, 2, seed=3)
    lat_check(c, lat_run(c))


# ------------------------------------------------------------------ expanded form
@pytest.mark.parametrize("lens,heads", [([1], 1), ([128], 1), ([129], 3), ([17, 64, 100, 128], 16), ([0, 5, 0, 700], 2),
                                        ([1000, 1, 333], 7), ([40] * 300, 1), ([260, 2000], 33)])
def test_expand(lens, heads):
    c = lat_case(lens, [min(n, 1) for n in lens], 1, seed=heads)
    g = torch.Generator().manual_seed(heads)
    w = (torch.randn(heads, 256, 512, generator=g) * 512 ** -0.5).to(BF).cuda()
    n = sum(lens)
    kv = torch.full((n + 5, heads, 256), 7.0, dtype=BF, device="cuda")
    kr = torch.full((n + 5, 64), 7.0, dtype=BF, device="cuda")
    ksl = dev(np.concatenate([[0], np.cumsum(lens)]), torch.int32)
    pkv.pkv_expand_latent(c["pool"], w, dev(c["tab"], torch.int32), dev(c["lens"], torch.int32), ksl, kv, kr)
    want, rope, bound = ref.expand(f64(c["pool"]), f64(w), c["tab"], lens)
    close(f64(kv)[:n], want, bound)
    assert np.array_equal(f64(kr)[:n], rope)
    assert (kv[n:] == 7).all() and (kr[n:] == 7).all()


def exp_case(lens, qs, heads, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens)
    qsl = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
    return dict(q=torch.randn(int(qsl[-1]) + pad, heads, 192, generator=g).to(BF).cuda(),
                kv=torch.randn(n, heads, 256, generator=g).to(BF).cuda(),
                kr=torch.randn(n, 64, generator=g).to(BF).cuda(), lens=np.array(lens, np.int32), qsl=qsl,
                ksl=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), scale=192 ** -0.5)


def exp_run(c, **kw):
    return pkv.pkv_attention_expanded(c["q"], c["kv"], c["kr"], dev(c["lens"], torch.int32), dev(c["qsl"], torch.int32),
                                      dev(c["ksl"], torch.int32), c["scale"], **kw)


def exp_check(c, out):
    n = int(c["qsl"][-1])
    want, bound = ref.expanded(f64(c["q"]), f64(c["kv"]), f64(c["kr"]), c["lens"], c["qsl"], c["scale"])
    close(f64(out)[:n], want[:n], bound[:n])


@pytest.mark.parametrize("heads", [1, 3, 16])
@pytest.mark.parametrize("lens,qs", [([1], [1]), ([128], [128]), ([129, 5], [129, 5]), ([70, 9, 300], [5, 9, 1]),
                                     ([200, 0, 130, 64, 1], [130, 0, 1, 64, 1]), ([1000, 67], [300, 66]),
                                     ([257] * 40, [33] * 40)])
def test_expanded(heads, lens, qs):
    c = exp_case(lens, qs, heads, seed=heads)
    exp_check(c, exp_run(c))


@pytest.mark.parametrize("heads,lens,qs", [(1, [6000], [1]), (2, [3000, 700], [200, 3]), (1, [900, 5000, 2], [129, 64, 2]),
                                           (130, [300], [200])])
def test_expanded_split_items(heads, lens, qs):
    c = exp_case(lens, qs, heads, seed=2)
    exp_check(c, exp_run(c))


@pytest.mark.parametrize("heads,lens,qs", [(16, [512] * 8, [512] * 8), (80, [700, 9, 0, 300], [514, 9, 0, 257]),
                                           (33, [2000], [1200]), (128, [321, 321], [193, 320]),
                                           (20, [256, 257, 384, 385, 511, 513, 600], [256, 257, 384, 129, 511, 513, 1])])
def test_expanded_in_pairs(heads, lens, qs):
    """Steps that take the form of two CTAs an item: whole pairs of query tiles, ones
    whose second has few tokens or none, lengths at tile edges, empty requests."""
    n, sms = sum(qs), torch.cuda.get_device_properties(0).multi_processor_count
    assert n >= 192 * len(lens) and n * heads >= 256 * sms  # the host's rule
    c = exp_case(lens, qs, heads, seed=heads)
    exp_check(c, exp_run(c))


def test_expanded_many_requests():
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 150, 500).tolist()
    c = exp_case(lens, [min(n, int(q)) for n, q in zip(lens, rng.integers(0, 140, 500))], 1, seed=3)
    exp_check(c, exp_run(c))


# ------------------------------------------------------------ special values
def test_absorbed_special_values_reach_their_rows_only():
    """A NaN or an infinity in one token's latent or rotated key, as the last but
    one, a middle and an early token of a chunk: later tokens see it, earlier ones
    must not (with several tokens to a work item they share its tiles)."""
    for heads, m, at in ((4, 12, 5), (16, 3, 1), (1, 64, 40), (20, 3, 2), (2, 40, 0)):
        for what in ("nan", "inf", "-inf"):
            for part in ("latent", "rope"):
                c = lat_case([100, 70], [m, min(m, 60)], heads, seed=m)
                # -inf scores need a query that makes them: every query 1 in that dim
                dim = 17 if part == "latent" else 530
                c["q"][:, :, dim] = 1
                pos = 100 - m + at
                c["pool"][c["tab"][0, pos // 16], pos % 16, dim] = float(what)
                lat_check(c, lat_run(c))


def test_absorbed_row_that_sees_only_minus_infinity():
    c = lat_case([3], [3], 2)
    c["q"][:, :, 5] = 1
    for j in range(3):
        c["pool"][c["tab"][0, 0], j, 5] = float("-inf")
    out = f64(lat_run(c))
    assert np.isnan(out).all()  # exp(-inf - -inf): no weights at all


def test_absorbed_extremes():
    """Scores from far apart, equal keys, zero queries, a growing maximum."""
    c = lat_case([700, 300], [2, 1], 24, seed=9)
    c["q"][0] *= 30
    c["q"][1] = 0
    p = c["pool"]
    ids = torch.from_numpy(c["tab"][0, :44].astype(np.int64)).cuda()
    p[ids] = p[ids] * (torch.arange(44, device="cuda")[:, None, None] / 8 + 0.1).to(BF)
    p[torch.from_numpy(c["tab"][1, :19].astype(np.int64)).cuda()] = 0.5
    p[c["tab"][0, 43], 12:] = float("nan")
    p[c["tab"][1, 18], 12:] = float("nan")
    lat_check(c, lat_run(c))


@pytest.mark.parametrize("heads,lens,qs", [(1, [200], [150]), (3, [400, 130], [256, 130]), (8, [700] * 8, [512] * 8),
                                           (20, [700] * 4, [520] * 4)])
def test_expanded_special_values_reach_their_rows_only(heads, lens, qs):
    """Values and keys that are not finite at several of a chunk's own tokens (the last
    set runs in pairs of CTAs)."""
    for where, what in (("v", "nan"), ("v", "inf"), ("v", "-inf"), ("k", "nan"), ("r", "nan"), ("v2", "inf")):
        c = exp_case(lens, qs, heads, seed=4)
        m, n = qs[0], lens[0]
        for i, at in enumerate((0, 1, m // 2, 127 % m, m - 2)):
            pos = n - m + at
            if where == "k":
                c["kv"][pos, i % heads, 7] = float(what)
            elif where == "r":
                c["kr"][pos, 3] = float(what)
            else:
                c["kv"][pos, i % heads, 128 + 9 * i + (60 if where == "v2" else 0)] = float(what)
        exp_check(c, exp_run(c))


def test_expanded_ignores_what_follows_a_request():
    """The rows of kv behind a request's end, another's or none's, hold NaN."""
    c = exp_case([100, 60, 33], [100, 60, 33], 2, seed=5)
    c["kv"][100:160] = float("nan")
    c["kr"][100:160] = float("nan")
    pad = torch.full((77, 2, 256), float("nan"), dtype=BF, device="cuda")
    c["kv"], c["kr"] = torch.cat([c["kv"], pad]), torch.cat([c["kr"], pad[:, 0, :64].contiguous()])
    out = f64(exp_run(c))
    want, bound = ref.expanded(f64(c["q"]), np.nan_to_num(f64(c["kv"])), np.nan_to_num(f64(c["kr"])), c["lens"], c["qsl"],
                               c["scale"])
    live = np.r_[0:100, 160:193]
    close(out[live], want[live], bound[live])
    assert np.isnan(out[100:160]).all()


def test_expand_special_values_stay_in_their_rows():
    c = lat_case([70, 300], [1, 1], 1, seed=6)
    w = torch.randn(3, 256, 512, device="cuda").to(BF)
    for r, j, v in ((0, 3, "nan"), (0, 69, "inf"), (1, 128, "-inf")):
        c["pool"][c["tab"][r, j // 16], j % 16, 40] = float(v)
    kv, kr = torch.empty(370, 3, 256, dtype=BF, device="cuda"), torch.empty(370, 64, dtype=BF, device="cuda")
    pkv.pkv_expand_latent(c["pool"], w, dev(c["tab"], torch.int32), dev(c["lens"], torch.int32),
                          dev([0, 70, 370], torch.int32), kv, kr)
    bad = [3, 69, 70 + 128]
    assert (~torch.isfinite(kv[bad])).all()
    keep = np.delete(np.arange(370), bad)
    pool = torch.nan_to_num(c["pool"].float(), nan=0, posinf=0, neginf=0)
    want, rope, bound = ref.expand(f64(pool), f64(w), c["tab"], c["lens"])
    close(f64(kv)[keep], want[keep], bound[keep])


# ------------------------------------------------------------ padding, errors, order of calls
@pytest.mark.parametrize("heads", [1, 16, 24, 64, 100, 128])
@pytest.mark.parametrize("lens,qs", [([9000], [1]), ([20000, 513], [1, 1]), ([6000, 7, 0, 5000], [2, 1, 0, 1]),
                                     ([3000] * 9, [1] * 9), ([2500] * 19, [1] * 19), ([2500] * 20, [1] * 20),
                                     ([40000], [17]), ([12000], [20])])
def test_absorbed_joins(heads, lens, qs):
    """Few long items in many pieces, on both sides of the choice of the joining kernel."""
    c = lat_case(lens, qs, heads, seed=heads)
    lat_check(c, lat_run(c))


def test_padded_steps_leave_other_rows():
    c = lat_case([40, 0, 300, 0], [1, 0, 3, 0], 16, pad=6)
    out = torch.full((10, 16, 512), 7.0, dtype=BF, device="cuda")
    lat_run(c, out=out)
    lat_check(c, out)
    assert (out[4:] == 7).all()
    e = exp_case([40, 0, 300, 0], [1, 0, 3, 0], 4, pad=6)
    out = torch.full((10, 4, 128), 7.0, dtype=BF, device="cuda")
    exp_run(e, out=out)
    exp_check(e, out)
    assert (out[4:] == 7).all()


BOUNDS = pkv._binding.PKV_ERR_DEVICE_BOUNDS


def test_bad_lengths_and_blocks_are_reported():
    """What the checks turn into an error: the request is skipped, the others are served."""
    c = lat_case([40, 50, 60, 70], [1, 1, 1, 1], 8)
    good = lat_run(c)
    for r, n in ((1, 0), (1, -5), (2, 10 ** 6)):
        bad = dict(c, lens=c["lens"].copy())
        bad["lens"][r] = n
        out = torch.full((4, 8, 512), 7.0, dtype=BF, device="cuda")
        lat_run(bad, out=out)
        assert pkv.pkv_get_device_error() == BOUNDS
        rest = [i for i in range(4) if i != r]
        assert (out[r] == 7).all() and torch.equal(out[rest], good[rest])
    bad = dict(c, tab=c["tab"].copy())
    bad["tab"][3, 2] = c["pool"].shape[0]
    out = lat_run(bad)
    assert pkv.pkv_get_device_error() == BOUNDS and torch.equal(out[:3], good[:3])
    bad["tab"][3, 2] = -1
    lat_run(bad)
    assert pkv.pkv_get_device_error() == BOUNDS

    n, w = 220, torch.randn(2, 256, 512, device="cuda").to(BF)
    kv, kr = (torch.full(s, 7.0, dtype=BF, device="cuda") for s in ((n, 2, 256), (n, 64)))
    args = (dev(c["tab"], torch.int32), dev(c["lens"], torch.int32))
    ksl = [0, 40, 90, 150, 220]
    pkv.pkv_expand_latent(c["pool"], w, *args, dev(ksl, torch.int32), kv, kr)
    want_kv, want_kr = kv.clone(), kr.clone()
    for starts, lost in (([0, 40, 89, 150, 220], (40, 150)), ([-1, 40, 90, 150, 220], (0, 40)), ([0, 40, 90, 150, 221], (150, 220))):
        kv.fill_(7), kr.fill_(7)
        pkv.pkv_expand_latent(c["pool"], w, *args, dev(starts, torch.int32), kv, kr)
        assert pkv.pkv_get_device_error() == BOUNDS
        live = np.r_[0:lost[0], lost[1]:220]
        assert (kv[lost[0]:lost[1]] == 7).all() and torch.equal(kv[live], want_kv[live]) and torch.equal(kr[live], want_kr[live])

    e = exp_case([40, 50, 60], [2, 50, 7], 2)
    good = exp_run(e)
    for key, i, v in (("lens", 1, 51), ("ksl", 3, 151), ("qsl", 3, 60), ("ksl", 0, -1)):
        bad = dict(e, **{key: e[key].copy()})
        bad[key][i] = v
        out = torch.full_like(good, 7)
        exp_run(bad, out=out)
        assert pkv.pkv_get_device_error() == BOUNDS
        r = i if key == "lens" else 2 if i == 3 else 0
        assert (out[e["qsl"][r]:e["qsl"][r + 1]] == 7).all()
        for o in range(3):
            if o != r:
                assert torch.equal(out[e["qsl"][o]:e["qsl"][o + 1]], good[e["qsl"][o]:e["qsl"][o + 1]])


def test_repeated_calls_agree():
    """The same call again and again, from a cache that is in L2 by then: the same
    bits every time (no order of arrival changes a sum)."""
    for c, run in ((lat_case([512] * 64, [1] * 64, 16), lat_run), (lat_case([700] * 100, [1] * 100, 128), lat_run),
                   (lat_case([64] * 200, [1] * 200, 33), lat_run), (lat_case([900, 5000], [5, 1], 16), lat_run),
                   (exp_case([600] * 8, [512] * 8, 16), exp_run), (exp_case([3000], [100], 2), exp_run)):
        ws = pkv.LatentWorkspace()
        first = run(c, workspace=ws).clone()
        for _ in range(60):
            assert torch.equal(run(c, workspace=ws), first)
        assert pkv.pkv_get_device_error() == 0


def test_one_workspace_serves_all_calls():
    """Calls of different sizes and kinds, one after the other on one workspace, on a
    stream that is not the current one."""
    ws, s = pkv.LatentWorkspace(), torch.cuda.Stream()
    cases = [(lat_case([3000, 20], [1, 3], 16), lat_run, lat_check), (exp_case([2000], [50], 2), exp_run, exp_check),
             (lat_case([5], [1], 128), lat_run, lat_check), (exp_case([300] * 3, [256] * 3, 3), exp_run, exp_check),
             (lat_case([900] * 20, [1] * 20, 64), lat_run, lat_check)]
    torch.cuda.synchronize()
    tensors = [[dev(c[k], torch.int32) for k in (("tab", "lens", "qsl") if "tab" in c else ("lens", "qsl", "ksl"))]
               for c, _, _ in cases]
    results = [torch.empty(*c["q"].shape[:2], 512 if "tab" in c else 128, dtype=BF, device="cuda") for c, _, _ in cases]
    torch.cuda.synchronize()
    for _ in range(2):
        for (c, _, _), t, out in zip(cases, tensors, results):
            if "tab" in c:
                pkv.pkv_attention_latent(c["q"], c["pool"], *t, c["scale"], out=out, workspace=ws, stream=s)
            else:
                pkv.pkv_attention_expanded(c["q"], c["kv"], c["kr"], *t, c["scale"], out=out, workspace=ws, stream=s)
    s.synchronize()
    for (c, _, check), out in zip(cases, results):
        check(c, out)


def test_without_a_workspace_on_another_stream():
    c, s = lat_case([3000, 20], [1, 3], 16), torch.cuda.Stream()
    t = [dev(c[k], torch.int32) for k in ("tab", "lens", "qsl")]
    out = torch.empty(4, 16, 512, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    pkv.pkv_attention_latent(c["q"], c["pool"], *t, c["scale"], out=out, stream=s)
    s.synchronize()
    lat_check(c, out)


@pytest.mark.parametrize("option", [dict(pdl=0), dict(early_plan=0)])
def test_launch_options(pkv_opts, option):
    pkv_opts(**option)
    c = lat_case([3000, 20, 77], [1, 3, 1], 16)
    lat_check(c, lat_run(c))
    c = lat_case([900] * 30, [1] * 30, 100)
    lat_check(c, lat_run(c))
    e = exp_case([2000, 5], [50, 5], 2)
    exp_check(e, exp_run(e))


def test_timeout_ends_the_call(pkv_opts):
    """With a limit of a microsecond waits run out: the calls return, report it, and the
    next ones (the workspace's head zeroed again) are right."""
    c, e = lat_case([5000] * 4, [1] * 4, 128), exp_case([3000], [300], 4)
    p = exp_case([600] * 8, [512] * 8, 16)
    ws = pkv.LatentWorkspace()
    saved = pkv.get_options()["wait_limit_us"]
    for run, case in ((lat_run, c), (exp_run, e), (exp_run, p)):
        pkv.set_options(wait_limit_us=1)
        for _ in range(3):
            run(case, workspace=ws)
        assert pkv.pkv_get_device_error() in (0, pkv._binding.PKV_ERR_TIMEOUT)
        pkv.set_options(wait_limit_us=saved)
        ws = pkv.LatentWorkspace()
    lat_check(c, lat_run(c, workspace=ws))
    exp_check(e, exp_run(e, workspace=ws))
    exp_check(p, exp_run(p, workspace=ws))
