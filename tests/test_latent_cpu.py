"""Host-side tests of the latent cache's operators and of the norm and rotation
ahead of the append: the plain 64-bit implementations against closed forms and
each other, and the refusals of the C ABI and the binding (nothing here reaches a
GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_195_gb300 as pkv
from paged_kv_cache_195_gb300 import _binding as b
from paged_kv_cache_195_gb300 import build as pkv_build

import lat_reference as ref


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


# ------------------------------------------------------------ the references
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_rotation_is_a_complex_product(rot, inter):
    rng = np.random.default_rng(rot)
    x, pos = rng.normal(size=(5, 3, 128)), np.array([0, 1, 7, 100, 4999])
    y, size = ref.rotate(x, ref.table(5000, rot)[pos], inter)
    lead = x[..., :rot]
    z = lead[..., 0::2] + 1j * lead[..., 1::2] if inter else lead[..., :rot // 2] + 1j * lead[..., rot // 2:]
    turn = z * np.exp(1j * pos[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot))[:, None]
    got = y[..., 0:rot:2] + 1j * y[..., 1:rot:2] if inter else y[..., :rot // 2] + 1j * y[..., rot // 2:rot]
    assert np.abs(got - turn).max() < 1e-6  # (the table is fp32)
    assert (y[..., rot:] == x[..., rot:]).all() and (np.abs(y) <= size + 1e-12).all()


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(0).normal(size=(4, 512)) * 10
    assert np.allclose(np.square(ref.norm(x, 1.0, 0.0)).mean(-1), 1)
    assert np.allclose(ref.norm(np.zeros(128), 3.0, 1e-6), 0)


def _case(seed, lens, qs, heads):
    rng = np.random.default_rng(seed)
    nb = [ref.cdiv(n, 16) for n in lens]
    ids = rng.permutation(sum(nb) + 2)
    tab = np.full((len(lens), max(nb)), -1)
    for r in range(len(lens)):
        tab[r, :nb[r]] = ids[sum(nb[:r]):sum(nb[:r + 1])]
    return (rng.normal(size=(sum(nb) + 2, 16, 576)), tab, np.concatenate([[0], np.cumsum(qs)]),
            rng.normal(size=(heads, 256, 512)) / 20, rng.normal(size=(sum(qs), heads, 192)))


def test_the_two_forms_agree():
    """q^T (W c) = (W^T q)^T c, and the sum of W c is W of the sum."""
    lens, qs = [5, 40, 17], [2, 1, 17]
    pool, tab, qsl, w, q = _case(1, lens, qs, 3)
    kv, rope, bound = ref.expand(pool, w, tab, lens)
    one, b1 = ref.expanded(q, kv, rope, lens, qsl, 0.07)
    taken = np.concatenate([np.einsum("thd,hdc->thc", q[..., :128], w[:, :128]), q[..., 128:]], -1)
    lat, b2 = ref.absorbed(taken, pool, tab, lens, qsl, 0.07)
    two = np.einsum("thc,hdc->thd", lat, w[:, 128:])
    assert np.abs(one - two).max() < 1e-12 * np.abs(one).max()
    for bb, o in ((b1, one), (b2, lat)):
        assert (bb > 0).all() and bb.max() < 0.03 * np.abs(o).max()
    assert (bound < 0.01 * np.abs(kv).max()).all()


def test_attention_is_softmax_attention():
    lens, qs = [40], [40]
    pool, tab, qsl, w, q = _case(2, lens, qs, 2)
    kv, rope, _ = ref.expand(pool, w, tab, lens)
    one, _ = ref.expanded(q, kv, rope, lens, qsl, 0.3)
    t = torch.from_numpy
    k = np.concatenate([kv[..., :128], np.repeat(rope[:, None], 2, 1)], -1)
    want = torch.nn.functional.scaled_dot_product_attention(
        t(q).transpose(0, 1), t(k).transpose(0, 1), t(np.ascontiguousarray(kv[..., 128:])).transpose(0, 1),
        is_causal=True, scale=0.3).transpose(0, 1).numpy()
    assert np.abs(one - want).max() < 1e-12


def test_references_keep_what_a_row_does_not_see_out():
    lens, qs = [20], [4]
    pool, tab, qsl, w, q = _case(3, lens, qs, 2)
    clean = ref.absorbed(np.zeros((4, 2, 576)) + 0.1, pool, tab, lens, qsl, 0.1)[0]
    pool[tab[0, 1], 2, 9] = np.nan  # position 18: the third token's
    pool[tab[0, 1], 4:] = np.nan    # behind the end
    got = ref.absorbed(np.zeros((4, 2, 576)) + 0.1, pool, tab, lens, qsl, 0.1)[0]
    assert (got[:2] == clean[:2]).all() and np.isnan(got[2:]).all()
    kv, rope, _ = ref.expand(pool, w, tab, lens)
    assert np.isnan(kv[18]).all() and np.isfinite(np.delete(kv, 18, 0)).all()
    o, _ = ref.expanded(q, kv, rope, lens, qsl, 0.1)
    assert np.isfinite(o[:2]).all() and np.isnan(o[2:]).all()


# ------------------------------------------------------------ refusals: the C ABI
FAKE = 0x1000  # never dereferenced: validation fails first
ODD = FAKE + 8


def _dims(**kw):
    d = dict(num_reqs=2, num_q_tokens=2, num_q_heads=16, num_kv_heads=1, head_dim=576, block_size=16, num_blocks=8,
             max_blocks_per_req=4)
    d.update(kw)
    return b.Dims(*[d[f] for f, _ in b.Dims._fields_])


def _rope(lib, q=FAKE, k=FAKE << 8, v=FAKE << 8, qs=2048, ks=256, vs=256, pos=FAKE, cs=FAKE, n=100, rot=128, wq=None, wk=None,
          eps=1e-6, slots=FAKE, out=FAKE, os_=2048, kp=FAKE, vp=FAKE, **kw):
    d = _dims(**{"num_kv_heads": 2, "head_dim": 128, **kw})
    return lib.pkv_norm_rope_append(q, k, v, qs, ks, vs, pos, cs, n, rot, 0, wq, wk, eps, slots, out, os_, kp, vp,
                                    ctypes.byref(d), None)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=64), b.PKV_ERR_UNSUPPORTED), (dict(block_size=32), b.PKV_ERR_UNSUPPORTED),
    (dict(num_q_tokens=-1), b.PKV_ERR_INVALID), (dict(num_q_heads=-1), b.PKV_ERR_INVALID),
    (dict(num_q_heads=4097), b.PKV_ERR_UNSUPPORTED), (dict(num_kv_heads=4097), b.PKV_ERR_UNSUPPORTED),
    (dict(rot=0), b.PKV_ERR_UNSUPPORTED), (dict(rot=24), b.PKV_ERR_UNSUPPORTED), (dict(rot=144), b.PKV_ERR_UNSUPPORTED),
    (dict(wq=FAKE, eps=0.0), b.PKV_ERR_INVALID), (dict(wk=FAKE, eps=float("nan")), b.PKV_ERR_INVALID),
    (dict(wk=FAKE, eps=2.0), b.PKV_ERR_INVALID), (dict(wk=FAKE, eps=-1e-6), b.PKV_ERR_INVALID),
    *[({name: None}, b.PKV_ERR_INVALID) for name in ("q", "k", "v", "pos", "cs", "slots", "out", "kp", "vp")],
    *[({name: ODD}, b.PKV_ERR_INVALID) for name in ("q", "k", "v", "cs", "out", "kp", "vp", "wq", "wk")],
    (dict(qs=2040), b.PKV_ERR_INVALID), (dict(qs=2052), b.PKV_ERR_INVALID), (dict(ks=255), b.PKV_ERR_INVALID),
    (dict(vs=0), b.PKV_ERR_INVALID), (dict(os_=-2048), b.PKV_ERR_INVALID),
    # q_out over the inputs: another stride, k's and v's rows, parts of one tensor that overlap
    (dict(os_=4096), b.PKV_ERR_INVALID), (dict(out=FAKE + 16), b.PKV_ERR_INVALID), (dict(out=FAKE << 8), b.PKV_ERR_INVALID),
    (dict(qs=2560, ks=2560, os_=2560, k=FAKE + 4080), b.PKV_ERR_INVALID),
    (dict(qs=2560, vs=2560, os_=2560, v=FAKE + 5120 - 496), b.PKV_ERR_INVALID)])
def test_norm_rope_append_refuses(lib, kw, code):
    assert _rope(lib, **kw) == code and lib.pkv_last_error()


def _append(lib, kv=FAKE, stride=576, pos=FAKE, cs=FAKE, n=100, w=None, eps=1e-6, slots=FAKE, pool=FAKE, q=None, qs=1024,
            qh=64, out=None, os_=1024, oh=64, **kw):
    return lib.pkv_append_latent(kv, stride, pos, cs, n, 0, w, eps, slots, pool, q, qs, qh, out, os_, oh,
                                 ctypes.byref(_dims(**kw)), None)


LATENT_DIMS = [(dict(head_dim=128), b.PKV_ERR_UNSUPPORTED), (dict(num_kv_heads=2), b.PKV_ERR_UNSUPPORTED),
               (dict(block_size=8), b.PKV_ERR_UNSUPPORTED), (dict(num_q_heads=-1), b.PKV_ERR_INVALID),
               (dict(num_blocks=-1), b.PKV_ERR_INVALID), (dict(num_blocks=1 << 27), b.PKV_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", [
    *LATENT_DIMS, (dict(num_q_heads=4097), b.PKV_ERR_UNSUPPORTED), (dict(num_q_tokens=-1), b.PKV_ERR_INVALID),
    (dict(w=FAKE, eps=0.0), b.PKV_ERR_INVALID), (dict(w=FAKE, eps=float("inf")), b.PKV_ERR_INVALID),
    *[({name: None}, b.PKV_ERR_INVALID) for name in ("kv", "pos", "cs", "slots", "pool")],
    *[({name: ODD}, b.PKV_ERR_INVALID) for name in ("kv", "cs", "pool", "w")],
    (dict(q=ODD, out=FAKE), b.PKV_ERR_INVALID), (dict(q=FAKE, out=ODD), b.PKV_ERR_INVALID),
    (dict(q=FAKE, out=None), b.PKV_ERR_INVALID), (dict(q=FAKE, out=FAKE, qs=1028), b.PKV_ERR_INVALID),
    (dict(q=FAKE, out=FAKE, oh=-64), b.PKV_ERR_INVALID), (dict(q=FAKE, out=FAKE, oh=32), b.PKV_ERR_INVALID),
    (dict(q=FAKE, out=FAKE, os_=64), b.PKV_ERR_INVALID), (dict(q=FAKE, out=FAKE, os_=0), b.PKV_ERR_INVALID),
    (dict(q=FAKE, out=FAKE, os_=1016), b.PKV_ERR_INVALID), (dict(q=FAKE, out=FAKE, oh=0), b.PKV_ERR_INVALID),
    (dict(q=FAKE, out=FAKE, qs=2048), b.PKV_ERR_INVALID), (dict(q=FAKE, out=FAKE + 128), b.PKV_ERR_INVALID),
    (dict(q=FAKE + 4080, out=FAKE), b.PKV_ERR_INVALID), (dict(q=FAKE, out=FAKE, os_=1 << 62, qs=1 << 62, oh=72), b.PKV_ERR_INVALID),
    (dict(stride=568), b.PKV_ERR_INVALID),
    (dict(stride=580), b.PKV_ERR_INVALID)])
def test_append_latent_refuses(lib, kw, code):
    assert _append(lib, **kw) == code and lib.pkv_last_error()


def _absorbed(lib, q=FAKE, pool=FAKE, tab=FAKE, lens=FAKE, qsl=FAKE, scale=0.1, out=FAKE, ws=FAKE, **kw):
    return lib.pkv_attention_latent(q, pool, tab, lens, qsl, scale, out, ctypes.byref(_dims(**kw)), ws, 1 << 40, None)


SCALES = [dict(scale=s) for s in (0.0, -0.1, float("inf"), float("nan"))]


@pytest.mark.parametrize("kw,code", [
    *LATENT_DIMS, (dict(num_q_heads=129), b.PKV_ERR_UNSUPPORTED), (dict(num_q_heads=0), b.PKV_ERR_INVALID),
    (dict(num_reqs=-1), b.PKV_ERR_INVALID), (dict(num_blocks=0), b.PKV_ERR_INVALID),
    *[({name: None}, b.PKV_ERR_INVALID) for name in ("q", "pool", "tab", "lens", "qsl", "out", "ws")],
    *[({name: ODD}, b.PKV_ERR_INVALID) for name in ("q", "pool", "out")], *[(s, b.PKV_ERR_INVALID) for s in SCALES]])
def test_absorbed_attention_refuses(lib, kw, code):
    assert _absorbed(lib, **kw) == code and lib.pkv_last_error()


def _expand(lib, pool=FAKE, w=FAKE, tab=FAKE, lens=FAKE, ksl=FAKE, kv=FAKE, kr=FAKE, rows=50, **kw):
    return lib.pkv_expand_latent(pool, w, tab, lens, ksl, kv, kr, rows, ctypes.byref(_dims(**kw)), None)


@pytest.mark.parametrize("kw,code", [
    *LATENT_DIMS, (dict(num_q_heads=4097), b.PKV_ERR_UNSUPPORTED), (dict(num_q_heads=0), b.PKV_ERR_INVALID),
    (dict(rows=-1), b.PKV_ERR_INVALID), (dict(num_blocks=0), b.PKV_ERR_INVALID),
    *[({name: None}, b.PKV_ERR_INVALID) for name in ("pool", "w", "tab", "lens", "ksl", "kv", "kr")],
    *[({name: ODD}, b.PKV_ERR_INVALID) for name in ("pool", "w", "kv", "kr")]])
def test_expand_refuses(lib, kw, code):
    assert _expand(lib, **kw) == code and lib.pkv_last_error()


def _expanded(lib, q=FAKE, kv=FAKE, kr=FAKE, lens=FAKE, qsl=FAKE, ksl=FAKE, scale=0.1, out=FAKE, rows=50, ws=FAKE, **kw):
    return lib.pkv_attention_expanded(q, kv, kr, lens, qsl, ksl, scale, out, rows, ctypes.byref(_dims(**kw)), ws, 1 << 40,
                                      None)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=192), b.PKV_ERR_UNSUPPORTED), (dict(num_q_heads=4097), b.PKV_ERR_UNSUPPORTED),
    (dict(num_q_heads=0), b.PKV_ERR_INVALID), (dict(rows=-1), b.PKV_ERR_INVALID), (dict(rows=0), b.PKV_ERR_INVALID),
    *[({name: None}, b.PKV_ERR_INVALID) for name in ("q", "kv", "kr", "lens", "qsl", "ksl", "out", "ws")],
    *[({name: ODD}, b.PKV_ERR_INVALID) for name in ("q", "kv", "kr", "out")], *[(s, b.PKV_ERR_INVALID) for s in SCALES]])
def test_expanded_attention_refuses(lib, kw, code):
    assert _expanded(lib, **kw) == code and lib.pkv_last_error()


def test_empty_steps_are_no_ops(lib):
    none = dict(num_q_tokens=0)
    assert _rope(lib, q=None, k=None, **none) == 0 and _append(lib, kv=None, **none) == 0
    assert _absorbed(lib, q=None, **none) == 0 and _absorbed(lib, q=None, num_reqs=0) == 0
    assert _expand(lib, pool=None, num_reqs=0) == 0 and _expand(lib, kv=None, rows=0) == 0
    assert _expanded(lib, q=None, **none) == 0 and _expanded(lib, q=None, num_reqs=0, rows=0) == 0


def test_workspace_size_refuses_other_dims(lib):
    assert lib.pkv_latent_workspace_size(ctypes.byref(_dims(head_dim=128))) == 0
    assert lib.pkv_last_error()


# ------------------------------------------------------------ refusals: the binding
def test_the_binding_refuses_cpu_tensors():
    BF, z = torch.bfloat16, torch.zeros
    i32, i64 = z(2, dtype=torch.int32), z(2, dtype=torch.int64)
    tab, qsl = z(2, 4, dtype=torch.int32), z(3, dtype=torch.int32)
    pool, cs = z(8, 16, 576, dtype=BF), z(10, 64)
    with pytest.raises(ValueError):
        pkv.pkv_norm_rope_append(z(2, 4, 128, dtype=BF), z(2, 1, 128, dtype=BF), z(2, 1, 128, dtype=BF), i64, cs, i64,
                                 z(8, 1, 16, 128, dtype=BF), z(8, 1, 16, 128, dtype=BF))
    with pytest.raises(ValueError):
        pkv.pkv_append_latent(z(2, 576, dtype=BF), i64, cs, i64, pool)
    with pytest.raises(ValueError):
        pkv.pkv_attention_latent(z(2, 16, 576, dtype=BF), pool, tab, i32, qsl, 0.1)
    with pytest.raises(ValueError):
        pkv.pkv_expand_latent(pool, z(4, 256, 512, dtype=BF), tab, i32, qsl, z(9, 4, 256, dtype=BF), z(9, 64, dtype=BF))
    with pytest.raises(ValueError):
        pkv.pkv_attention_expanded(z(2, 4, 192, dtype=BF), z(9, 4, 256, dtype=BF), z(9, 64, dtype=BF), i32, qsl, qsl, 0.1)
    for call in (pkv.pkv_norm_rope_append, pkv.pkv_append_latent, pkv.pkv_attention_latent, pkv.pkv_expand_latent,
                 pkv.pkv_attention_expanded):
        with pytest.raises((TypeError, ValueError)):
            call(*[[1.0]] * 8)
