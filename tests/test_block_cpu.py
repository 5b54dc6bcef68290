"""Host-side tests of the block-scaled e4m3 cache's operators: the plain
64-bit implementations against closed forms and the fp64 oracle, and the
refusals of the C ABI and the binding (nothing here reaches a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_195_gb300 as pkv
from paged_kv_cache_195_gb300 import _binding as b
from paged_kv_cache_195_gb300 import build as pkv_build

import blk_reference as ref


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


# ------------------------------------------------------------ the references
def test_encode_agrees_with_the_oracle():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.normal(0, 1, 2000) * 2.0 ** rng.integers(-12, 11, 2000),
                        (ref._GRID[1:] + ref._GRID[:-1]) / 2, -(ref._GRID[1:] + ref._GRID[:-1]) / 2,
                        ref._GRID, [np.inf, -np.inf, 1e9, -0.0]])
    x = x.astype(np.float32).astype(np.float64)
    assert [int(c) for c in ref.encode(x)] == [oracle.e4m3_encode(float(v)) for v in x]
    assert ref.encode(np.array([np.nan]))[0] == 0x7F


@pytest.mark.parametrize("top,want", [(0.0, 2.0 ** -126), (448.0, 1.0), (449.0, 2.0), (3.5, 2.0 ** -7),
                                      (3.52, 2.0 ** -6), (3.3e38, 2.0 ** 120), (1e-40, 2.0 ** -126)])
def test_need_scale(top, want):
    assert ref.need_scale(top) == want


def test_append_keeps_and_rescales():
    # One head, one block: a token of size 1, then one of size 1000, then a restart.
    table, one = np.array([[3]]), np.ones((1, 1, 128))
    pools = [np.full((4, 1, 16, 128), 0x7F, np.uint8) for _ in range(2)]
    scales = [np.full((4, 1), np.nan, np.float32) for _ in range(2)]
    pools, scales = ref.append(one, -one, table, [1], [0, 1], pools, scales)
    assert scales[0][3, 0] == 2.0 ** -8 and (ref.E4M3[pools[0][3, 0, 0]] == 256).all()
    pools, scales = ref.append(1000 * one, 0 * one, table, [2], [0, 1], pools, scales)
    assert scales[0][3, 0] == 4 and (ref.E4M3[pools[0][3, 0, 0]] * 4 == 1).all()
    assert (ref.E4M3[pools[0][3, 0, 1]] == 256).all()  # 250 ties between 240 and 256's grid: 250 -> 256
    assert scales[1][3, 0] == 2.0 ** -8 and (ref.E4M3[pools[1][3, 0, 0]] == -256).all()
    pools, scales = ref.append(one, one, table, [1], [0, 1], pools, scales)
    assert scales[0][3, 0] == 2.0 ** -8
    assert (pools[0][[0, 1, 2]] == 0x7F).all() and (pools[0][3, 0, 2:] == 0x7F).all()


def test_attention_agrees_with_the_oracle_over_one_scale_per_head():
    rng = np.random.default_rng(2)
    lens, qsl, hq, hkv = [1, 17, 40], [0, 1, 2, 7], 6, 2
    table = np.array([[0, 9, 9], [1, 2, 9], [3, 4, 5]], np.int32)
    pools = [rng.integers(0, 120, (8, hkv, 16, 128)).astype(np.uint8) for _ in range(2)]
    per_head = [np.array([0.004, 0.003], np.float32), np.array([0.0035, 0.0041], np.float32)]
    scales = [np.tile(s, (8, 1)) for s in per_head]
    q = rng.normal(0, 1, (7, hq, 128))
    q = torch.tensor(q).bfloat16()
    out, bound = ref.attention(q.double().numpy(), pools, scales, table, lens, qsl, 0.09)
    want = oracle.paged_attention_fp8(q.view(torch.int16).numpy().view(np.uint16), pools[0], pools[1],
                                      per_head[0], per_head[1], table, np.array(lens, np.int32),
                                      np.array(qsl, np.int32), 0.09)
    assert np.abs(out - want).max() < 1e-6 * np.abs(want).max()
    assert (bound > 0).all() and (bound < 0.02 * np.abs(want).max()).all()


def test_build_and_release_are_inverse():
    table = np.full((3, 4), -1, np.int32)
    fl = np.arange(8, dtype=np.int32)
    t, lens, qsl, slots, left, refused = ref.build([0, 0, 0], [17, 0, 5], fl, 8, table, 24)
    assert lens.tolist() == [17, 0, 5] and qsl.tolist() == [0, 17, 17, 22] and (left, refused) == (5, 0)
    assert t[0, :2].tolist() == [7, 6] and t[2, 0] == 5 and slots[16] == 6 * 16 and slots[-2:].tolist() == [-1, -1]
    fl2, n = ref.release(t, lens, [0, 0, 0], fl, left)
    assert n == 8 and sorted(fl2.tolist()) == list(range(8))


# ------------------------------------------------------------ refusals
def _dims(**kw):
    d = dict(num_reqs=2, num_q_tokens=2, num_q_heads=12, num_kv_heads=2, head_dim=128,
             block_size=16, num_blocks=8, max_blocks_per_req=4)
    d.update(kw)
    return b.Dims(*[d[f] for f, _ in b.Dims._fields_])


FAKE = 0x1000  # never dereferenced: validation fails first


def _call(lib, name, d, null=None, odd=None):
    n = {"pkv_build_step": 10, "pkv_release_blocks": 6, "pkv_append_fp8_block": 9,
         "pkv_attention_fp8_block": 8}[name]
    args = [FAKE] * n
    if null is not None:
        args[null] = None
    if odd is not None:
        args[odd] = FAKE + 8
    if name == "pkv_attention_fp8_block":
        return lib.pkv_attention_fp8_block(*args, 0.1, FAKE, ctypes.byref(d), None, 0, None)
    return getattr(lib, name)(*args, ctypes.byref(d), None)


NAMES = ["pkv_build_step", "pkv_release_blocks", "pkv_append_fp8_block", "pkv_attention_fp8_block"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("kw,code", [(dict(block_size=32), b.PKV_ERR_UNSUPPORTED),
                                     (dict(num_reqs=-1), b.PKV_ERR_INVALID),
                                     (dict(num_q_tokens=-1), b.PKV_ERR_INVALID),
                                     (dict(max_blocks_per_req=-1), b.PKV_ERR_INVALID),
                                     (dict(max_blocks_per_req=1 << 27), b.PKV_ERR_UNSUPPORTED),
                                     (dict(num_reqs=70000), b.PKV_ERR_UNSUPPORTED)])
def test_bad_dims(lib, name, kw, code):
    assert _call(lib, name, _dims(**kw)) == code
    assert lib.pkv_last_error().decode()


@pytest.mark.parametrize("name", NAMES[:3])
def test_too_many_token_rows(lib, name):
    assert _call(lib, name, _dims(num_q_tokens=(1 << 30) + 1)) == b.PKV_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["pkv_append_fp8_block", "pkv_attention_fp8_block"])
@pytest.mark.parametrize("kw,code", [(dict(head_dim=64), b.PKV_ERR_UNSUPPORTED),
                                     (dict(num_kv_heads=0), b.PKV_ERR_INVALID)])
def test_bad_heads(lib, name, kw, code):
    assert _call(lib, name, _dims(**kw)) == code


@pytest.mark.parametrize("kw,code", [(dict(num_q_heads=13), b.PKV_ERR_INVALID),
                                     (dict(num_q_heads=18), b.PKV_ERR_UNSUPPORTED),
                                     (dict(num_blocks=1 << 26), b.PKV_ERR_UNSUPPORTED)])
def test_attention_dims(lib, kw, code):
    assert _call(lib, "pkv_attention_fp8_block", _dims(**kw)) == code


@pytest.mark.parametrize("name,args", [("pkv_build_step", [0, 1, 2, 3, 4, 5, 6, 7, 8]),
                                       ("pkv_release_blocks", range(6)),
                                       ("pkv_append_fp8_block", range(9)),
                                       ("pkv_attention_fp8_block", range(8))])
def test_null_pointers(lib, name, args):
    for i in args:
        assert _call(lib, name, _dims(), null=i) == b.PKV_ERR_INVALID, i


@pytest.mark.parametrize("name,args", [("pkv_append_fp8_block", (0, 1, 5, 6)),
                                       ("pkv_attention_fp8_block", (0, 1, 2))])
def test_misaligned(lib, name, args):
    for i in args:
        assert _call(lib, name, _dims(), odd=i) == b.PKV_ERR_INVALID, i


def test_empty_steps_are_no_ops(lib):
    for name in NAMES[2:]:
        assert _call(lib, name, _dims(num_reqs=0, num_q_tokens=0)) == b.PKV_OK


def _cpu():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kv = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    pool, sc = torch.zeros(4, 2, 16, 128, dtype=torch.uint8), torch.zeros(4, 2)
    return i, kv, pool, sc


def test_binding_refuses_cpu_tensors():
    i, kv, pool, sc = _cpu()
    with pytest.raises(ValueError):
        pkv.pkv_append_fp8_block(kv, kv, i(2, 4), i(2), i(3), pool, pool, sc, sc)
    with pytest.raises(ValueError):
        pkv.pkv_attention_fp8_block(torch.zeros(2, 4, 128, dtype=torch.bfloat16), pool, pool, sc, sc,
                                    i(2, 4), i(2), i(3), 0.1)
    with pytest.raises(ValueError):
        pkv.pkv_build_step(i(2), i(2), i(4), i(1), i(2, 4), i(2), i(3),
                           torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        pkv.pkv_release_blocks(i(2, 4), i(2), i(2), i(4), i(1))
    with pytest.raises(TypeError):
        pkv.pkv_release_blocks(None, i(2), i(2), i(4), i(1))
