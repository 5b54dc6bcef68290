"""Calls over a latent cache whose waits run out: the testing option debug_withhold_q
keeps the kernels from loading what their first products need, so that every wait
ends by its limit.  The calls come back, report PKV_ERR_TIMEOUT, write nothing but
the step's own rows, and the next calls are right.  Nothing here faults or traps the
GPU: the kernels stop waiting by themselves."""
import time

import numpy as np
import pytest
import torch

import paged_kv_cache_195_gb300 as pkv
from paged_kv_cache_195_gb300 import build as pkv_build

import lat_reference as ref
from test_gpu_latent import close, dev, exp_case, exp_check, exp_run, f64, lat_case, lat_check, lat_run

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
GUARD = 64  # rows behind a step's


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


def withheld(pkv_opts, call):
    """`call` with the first loads withheld: it must come back, with a timeout."""
    torch.cuda.synchronize()
    assert pkv.pkv_get_device_error() == 0
    saved = pkv.get_options()
    pkv_opts(wait_limit_us=1000, debug_withhold_q=1)
    t0 = time.perf_counter()
    call()
    rc = pkv.pkv_get_device_error()  # synchronises the stream
    pkv_opts(wait_limit_us=saved["wait_limit_us"], debug_withhold_q=0)
    assert rc == pkv._binding.PKV_ERR_TIMEOUT, (rc, pkv.pkv_last_error())
    assert time.perf_counter() - t0 < 10


def stale_workspace(tokens):
    """A workspace full of records of some earlier call: items of one piece each, whose
    rows would be the guard's of the step at hand."""
    ws = pkv.LatentWorkspace()
    off = ws.ptr - ws.buf.data_ptr()
    words = ws.buf[off:off + ws.nbytes // 16 * 16].view(torch.int32)
    records = 256 // 4, 256 // 4 + 2 * 8 * torch.cuda.get_device_properties(0).multi_processor_count
    words[32] = 2 * torch.cuda.get_device_properties(0).multi_processor_count  # (the count of pieces)
    words[records[0]:records[1]] = torch.tensor([1, tokens, 4, 0], dtype=torch.int32,
                                                device="cuda").repeat((records[1] - records[0]) // 4)
    words[records[1]:] = 0x3f800000  # 1.0
    return ws


def pieces(tiles, ctas):
    """Pieces that the expanded form cuts items of so many key tiles into."""
    least = max(2, -(-sum(tiles) // ctas))
    n = lambda s: sum(-(-t // s) for t in tiles)
    for s in range(least, 2 * least, (least + 7) // 8):
        if n(s) <= ctas:
            return n(s)
    return n(least)


@pytest.mark.parametrize("lens,qs,heads", [
    ([250] * 80 + [44 * 128] * 20, [1] * 100, 1),  # more pieces than CTAs: some are never taken
    ([3000], [300], 4), ([6000], [1], 1),          # split, a CTA each
    ([300, 20], [100, 20], 3),                     # whole
    ([600] * 8, [512] * 8, 16)])                   # in pairs
def test_expanded_form_without_its_queries(pkv_opts, lens, qs, heads):
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    if len(lens) == 100:
        assert 3 * len(lens) < 2 * ctas < 2 * pieces([-(-n // 128) for n in lens], ctas)
    c = exp_case(lens, qs, heads)
    T = sum(qs)
    ws = stale_workspace(T)
    out = torch.full((T + GUARD, heads, 128), 7.0, dtype=BF, device="cuda")
    withheld(pkv_opts, lambda: exp_run(c, out=out[:T], workspace=ws))
    assert (out == 7).all(), "an aborted call wrote output"
    ws.buf[:ws.ptr - ws.buf.data_ptr() + 128].zero_()
    for _ in range(2):  # TMEM and the aborted CTAs' state are gone
        exp_check(c, exp_run(c, out=out[:T], workspace=ws))
        assert (out[T:] == 7).all()


@pytest.mark.parametrize("lens,qs,heads", [
    ([5000] * 4, [1] * 4, 128), ([32768], [1], 16),  # few rows, in pieces
    ([900] * 200, [1] * 200, 100),                   # ranges that cut rows
    ([17, 64, 100, 128], [1] * 4, 16),               # whole
    ([300, 70, 0, 9], [60, 5, 0, 1], 16)])
def test_absorbed_form_without_its_queries(pkv_opts, lens, qs, heads):
    c = lat_case(lens, qs, heads)
    T = sum(qs)
    ws = stale_workspace(T)
    out = torch.full((T + GUARD, heads, 512), 7.0, dtype=BF, device="cuda")
    withheld(pkv_opts, lambda: lat_run(c, out=out[:T], workspace=ws))
    assert (out == 7).all(), "an aborted call wrote output"
    for _ in range(2):
        lat_check(c, lat_run(c, out=out[:T], workspace=ws))
        assert (out[T:] == 7).all()


@pytest.mark.parametrize("lens,heads", [([701], 16), ([17, 64, 0, 300], 1), ([3000] * 4, 32)])
def test_expansion_without_its_weights(pkv_opts, lens, heads):
    c, n = lat_case(lens, [0] * len(lens), 1), sum(lens)
    w = (torch.randn(heads, 256, 512, generator=torch.Generator().manual_seed(1)) / 20).to(BF).cuda()
    kv = torch.full((n + GUARD, heads, 256), 7.0, dtype=BF, device="cuda")
    kr = torch.full((n + GUARD, 64), 7.0, dtype=BF, device="cuda")
    args = [dev(x, torch.int32) for x in (c["tab"], c["lens"], np.concatenate([[0], np.cumsum(lens)]))]
    withheld(pkv_opts, lambda: pkv.pkv_expand_latent(c["pool"], w, *args, kv, kr))
    assert (kv == 7).all() and (kr[n:] == 7).all()  # (the rotated keys need no weights)
    pkv.pkv_expand_latent(c["pool"], w, *args, kv, kr)
    want, rope, bound = ref.expand(f64(c["pool"]), f64(w), c["tab"], lens)
    close(f64(kv)[:n], want, bound)
    assert np.array_equal(f64(kr)[:n], rope) and (kv[n:] == 7).all() and (kr[n:] == 7).all()
