"""Calls over a latent cache right behind the kernel that writes what they plan by: the
running sum of the lengths, computed on the stream, other ones each time."""
import pytest
import torch

import paged_kv_cache_195_gb300 as pkv
from paged_kv_cache_195_gb300 import build as pkv_build

from test_gpu_latent import dev, exp_case, lat_case

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


def steps(lengths, call, out):
    """`call(lens, sums)` with each step's lengths, first waited for, then all in a row:
    the same results."""
    lens, sums = dev(lengths[0], torch.int32), torch.zeros(len(lengths[0]) + 1, dtype=torch.int32, device="cuda")
    sets = [dev(n, torch.int32) for n in lengths]
    want = []
    for n in sets:
        lens.copy_(n)
        torch.cumsum(lens, 0, dtype=torch.int32, out=sums[1:])
        torch.cuda.synchronize()
        [o.fill_(7) for o in out]
        torch.cuda.synchronize()
        call(lens, sums)
        want.append([o.clone() for o in out])
    assert not torch.equal(want[0][0], want[1][0])
    got = []
    for i in range(40):
        [o.fill_(7) for o in out]
        lens.copy_(sets[i % len(sets)])
        torch.cumsum(lens, 0, dtype=torch.int32, out=sums[1:])
        call(lens, sums)
        got.append([o.clone() for o in out])
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % len(sets)])), i


@pytest.mark.parametrize("lengths", [[[700, 1], [1, 700]], [[100, 0, 900, 33], [33, 900, 0, 100], [516, 517, 0, 0]],
                                     [[20 + i % 7 for i in range(300)], [26 - i % 7 for i in range(300)]]])
def test_sums_ahead_of_the_expansion(lengths):
    R, heads = len(lengths[0]), 4
    c = lat_case([max(n) for n in zip(*lengths)], [0] * R, 1)
    rows = max(map(sum, lengths)) + 40
    g = torch.Generator().manual_seed(1)
    w, tab = (torch.randn(heads, 256, 512, generator=g) / 20).to(BF).cuda(), dev(c["tab"], torch.int32)
    kv, kr = torch.empty(rows, heads, 256, dtype=BF, device="cuda"), torch.empty(rows, 64, dtype=BF, device="cuda")
    steps(lengths, lambda lens, sums: pkv.pkv_expand_latent(c["pool"], w, tab, lens, sums, kv, kr), (kv, kr))


@pytest.mark.parametrize("heads,qs,lengths", [
    (2, [50, 1], [[2000, 1], [60, 1500]]), (3, [100, 0, 9], [[100, 50, 20], [300, 0, 9]]),
    (40, [256, 512], [[300, 900], [700, 520]])])
def test_sums_ahead_of_the_expanded_form(heads, qs, lengths):
    c = exp_case([max(n) for n in zip(*lengths)], qs, heads)
    ws, qsl = pkv.LatentWorkspace(), dev(c["qsl"], torch.int32)
    out = torch.empty(sum(qs), heads, 128, dtype=BF, device="cuda")
    steps(lengths, lambda lens, sums: pkv.pkv_attention_expanded(c["q"], c["kv"], c["kr"], lens, qsl, sums, c["scale"],
                                                                 out=out, workspace=ws), (out,))
