"""A mixed step over a latent cache, split between the two forms as the header says:
decodes ahead of chunks, each form given its part of the step's arrays."""
import numpy as np
import pytest
import torch

import paged_kv_cache_195_gb300 as pkv
from paged_kv_cache_195_gb300 import build as pkv_build

import lat_reference as ref
from test_gpu_latent import close, dev, f64, lat_case

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    pkv.load_library()


@pytest.mark.parametrize("lens,qs,D,heads", [
    ([70, 1, 300, 200, 64, 33], [1, 1, 1, 150, 64, 5], 3, 16), ([2000, 40, 900, 700], [1, 2, 300, 700], 2, 5)])
def test_decodes_absorbed_and_chunks_expanded(lens, qs, D, heads):
    g = torch.Generator().manual_seed(D)
    c = lat_case(lens, qs, heads)
    w = (torch.randn(heads, 256, 512, generator=g) / 20).to(BF).cuda()
    T, qsl = sum(qs), c["qsl"]
    tab, n, starts = dev(c["tab"], I32), dev(lens, I32), dev(qsl, I32)
    d = int(qsl[D])  # the decodes' rows
    lat = pkv.pkv_attention_latent(c["q"][:d], c["pool"], tab[:D], n[:D], starts[:D + 1], c["scale"])
    want, bound = ref.absorbed(f64(c["q"][:d]), f64(c["pool"]), c["tab"][:D], lens[:D], qsl[:D + 1], c["scale"])
    close(lat, want, bound, "decodes")

    q = torch.randn(T, heads, 192, generator=g).to(BF).cuda()
    rows = torch.zeros(len(lens) - D + 1, dtype=I32, device="cuda")
    torch.cumsum(n[D:], 0, dtype=I32, out=rows[1:])
    kv = torch.empty(sum(lens[D:]), heads, 256, dtype=BF, device="cuda")
    kr = torch.empty(sum(lens[D:]), 64, dtype=BF, device="cuda")
    pkv.pkv_expand_latent(c["pool"], w, tab[D:], n[D:], rows, kv, kr)
    out = pkv.pkv_attention_expanded(q[d:], kv, kr, n[D:], starts[D:] - starts[D], rows, c["scale"])
    want, bound = ref.expanded(f64(q[d:]), f64(kv), f64(kr), lens[D:], np.array(qsl[D:]) - d, c["scale"])
    close(out, want, bound, "chunks")
    kv64, _, kv_bound = ref.expand(f64(c["pool"]), f64(w), c["tab"][D:], lens[D:])
    close(kv, kv64, kv_bound, "kv")
    assert pkv.pkv_get_device_error() == 0
