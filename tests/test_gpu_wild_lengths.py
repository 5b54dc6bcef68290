"""Numbers on the device that are out of range.  Start offsets so far out that their
differences wrap: the requests are skipped, and nothing is written for them.  Blocks
outside the pool: keys of zeros."""
import pytest
import torch

import paged_kv_cache_195_gb300 as pkv
from paged_kv_cache_195_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
MOST, LEAST = 2 ** 31 - 1, -2 ** 31
# From the largest number to the smallest: MOST + 1 = LEAST, "one token"; and 20 further on.
WILD = [[0, MOST, LEAST, 4], [0, MOST - 9, LEAST + 10, 4]]


# (the tensor-core prefill of bf16 pools skips such a chunk without a word)
EITHER = (0, pkv._binding.PKV_ERR_DEVICE_BOUNDS)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    pkv.load_library()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def zeros(*shape):
    return torch.zeros(*shape, dtype=BF, device="cuda")


def untouched(*tensors, reports=(pkv._binding.PKV_ERR_DEVICE_BOUNDS,)):
    torch.cuda.synchronize()
    assert pkv.pkv_get_device_error() in reports
    assert all((t == 7).all() for t in tensors)


@pytest.mark.parametrize("start", WILD)
@pytest.mark.parametrize("heads", [1, 4, 8])
def test_attention(start, heads):
    n = start[2] - start[1] + 2 ** 32
    table = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    lens = i32(n, n, n)
    for hq, hkv in ((heads, 1), (2 * heads, 2)):
        q, out = zeros(64, hq, 128), torch.full((64, hq, 128), 7.0, dtype=BF, device="cuda")
        pool = zeros(4, hkv, 16, 128)
        pkv.pkv_attention(q, pool, pool, table, lens, i32(*start), 0.1, out=out)
        untouched(out, reports=EITHER)
        codes = torch.zeros(4, hkv, 16, 128, dtype=torch.uint8, device="cuda")
        ones = torch.ones(hkv, device="cuda")
        pkv.pkv_attention_fp8kv(q, codes, codes, ones, ones, table, lens, i32(*start), 0.1, out=out)
        untouched(out, reports=EITHER)
        scales = torch.ones(4, hkv, device="cuda")
        pkv.pkv_attention_fp8_block(q, codes, codes, scales, scales, table, lens, i32(*start), 0.1, out=out)
        untouched(out, reports=EITHER)


@pytest.mark.parametrize("start", WILD)
@pytest.mark.parametrize("heads", [1, 16, 128])
def test_latent_cache(start, heads):
    n = start[2] - start[1] + 2 ** 32
    table = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    lens = i32(n, n, n)
    pool = zeros(4, 16, 576)
    out = torch.full((64, heads, 512), 7.0, dtype=BF, device="cuda")
    pkv.pkv_attention_latent(zeros(64, heads, 576), pool, table, lens, i32(*start), 0.1, out=out)
    untouched(out)
    kv = torch.full((100, heads, 256), 7.0, dtype=BF, device="cuda")
    kr = torch.full((100, 64), 7.0, dtype=BF, device="cuda")
    pkv.pkv_expand_latent(pool, zeros(heads, 256, 512), table, lens, i32(*start), kv, kr)
    untouched(kv, kr)
    out = torch.full((64, heads, 128), 7.0, dtype=BF, device="cuda")
    rows = i32(0, n, 2 * n, 3 * n)
    for qsl, ksl in ((i32(*start), rows), (i32(0, 1, 2, 3), i32(*start)), (i32(*start), i32(*start))):
        pkv.pkv_attention_expanded(zeros(64, heads, 192), kv, kr, lens, qsl, ksl, 0.1, out=out)
        untouched(out)


@pytest.mark.parametrize("block", [-1, 9, MOST, LEAST])
def test_expansion_of_blocks_outside_the_pool(block):
    """Rows of zeros in kv and in k_rope, whatever they held."""
    g = torch.Generator().manual_seed(0)
    pool, w = (torch.randn(*s, generator=g).to(BF).cuda() for s in ((9, 16, 576), (3, 256, 512)))
    table = i32(*range(9)).reshape(1, 9).contiguous()
    kv = torch.full((150, 3, 256), 7.0, dtype=BF, device="cuda")
    kr = torch.full((150, 64), 7.0, dtype=BF, device="cuda")
    pkv.pkv_expand_latent(pool, w, table, i32(141), i32(0, 141), kv, kr)
    assert pkv.pkv_get_device_error() == 0
    want = kv.clone(), kr.clone()
    table[0, 1] = table[0, 8] = block
    kv.fill_(7), kr.fill_(7)
    pkv.pkv_expand_latent(pool, w, table, i32(141), i32(0, 141), kv, kr)
    assert pkv.pkv_get_device_error() == pkv._binding.PKV_ERR_DEVICE_BOUNDS
    for t, x in zip((kv, kr), want):
        x[16:32] = x[128:141] = 0
        assert torch.equal(t, x)
