"""Keys and values of a chunk's own tokens that are both not finite."""
import pytest
import torch

import paged_kv_cache_195_gb300 as pkv
from paged_kv_cache_195_gb300 import build as pkv_build

from test_gpu_latent import exp_case, exp_check, exp_run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    pkv.load_library()


@pytest.mark.parametrize("heads,lens,qs", [(1, [200], [150]), (2, [2000], [100]), (8, [700] * 8, [512] * 8)])
def test_weight_of_zero_times_an_infinity(heads, lens, qs):
    """Scored -inf, a token weighs nothing, and its infinite value makes a NaN where it
    is seen and nothing elsewhere.  (The last set runs in pairs, the second is split.)"""
    n, m = lens[0], qs[0]
    for part, what in (("k", "inf"), ("k", "-inf"), ("r", "-inf")):
        c = exp_case(lens, qs, heads, seed=8)
        # every query has a 1 where the key is -inf
        c["q"][:, :, 7 if part == "k" else 130] = -1 if what == "inf" else 1
        for at in (0, 3, m // 2, m - 2):
            pos = n - m + at
            if part == "k":
                c["kv"][pos, :, 7] = float(what)
            else:
                c["kr"][pos, 2] = float(what)
            if at != 3:
                c["kv"][pos, heads - 1, 128 + at % 128] = float("inf")
        exp_check(c, exp_run(c))
        assert pkv.pkv_get_device_error() == 0
