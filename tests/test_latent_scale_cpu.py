"""Scales that the softmax's base 2 takes out of fp32's range are refused."""
import math

import numpy as np
import pytest

from paged_kv_cache_195_gb300 import _binding as b

from test_latent_cpu import _absorbed, _expanded, lib  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("scale", [float(np.finfo(np.float32).max), 2.0 ** 128 / math.log2(math.e) * (1 + 2.0 ** -20)])
@pytest.mark.parametrize("call", [_absorbed, _expanded])
def test_scales_past_fp32_in_base_2(lib, call, scale):  # noqa: F811
    with np.errstate(over="ignore"):
        assert np.isfinite(np.float32(scale)) and np.isinf(np.float32(scale) * np.float32(math.log2(math.e)))
    assert call(lib, scale=scale) == b.PKV_ERR_INVALID and lib.pkv_last_error()
