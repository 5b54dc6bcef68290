"""Queries rotated into memory of the latents that the same call reads: refused."""
import pytest

from paged_kv_cache_195_gb300 import _binding as b

from test_latent_cpu import FAKE, _append, lib  # noqa: F401  (lib: a fixture)

FAR = FAKE << 8
# Joint rows of [16 heads of 160 | 576]: the heads' last 64 dims, and the latents.
JOINT = 16 * 160 + 576


@pytest.mark.parametrize("kw", [
    dict(out=FAKE), dict(out=FAKE + 1024), dict(out=FAKE + 2 * 576 + 64, num_q_tokens=3),
    dict(kv=FAKE + 2 * 1024 - 16),                                                  # the last head's end
    dict(kv=FAKE, stride=JOINT, out=FAKE + 1136, os_=JOINT, oh=160),                # side by side, but for 8 dims
    dict(kv=FAKE + 2 * 16 * 160, stride=JOINT, out=FAKE + 2 * 104, os_=JOINT, oh=160),
    dict(kv=FAKE + 1024, stride=8192, os_=64, oh=128),                              # heads outermost
    dict(kv=FAKE, q=1 << 60, os_=1 << 62, oh=1 << 50, num_q_tokens=1)])
def test_queries_over_the_latents(lib, kw):  # noqa: F811
    kw = dict(dict(kv=FAKE, q=FAR, out=FAKE), **kw)
    assert _append(lib, **kw) == b.PKV_ERR_INVALID and b"q_rope_out and kv" in lib.pkv_last_error()


@pytest.mark.parametrize("kw", [
    dict(out=FAKE + 2 * (576 + 576)),                                               # right behind
    dict(kv=FAKE + 2 * 16 * 160, stride=JOINT, q=FAKE + 192, qs=JOINT, qh=160, out=FAKE + 192, os_=JOINT, oh=160),
    dict(kv=FAKE, stride=JOINT, q=FAKE + 1152, qs=JOINT, qh=160, out=FAKE + 1152, os_=JOINT, oh=160)])
def test_queries_beside_the_latents(lib, kw):  # noqa: F811
    """Parts of joint rows: refused by nothing but the missing device (or, on a GPU machine,
    not called at all)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are none")
    kw = dict(dict(kv=FAKE, q=FAR, out=FAKE), **kw)
    assert _append(lib, **kw) == b.PKV_ERR_CUDA
