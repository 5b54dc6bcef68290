"""What the kernels' sources must not hold, whatever a measurement says for it."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).parent.parent / "paged_kv_cache_195_gb300" / "csrc"


@pytest.mark.parametrize("path", sorted(CSRC.glob("*.cu*")), ids=lambda p: p.name)
def test_copies_go_to_one_cta(path):
    """No multicast copy: every rank of a job on several GPUs loads this library, and a
    pool may be any memory that its GPU can read."""
    text = re.sub(r'"\s*"', "", path.read_text())  # (instructions in several pieces)
    assert not re.findall(r"cp\.async\.bulk[^;]*multicast", text)
