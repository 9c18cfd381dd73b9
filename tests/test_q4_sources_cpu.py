"""Properties of the q4 kernels' sources that no run can show reliably."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_varlen_gb300", "csrc")
Q4 = sorted(glob.glob(os.path.join(CSRC, "*q4*")))


def _code(path):
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("path", Q4, ids=os.path.basename)
def test_no_load_assumes_that_a_pool_is_read_only(path):
    """A q4 kernel is launched while the one before it, an append perhaps, may
    still run: a non-coherent load (ld.global.nc, __ldg, a __restrict__ pointer
    to const) may give what the pool held before.  The other load intrinsics
    are not ordered with the wait for that kernel by their definition either:
    the volatile loads of q4.cuh are."""
    assert not re.search(r"__ld(g|c[agsv]|lu)\s*\(|ld\.global[.\w]*\.nc|\b__restrict__\b", _code(path))
