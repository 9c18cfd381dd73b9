"""What include/pa.h says of a call's errors is what the call answers."""
import os
import re

import pytest

from paged_kv_decode_varlen_gb300 import binding as b
from tests.test_step_cpu import _attn, _decode

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pa.h")


def comment_before(name):
    """The header's comment above the declaration of `name`, in one line."""
    text = open(HEADER).read()
    end = re.search(r"\n(pa_status|size_t) %s\(" % name, text).start()
    return re.sub(r"\s*\n \*\s*", " ", text[text.rindex("/*", 0, end):end])


@pytest.mark.parametrize("R", [-1, 65536, 1 << 20])
def test_a_number_of_rows_out_of_range(R):
    assert _decode(R=R) == _attn(R=R) == b.PA_ERR_INVALID_ARG
    said = re.search(r"num_reqs is 0 \.\. 65535 \((\w+) otherwise\)", comment_before("pa_decode_window"))
    assert getattr(b, said.group(1)) == b.PA_ERR_INVALID_ARG
