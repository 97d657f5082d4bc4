"""The kernels of the operators on expert-grouped rows are launched while the kernel before them still runs, and wait
for its end.  What they read may be what it writes, and the read-only path (ld.global.nc) holds only for memory that
does not change in a kernel's lifetime: the compiler may move such a load in front of the wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_topk_ids_gb300", "csrc")


@pytest.mark.parametrize("name", ["sort_rows.cu", "quant_fp8.cu", "product_fp8.cu"])
def test_no_load_through_the_read_only_path(name):
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert "pdl_wait()" in code
    assert not re.findall(r"__ldg|ld\.global\.nc|__restrict__", code)
