"""CPU: an order in the prefix kernel that no run can show to be wrong without hanging."""
from __future__ import annotations

import os

from tests.conftest import ROOT


def test_tensor_memory_is_taken_after_the_dependency_wait():
    """The allocation waits without a limit: taken while the stream's earlier kernel still runs on the SM, it could keep
    that kernel from the columns it needs to end."""
    with open(os.path.join(ROOT, "query_aware_sparse_block_gb300", "csrc", "prefix_decode.cu")) as f:
        kernel = f.read().split("void __launch_bounds__(kThreads, 1) prefix_kernel(", 1)[1]
    assert kernel.count("tmem_alloc(") == 1
    assert kernel.index("griddepcontrol.wait;") < kernel.index("tmem_alloc(")
