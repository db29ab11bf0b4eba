"""Tree attention at the edges of what its calls allow: page tables that do not
fit together, sinks of minus infinity, caches past 4 GB, and kernels that start
beside the one before.
"""
import numpy as np
import pytest
import torch

import prefill_decode_paged_pod_gb300 as pod


@pytest.fixture(scope="module", autouse=True)
def built():
    from prefill_decode_paged_pod_gb300 import _build
    _build.build()
    pod.load_library()


# ------------------------------------------------------------------ page tables (host)
@pytest.mark.parametrize("kv_indptr,n", [([0, 40, 2], 2), ([0, 1, 40, 2], 3), ([0, 40, 2, 2], 3)])
def test_no_page_is_read_before_the_table_is_known_to_fit(kv_indptr, n):
    """An indptr that rises past the indices and comes back is refused for that,
    before an entry behind the indices is read (there are wrong ones behind these)."""
    store = np.full(64, -7, dtype=np.int32)
    store[:2] = [0, 1]
    with pytest.raises(pod.PodError, match="an indptr decreases"):
        pod.pod_tree_plan(np.arange(n + 1), kv_indptr, store[:2], [1] * n, 8, 2, 128, 16, dtype=torch.float16,
                          num_pages=2, num_sms=4)
