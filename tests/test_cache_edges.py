"""The operators around the cache at the edges of what their calls allow: slots
of positions that no page holds, rows of any magnitude, angles of far positions,
caches past 4 GB, and kernels that start beside the one before.
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


# ------------------------------------------------------------------ slots (host)
INDPTR, INDICES = np.array([0, 2, 2, 5], np.int32), np.array([7, 3, 9, 0, 4], np.int32)


@pytest.mark.parametrize("tensors", [False, True])
def test_positions_without_a_page_are_padding_rows(tensors):
    """Before the first page, behind the last (another request's, or the table's
    end), a request without pages, requests that are not there."""
    req = np.array([0, 0, 0, 1, 2, 2, 2, -1, 3, 2, 0])
    pos = np.array([-1, 7, 8, 0, -4, 11, 12, 0, 0, 1 << 40, 0])
    want = [-1, 15, -1, -1, -1, 19, -1, -1, -1, -1, 28]
    conv = torch.from_numpy if tensors else np.asarray
    s = pod.pod_kv_slots(conv(INDPTR), conv(INDICES), 4, conv(req), conv(pos))
    assert s.tolist() == want and str(s.dtype).endswith("int64")


@pytest.mark.parametrize("tensors", [False, True])
def test_slots_of_an_empty_table_and_past_32_bits(tensors):
    conv = torch.from_numpy if tensors else np.asarray
    none = np.zeros(0, np.int32)
    s = pod.pod_kv_slots(conv(np.zeros(3, np.int32)), conv(none), 16, conv(np.array([0, 1])), conv(np.array([0, 3])))
    assert s.tolist() == [-1, -1]
    s = pod.pod_kv_slots(conv(np.zeros(1, np.int32)), conv(none), 16, conv(none), conv(none))
    assert s.tolist() == []
    big = np.array([2 ** 31 - 1], np.int32)
    pos = np.array([5], np.int32)               # (32-bit positions, a slot of 36 bits)
    s = pod.pod_kv_slots(conv(np.array([0, 1], np.int32)), conv(big), 16, conv(np.array([0], np.int32)), conv(pos))
    assert s.tolist() == [(2 ** 31 - 1) * 16 + 5]
