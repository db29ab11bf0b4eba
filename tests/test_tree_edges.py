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


# ------------------------------------------------------------------ sinks
def tree_case(**kw):
    from test_tree_attention import Case
    return Case(**kw)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [5, 12, 40], ids=["copies4", "copies2", "one"])
@pytest.mark.parametrize("fmt", ["16bit", "block"])
@pytest.mark.parametrize("sms", [0, 1])
def test_rows_without_keys_are_zero_whatever_their_sink(n, fmt, sms):
    """exp(sink) of 0, of a subnormal number, of 1 and of infinity, over no keys at
    all and over some; with one SM the tiles lie in other CTAs' work."""
    c = tree_case(n=[n, 3], kv_len=[n, 70], H=8, Hk=2, d=128, ps=16, fmt=fmt, mask="random", sinks=True, seed=3)
    c.sinks[:] = torch.tensor([-torch.inf, -95.0, -102.0, -88.0, 0.0, 60.0, -torch.inf, -1e30])
    out, lse = c.run(num_sms=sms)
    assert (out[0] == 0).all() and (lse[0] == -torch.inf).all()
    c.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("L,pieces", [(1100, 4), (3000, 6)], ids=["few", "many"])
def test_split_rows_without_keys_are_zero_whatever_their_sink(L, pieces):
    """The same where the tiles are cut and merged, in a few pieces and in many."""
    c = tree_case(n=[L], kv_len=[L], H=2, Hk=1, d=64, ps=16, mask="random", sinks=True, seed=3)
    c.bits[0][L // 2:] = 0
    c.packed = torch.from_numpy(np.packbits(c.bits[0].reshape(-1), bitorder="little"))
    c.sinks[:] = torch.tensor([-torch.inf, -95.0])
    groups = pod.pod_tree_plan_table(c.plan(num_sms=152), 2).reshape(-1, 8)
    assert (groups[:, 4] == pieces).all() and len(groups)
    out, lse = c.run(num_sms=152)
    empty = c.bits[0].sum(1) == 0
    assert (out.cpu()[empty] == 0).all() and (lse.cpu()[empty] == -torch.inf).all()
    c.check(out, lse)
