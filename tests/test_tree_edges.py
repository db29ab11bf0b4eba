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


# ------------------------------------------------------------------ caches past 4 GB
@pytest.mark.gpu
@pytest.mark.parametrize("fmt,ps,layout", [("16bit", 16, "NHD"), ("16bit", 3, "HND"), ("block", 16, "HND"),
                                           ("block", 3, "NHD"), ("scaled", 16, "NHD"), ("scaled", 1, "NHD")])
def test_pages_behind_the_first_4_gb(fmt, ps, layout):
    """The few used pages at the end of a pool of more than 2^32 bytes, loaded by TMA
    and gathered: the result of a short pool."""
    c = tree_case(n=[7, 30], kv_len=[300, 64], H=16, Hk=8, d=128, ps=ps, fmt=fmt, layout=layout, seed=3)
    want = c.run()
    c.check(*want)
    page = 2 * ps * c.Hk * c.d * (2 if fmt == "16bit" else 1)
    first = 2 ** 32 // page + 1000
    q, kv, more = c.args()
    big = torch.zeros((first + c.pages,) + tuple(kv.shape[1:]), dtype=kv.dtype, device="cuda")
    big[first:] = kv
    if more["kv_scales"] is not None:
        s = torch.zeros((first + c.pages,) + tuple(c.scales.shape[1:]), dtype=torch.uint8, device="cuda")
        s[first:] = more["kv_scales"]
        more["kv_scales"] = s
    c.kv_indices = c.kv_indices + np.int32(first)
    c.pages += first
    h = c.plan()
    ws = torch.empty(pod.pod_tree_workspace_size(h), dtype=torch.uint8, device="cuda")
    pod.pod_tree_bind_workspace(h, ws)
    out, lse = pod.pod_tree_run(h, q, big, ws, **more)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------ one behind the other
@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["16bit", "scaled", "block"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("long", [1200, 500], ids=["merged", "whole"])
def test_nothing_but_these_kernels_in_the_stream(fmt, d, long):
    """Layers whose stream holds no other kernel: a write of the last output's rows,
    read where they lie, and the attention over it, into kept buffers. The merge of one
    layer lies right before the write and the attention of the next, which rewrite the
    cache and the partial rows; results are those of waiting for each call."""
    c = tree_case(n=[9, 30, 4], kv_len=[long, 400, 40], H=8, Hk=2, d=d, ps=16, fmt=fmt, seed=2)
    h = c.plan(num_sms=152)
    assert (len(pod.pod_tree_plan_table(h, 2)) > 0) == (long == 1200)
    ws = torch.empty(pod.pod_tree_workspace_size(h), dtype=torch.uint8, device="cuda")
    pod.pod_tree_bind_workspace(h, ws)
    req = np.repeat(np.arange(3), c.n)
    at = np.concatenate([np.arange(a - b, a) for a, b in zip(c.kv_len, c.n)])
    slots = torch.from_numpy(pod.pod_kv_slots(c.kv_indptr, c.kv_indices, c.ps, req, at)).cuda()

    def layers(wait, n=12):
        q, kv, more = c.args()
        outs = [q] + [torch.empty_like(q) for _ in range(n)]
        lses = [torch.empty(q.shape[:2], dtype=torch.float32, device="cuda") for _ in range(n)]
        torch.cuda.synchronize()
        for i in range(n):
            new = outs[i][:, 2 * (i % 3):2 * (i % 3) + 2]
            pod.pod_append_kv(new, new, kv, slots, kv_scales=more["kv_scales"], k_scale=c.ks, v_scale=c.vs)
            if wait:
                torch.cuda.synchronize()
            pod.pod_tree_run(h, outs[i], kv, ws, out=outs[i + 1], lse=lses[i], **more)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs[1:], lses
    want, got = layers(True), layers(False)
    for w, x in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, x))
    assert got[0][-1].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["16bit", "scaled", "block"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("long", [1200, 500], ids=["merged", "whole"])
def test_runs_on_one_workspace_right_behind_each_other(fmt, d, long):
    """Runs of one plan with different queries, nothing between them: an attention
    right behind the merge before, which reads the partial rows that it rewrites, or
    right behind another attention."""
    c = tree_case(n=[9, 30, 4], kv_len=[long, 400, 40], H=8, Hk=2, d=d, ps=16, fmt=fmt, seed=2)
    h = c.plan(num_sms=152)
    assert (len(pod.pod_tree_plan_table(h, 2)) > 0) == (long == 1200)
    ws = torch.empty(pod.pod_tree_workspace_size(h), dtype=torch.uint8, device="cuda")
    pod.pod_tree_bind_workspace(h, ws)
    q, kv, more = c.args()
    g = torch.Generator(device="cuda").manual_seed(1)
    qs = [torch.randn(q.shape, generator=g, device="cuda").to(c.dtype) for _ in range(16)]
    want = []
    for x in qs:
        want.append(pod.pod_tree_run(h, x, kv, ws, **more))
        torch.cuda.synchronize()
    got = [(torch.empty_like(a), torch.empty_like(b)) for a, b in want]
    torch.cuda.synchronize()
    for x, (o, l) in zip(qs, got):
        pod.pod_tree_run(h, x, kv, ws, out=o, lse=l, **more)
    torch.cuda.synchronize()
    for (a, b), (o, l) in zip(want, got):
        assert torch.equal(a, o) and torch.equal(b, l)
    assert pod.pod_tree_read_device_status(h, ws) == 0


# ------------------------------------------------------------------ one workspace, several plans
@pytest.mark.gpu
def test_a_workspace_holds_the_plan_bound_last():
    """A run of a plan whose workspace holds another one by now would read that one's
    tables: it is refused, and runs again once it is bound again."""
    a = tree_case(n=[9, 30, 4], kv_len=[1200, 400, 40], H=8, Hk=2, d=128, ps=16, seed=2)
    b = tree_case(n=[3], kv_len=[70], H=8, Hk=2, d=128, ps=16, seed=3)
    plans = [x.plan() for x in (a, b)]
    ws = torch.empty(max(pod.pod_tree_workspace_size(h) for h in plans), dtype=torch.uint8, device="cuda")
    tensors = [x.args() for x in (a, b)]

    def run(i, w=ws):
        q, kv, more = tensors[i]
        return pod.pod_tree_run(plans[i], q, kv, w, **more)
    pod.pod_tree_bind_workspace(plans[0], ws)
    a.check(*run(0))
    pod.pod_tree_bind_workspace(plans[1], ws)
    with pytest.raises(pod.PodError, match="another plan has been bound"):
        run(0)
    b.check(*run(1))
    pod.pod_tree_bind_workspace(plans[0], ws)
    with pytest.raises(pod.PodError, match="another plan has been bound"):
        run(1)
    a.check(*run(0))
    # a plan of pod_run takes it too
    h = pod.pod_plan(None, None, None, None, [0, 1], [0, 1], [0], [16], 8, 2, 128, 16, True, -1, None,
                     dtype=torch.bfloat16, p_num_pages=0, d_num_pages=1)
    other = torch.empty(max(ws.numel(), pod.pod_workspace_size(h)), dtype=torch.uint8, device="cuda")
    pod.pod_tree_bind_workspace(plans[0], other)
    pod.pod_bind_workspace(h, other)
    with pytest.raises(pod.PodError, match="another plan has been bound"):
        run(0, other)
    # the plan that took it is gone, and this one has moved on and come back
    pod.pod_tree_bind_workspace(plans[1], ws)
    pod.pod_tree_bind_workspace(plans[0], ws)
    pod.pod_tree_destroy(plans[1])
    a.check(*run(0))
    pod.pod_tree_bind_workspace(plans[0], other)
    with pytest.raises(pod.PodError, match="differs"):
        run(0)
    a.check(*run(0, other))


def test_a_workspace_is_a_whole_piece_of_the_device():
    """A host tensor, and an expanded one that is shorter than its elements, are refused
    before anything is copied."""
    c = tree_case(n=[3], kv_len=[70], H=8, Hk=2, d=128, ps=16, seed=3)
    h = c.plan(num_sms=4)
    n = pod.pod_tree_workspace_size(h)
    host = torch.empty(n, dtype=torch.uint8)

    class OnDevice:                                   # (what is asked of a tensor before its pointer)
        is_cuda = True

        def __init__(self, t):
            self.is_contiguous, self.data_ptr, self.numel = t.is_contiguous, t.data_ptr, t.numel
            self.element_size, self.get_device = t.element_size, lambda: 0
    for ws in (host, OnDevice(host[:1].expand(n)), OnDevice(torch.empty(2 * n, dtype=torch.uint8)[::2])):
        with pytest.raises(pod.PodError, match="contiguous CUDA tensor"):
            pod.pod_tree_bind_workspace(h, ws)
        with pytest.raises(pod.PodError, match="contiguous CUDA tensor"):
            c.plan(num_sms=4, workspace=ws)
