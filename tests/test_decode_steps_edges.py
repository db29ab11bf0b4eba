"""Decode steps whose tables live on the device: values and calls at their edges,
beside tests/test_decode_steps.py, whose 64-bit definitions these use.
"""
import math

import numpy as np
import pytest
import torch

import prefill_decode_paged_pod_gb300 as pod
from test_decode_steps import built, select64, table_of    # noqa: F401

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ selection
@gpu
@pytest.mark.parametrize("d,dtype,n,batch", [(64, "bf16", 40, 2), (128, "fp16", 333, 3), (256, "bf16", 200, 2),
                                             (128, "bf16", 700, 70)])
def test_select_passes_over_pages_outside_the_pool(d, dtype, n, batch):
    """Every page of the pool scores below 0; pages outside it, at any place of a row, never win."""
    dt, hk, ps, H = DT[dtype], 2, 16, 8
    r = np.random.RandomState(n)
    tab = r.randint(0, 300, (batch, n)).astype(np.int32)
    off = r.rand(batch, n) < 0.3
    off[0, -3:] = off[1, :2] = True
    tab[off] = r.choice([-1, 300, (1 << 31) - 1, -(1 << 31)], int(off.sum()))
    lens = [n * ps - int(x) for x in r.randint(0, ps, batch)]
    g = torch.Generator().manual_seed(d)
    x = -torch.rand((2, 300, hk, d), generator=g) - 0.5
    bounds = torch.stack([torch.minimum(x[0], x[1]), torch.maximum(x[0], x[1])], 2).to(dt).cuda()
    q = (torch.rand((batch, H, d), generator=g) + 0.1).to(dt).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for k, last in ((1, 0), (9, 1), (n // 2, 0)):
        got = pod.pod_select_pages(q, bounds, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                   k, ps, keep_last=last, status=status)
        assert torch.equal(got.cpu(), select64(q, bounds, tab, lens, ps, k, 0, last))
        assert status.item() == 4
