"""Decode steps whose tables live on the device: values and calls at their edges,
beside tests/test_decode_steps.py, whose 64-bit definitions these use.
"""
import math
import os
import re

import numpy as np
import pytest
import torch

import prefill_decode_paged_pod_gb300 as pod
from test_decode_steps import (DEC, attend64, built, c_call, check, dense_keys, fmt_args, make_bounds,    # noqa: F401
                               make_cache, select64, table_of, values64)

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


@gpu
@pytest.mark.parametrize("e", [-64, -70, -76, -100, -125])
@pytest.mark.parametrize("d,n,G", [(64, 90, 4), (128, 700, 2), (256, 9000, 1)])
def test_select_with_products_below_fp32(e, d, n, G):
    """Queries and bounds of some 2^e: their products are subnormal in fp32, or 0, and the choice is still that of 64 bits."""
    dt, hk, ps = torch.bfloat16, 2, 16
    tab, pages = table_of([n * ps, n * ps - 5], ps, 3)
    bounds = make_bounds(pages, hk, d, torch.float32, 4).mul(2.0 ** e).to(dt)
    q = (torch.randn((2, hk * G, d), generator=torch.Generator().manual_seed(5)) * 2.0 ** e).to(dt).cuda()
    lens = [n * ps, n * ps - 5]
    for k in (5, n // 3):
        got = pod.pod_select_pages(q, bounds, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                   k, ps)
        assert torch.equal(got.cpu(), select64(q, bounds, tab, lens, ps, k, 0, 1))


# ------------------------------------------------------------------ bounds
@gpu
@pytest.mark.parametrize("fmt,dtype,d,ps,layout,far", [("16bit", "bf16", 128, 16, "NHD", False), ("16bit", "fp16", 64, 3, "HND", False),
                                                      ("scaled", "bf16", 256, 40, "HND", False), ("block", "fp16", 128, 16, "NHD", False),
                                                      ("block", "bf16", 64, 33, "HND", True), ("scaled", "fp16", 128, 1, "NHD", False)])
def test_bounds_of_channels_without_a_number(fmt, dtype, d, ps, layout, far):
    """Both are NaN, so the page is attended and its NaN shows as it does over all keys; one number among
    NaNs is the bound."""
    dt, hk, n = DT[dtype], 2, 12
    lens = [n * ps]
    tab, pages = table_of(lens, ps, 1)
    kv, sc = make_cache(pages, ps, hk, d, layout, fmt, dt, 2)
    if far:
        sc[:, 0, :, ::2] = 90
    raw = kv.view(torch.int16) if fmt == "16bit" else kv.view(torch.uint8)
    nan = 0x7fff if fmt == "16bit" else 0x7f
    page = int(tab[0, 4])
    keys = raw[page, 0] if layout == "NHD" else raw[page, 0].transpose(0, 1)       # [ps, hk, d]
    keys[:, 1, 5] = nan
    keys[1:, 0, 6] = nan
    bounds = torch.zeros((pages, hk, 2, d), dtype=dt, device="cuda")
    args = fmt_args(fmt, sc)
    args.pop("v_scale", None)
    slots = torch.from_numpy((tab[0, :n, None].astype(np.int64) * ps + np.arange(ps)).reshape(-1)).cuda()
    pod.pod_page_bounds(kv, bounds, slots, kv_layout=layout, **args)
    want = torch.zeros((pages, hk, 2, d), dtype=torch.bool)
    want[page, 1, :, 5] = True
    assert torch.equal(bounds.isnan().cpu(), want)
    b = bounds.double().cpu()
    one = values64(kv, sc, layout, fmt)[page, 0, 0, 0, 6].float().double()       # (code * scale in fp32)
    near = abs(one) * torch.finfo(dt).eps + torch.finfo(dt).tiny * torch.finfo(dt).eps
    assert one - near <= b[page, 0, 0, 6] <= one <= b[page, 0, 1, 6] <= one + near
    q = torch.randn((1, 2 * hk, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    t, ln = torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    sel = pod.pod_select_pages(q, bounds, t, ln, 2, ps)
    assert 4 in sel[0, 1].tolist()
    args = fmt_args(fmt, sc)
    for pages_ in (sel, None):
        out, lse = pod.pod_paged_decode(q, kv, t, ln, pages=pages_, kv_layout=layout, **args)
        assert out[0, 2:].isnan().all() and lse[0, 2:].isnan().all()


# ------------------------------------------------------------------ decode
@gpu
@pytest.mark.parametrize("n,pad", [(16, 0), (40, 0), (40, 3000), (3000, 0)])
@pytest.mark.parametrize("nats", [16, 20])
@pytest.mark.parametrize("fmt,dtype,d,G", [("16bit", "bf16", 128, 4), ("16bit", "fp16", 128, 4), ("16bit", "fp16", 64, 12),
                                           ("scaled", "bf16", 128, 8), ("scaled", "fp16", 64, 3), ("scaled", "bf16", 256, 4),
                                           ("block", "bf16", 128, 8), ("block", "fp16", 128, 16), ("block", "bf16", 64, 16),
                                           ("block", "fp16", 256, 5)])
def test_one_key_takes_the_weight_and_has_no_value(fmt, dtype, d, G, nats, n, pad):
    """One key lies 16 or 20 nats above the others and its V is 0, so the output is made of small
    weights alone. A weight is off by `part` of itself (2^-17 and 2^-22 in two parts of bf16 and fp16,
    2^-11 in one part of fp16) and, where fp16 carries it, by `floor` of the largest (2^-43, 2^-38 in one
    part; under block scales, of the largest weight times its V's scale); by d 2^-23 A for the sum of its logit
    (A: that of the products' magnitudes; 0 for the one key, a single product), by 2^-23 |s| log2(e) for each of two
    roundings of the logit s, and by 2^-21 for exponentials and joins, which the denominator has too; the output is
    rounded to eps / 2, or half a step of the type's smallest numbers."""
    dt, hk, ps = DT[dtype], 2, 16
    tab, pages = table_of([n], ps, 1, pad=pad)
    kv, sc = make_cache(pages, ps, hk, d, "NHD", fmt, dt, 2)
    top, scale = 5, 1 / math.sqrt(d)
    at = (int(tab[0, top // ps]), slice(None), top % ps)
    kv[:, 0, :, :, 0] = 0
    # (V of some thousands, so that fp16 holds what is left of it)
    args = fmt_args(fmt, sc)
    if fmt == "16bit":
        kv[:, 1] *= 4096
    elif fmt == "scaled":
        args["v_scale"] *= 4096
    else:
        sc[:, 1] += 12
    kv[at] = 0
    # (logits of the others: N(0, 0.25) or so, under one block scale)
    q = torch.randn((1, hk * G, d), generator=torch.Generator().manual_seed(3)) * 0.25
    q[..., 0] = 32.0
    q = q.to(dt).cuda()
    if fmt == "block":
        sc[:, 0] = 120
        sc[at] = 127
    code = nats / scale / 32 / (0.034375 if fmt == "scaled" else 1.0)
    assert code < 448
    kv[at[0], 0, at[2], :, 0] = torch.tensor(code).to(kv.dtype)
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                                    **args)
    x = values64(kv, sc, "NHD", fmt)
    if fmt == "scaled":
        x[:, 1] *= 4096
    page, slot = dense_keys(tab[0], n, ps, 1, -1)[0]
    got = out[0].double().cpu()
    for h in range(hk * G):
        k, v, qh = x[page, 0, slot, h // G], x[page, 1, slot, h // G], q[0, h].double().cpu()
        s = k @ qh * scale
        p = torch.exp(s - s.max())
        assert s.argmax() == top and (v[top] == 0).all()
        z = p.sum()
        want, B = p @ v / z, p @ v.abs() / z
        A = scale * (k.abs() @ qh.abs())
        A[top] = 0
        rel = 2.0 ** -22 * 1.4427 * s.abs().max() + 2.0 ** -21
        part, floor = (2.0 ** -17, 0.0) if fmt == "16bit" and dt == torch.bfloat16 else (2.0 ** -22, 2.0 ** -43)
        if fmt != "16bit" and dt == torch.bfloat16:
            part, floor = 2.0 ** -11, 2.0 ** -38
        unit = torch.ones(n, dtype=torch.float64)
        if fmt == "block":
            unit = torch.exp2(sc.cpu().double()[page, 1, slot, h // G] - 127)
        low = floor * (p * unit).max() * (v.abs() / unit[:, None]).sum(0) / z
        tol = torch.finfo(dt).eps / 2 * want.abs() * (1 + 2.0 ** -7) + (2 * rel + part) * B + low \
            + d * 2.0 ** -23 * (p * A) @ v.abs() / z + torch.finfo(dt).tiny * torch.finfo(dt).eps / 2
        err = (got[h] - want).abs()
        assert (err <= tol).all(), (h, (err / tol).max(), (err / B).max())


@gpu
@pytest.mark.parametrize("byte,most", [(0, 448.0), (1, 448.0), (254, 1.0)])
@pytest.mark.parametrize("n,pad", [(1, 0), (50, 0), (3000, 0), (50, 3000)])
def test_smallest_and_largest_scales_of_values(byte, most, n, pad):
    """V scales at the ends of the exponent byte: 2^-127 times a code is a bf16 number."""
    dt, hk, G, d, ps = torch.bfloat16, 2, 4, 64, 16
    tab, pages = table_of([n], ps, 1, pad=pad)
    kv, sc = make_cache(pages, ps, hk, d, "NHD", "block", dt, 2)
    codes = torch.rand(kv[:, 1].shape, generator=torch.Generator().manual_seed(4)) * most
    kv[:, 1] = codes.to(kv.dtype).cuda()
    sc[:, 1] = byte
    q = torch.randn((1, hk * G, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                                    kv_scales=sc)
    x = values64(kv, sc, "NHD", "block")
    want, wlse, A, B = attend64(q[0].double().cpu().numpy(), x, dense_keys(tab[0], n, ps, hk, -1), 1 / 8, None)
    # weights in one part: 2^-11; x + e is rounded twice at some 2^7: 2^-17 of log2 each; the rest as in check()
    rel = 2 * (d * 2.0 ** -23 * A + 2.0 ** -16)[:, None] + 2.0 ** -11
    tol = np.abs(want) * 2.0 ** -8 * (1 + 2.0 ** -7) + rel * B
    assert (np.abs(out[0].double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(lse[0].double().cpu().numpy() - wlse) <= 1e-3).all() and want.any()


@gpu
@pytest.mark.parametrize("n,pad", [(1, 0), (40, 0), (3000, 0), (40, 3000), (3000, 3000)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("fmt,dtype,mag", [(f, t, m) for f in ("16bit", "scaled", "block") for t in ("bf16", "fp16")
                                           for m in (1e5, 2e7, 7e7, 3e8, 1e12, 1e30) if t == "bf16" or m < 4e8])
def test_logits_of_any_size(fmt, dtype, mag, sign, n, pad):
    """Logits of some `mag`, single products whose nearest neighbours are a sixteenth of that apart, so that the keys
    of the largest one share the weight. In fp32 a logit is then off by more than its exponential can bear, but equal
    ones are equal: the result is the mean of these keys' values, off by 2^-11 of each weight (and of their sum) at
    most, and by its own rounding."""
    dt, hk, G, d, ps = DT[dtype], 2, 4, 64, 16
    tab, pages = table_of([n], ps, 1, pad=pad)
    kv, sc = make_cache(pages, ps, hk, d, "NHD", fmt, dt, 2)
    g = torch.Generator().manual_seed(3)
    kv[:, 0] = 0
    kv[:, 0, ..., 0] = (torch.randint(16, 32, kv[:, 0, ..., 0].shape, generator=g).float() * sign).to(kv.dtype).cuda()
    if fmt == "block":
        sc[:, 0] = 127
    q = torch.zeros((1, hk * G, d))
    q[..., 0] = mag / 2 if mag > 4e8 else mag * 8 / 24            # (s = 1/8, k of 16 to 31)
    args = fmt_args(fmt, sc)
    x = values64(kv, sc, "NHD", fmt)
    if mag <= 4e8 and dtype == "fp16":                            # (fp16 ends at 65504: the scale takes the rest)
        args["sm_scale"] = mag / 24 / 4096
        q[..., 0] = 4096.0
    q = q.to(dt).cuda()
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                                    **args)
    page, slot = dense_keys(tab[0], n, ps, 1, -1)[0]
    for h in range(hk * G):
        k, v = x[page, 0, slot, h // G, 0], x[page, 1, slot, h // G]
        top = v[k == k.max()]
        err = (out[0, h].double().cpu() - top.mean(0)).abs()
        tol = torch.finfo(dt).eps / 2 * top.mean(0).abs() * (1 + 2.0 ** -7) + 2 * (2.0 ** -11 + 2.0 ** -20) * top.abs().mean(0)
        assert (err <= tol + torch.finfo(dt).tiny).all(), (h, err.max())
        want = float(q[0, h, 0].double() * k.max() * (args.get("sm_scale") or 1 / 8)) * 1.4426950408889634
        assert abs(lse[0, h].item() - want) <= abs(want) * 2.0 ** -20 + 13


@gpu
@pytest.mark.parametrize("pad", [0, 3000])
@pytest.mark.parametrize("fmt,dtype,e", [(f, "bf16", e) for f in ("16bit", "scaled", "block") for e in (-127, -100, 60, 110)]
                         + [(f, "fp16", e) for f in ("16bit", "scaled", "block") for e in (-16, 12)])
def test_queries_of_any_magnitude(fmt, dtype, e, pad):
    """Queries of some 2^e, subnormal ones among them, under a scale of some 2^-e."""
    dt, hk, H, d, ps = DT[dtype], 2, 10, 128, 16
    lens = [600, 3]
    tab, pages = table_of(lens, ps, 1, pad=pad)
    kv, sc = make_cache(pages, ps, hk, d, "NHD", fmt, dt, 2)
    q = (torch.randn((2, H, d), generator=torch.Generator().manual_seed(3), dtype=torch.float64) * 2.0 ** e).to(dt).cuda()
    scale = 2.0 ** -(e + 3)
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    sm_scale=scale, **fmt_args(fmt, sc))
    x = values64(kv, sc, "NHD", fmt)
    ref = [attend64(q[i].double().cpu().numpy(), x, dense_keys(tab[i], n, ps, hk, -1), scale, None) for i, n in enumerate(lens)]
    check(out, lse, *(np.stack(y) for y in zip(*ref)), d, dt, fmt)


@gpu
@pytest.mark.parametrize("pad", [0, 3000])
@pytest.mark.parametrize("e", [-120, -110, -90, 90, 110, 118])
def test_keys_and_queries_far_apart(e, pad):
    """Queries of some 2^e over keys whose block scales make up for them."""
    dt, hk, H, d, ps = torch.bfloat16, 2, 10, 128, 16
    lens = [600, 3]
    tab, pages = table_of(lens, ps, 1, pad=pad)
    kv, sc = make_cache(pages, ps, hk, d, "NHD", "block", dt, 2, 119, 122)
    sc[:, 0] -= e
    q = (torch.randn((2, H, d), generator=torch.Generator().manual_seed(3)) * 2.0 ** e).to(dt).cuda()
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    kv_scales=sc)
    x = values64(kv, sc, "NHD", "block")
    scale = 1 / math.sqrt(d)
    ref = [attend64(q[i].double().cpu().numpy(), x, dense_keys(tab[i], n, ps, hk, -1), scale, None) for i, n in enumerate(lens)]
    check(out, lse, *(np.stack(y) for y in zip(*ref)), d, dt, "block")


@gpu
@pytest.mark.parametrize("H,hk,d,ps,fmt,dtype", [(72, 4, 128, 1, "16bit", "bf16"), (40, 4, 256, 2, "block", "fp16"),
                                                 (160, 8, 64, 3, "scaled", "bf16")])
def test_small_pages_and_two_tiles_of_heads(H, hk, d, ps, fmt, dtype):
    """Four KV heads a CTA, and more query heads a KV head than one tile holds."""
    dt, B = DT[dtype], 130
    r = np.random.RandomState(4)
    lens = [int(x) for x in r.choice([0, 1, 5, 63, 64, 65, 200], B)]
    lens[7], lens[60] = 3000, 1111
    tab, pages = table_of(lens, ps, 1, pad=9000 // ps)
    kv, sc = make_cache(pages, ps, hk, d, "NHD", fmt, dt, 2)
    q = torch.randn((B, H, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    **fmt_args(fmt, sc))
    x = values64(kv, sc, "NHD", fmt)
    at = [7, 60] + list(range(20, 30)) + [B - 1]
    ref = [attend64(q[i].double().cpu().numpy(), x, dense_keys(tab[i], lens[i], ps, hk, -1), 1 / math.sqrt(d), None) for i in at]
    check(out[at], lse[at], *(np.stack(y) for y in zip(*ref)), d, dt, fmt)


@gpu
@pytest.mark.parametrize("extra", [0, 2100])
def test_tables_that_are_slices(extra):
    """A wider table's columns and every other row: selection and both decode kernels."""
    dt, hk, H, d, ps = torch.float16, 2, 8, 64, 16
    lens = [300, 17, 0, 640]
    tab, pages = table_of(lens, ps, 1, pad=extra)
    kv, _ = make_cache(pages, ps, hk, d, "NHD", "16bit", dt, 2)
    bounds = make_bounds(pages, hk, d, dt, 4)
    big = torch.full((8, tab.shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    t = big[::2, 3:-2]
    t.copy_(torch.from_numpy(tab))
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn((4, H, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    sel = pod.pod_select_pages(q, bounds, t, ln, 4, ps)
    assert torch.equal(sel.cpu(), select64(q, bounds, tab, lens, ps, 4, 0, 1))
    for pages_ in (None, sel):
        want = pod.pod_paged_decode(q, kv, t.contiguous(), ln, pages=pages_)
        got = pod.pod_paged_decode(q, kv, t, ln, pages=pages_)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_captured_between_copies_fills_and_other_branches():
    """In a graph whose nodes before the calls are a copy, a fill and a kernel of another stream."""
    dt, hk, H, d, ps, B = torch.bfloat16, 2, 8, 64, 16, 5
    lens = [300, 17, 0, 640, 4000]
    tab, pages = table_of(lens, ps, 1)
    kv, _ = make_cache(pages, ps, hk, d, "NHD", "16bit", dt, 2)
    bounds = make_bounds(pages, hk, d, dt, 4)
    t, ln = torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    host = torch.randn((B, H, d), generator=torch.Generator().manual_seed(3)).to(dt).pin_memory()
    q, side = torch.empty((B, H, d), dtype=dt, device="cuda"), torch.zeros((B, H, d), dtype=dt, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        q.copy_(host, non_blocking=True)
        status.zero_()
        sel = pod.pod_select_pages(q, bounds, t, ln, 4, ps, status=status)
        now, other = torch.cuda.current_stream(), streams[1]
        other.wait_stream(now)
        with torch.cuda.stream(other):
            side.copy_(q).mul_(2)
            beside = pod.pod_paged_decode(side, kv, t, ln)
        here = pod.pod_paged_decode(q, kv, t, ln, pages=sel)
        now.wait_stream(other)
        return (sel,) + here + beside + pod.pod_paged_decode(side, kv, t, ln, status=status)

    streams = [torch.cuda.Stream() for _ in range(2)]
    with torch.cuda.stream(streams[0]):
        want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        got = step()
    for _ in range(5):
        for x in got:
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and status.item() == 0
    assert torch.equal(want[3], want[5])


# ------------------------------------------------------------------ the step as a whole
@gpu
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [1, 0, 1, 1], [0, 5, 0, 1], [3, 0, -2, 0]])
def test_the_step_of_the_readme(new):
    """Its text as it stands: every request with rows attends its own keys, others sitting out or not."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        code, = (x for x in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "pod_step_tables" in x)
    dt, H, Hk, d, page_size, B = torch.bfloat16, 8, 2, 64, 16, 4
    lens, pages = [40, 100, 7, 64], 40
    kv, _ = make_cache(pages, page_size, Hk, d, "NHD", "16bit", dt, 2)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")    # noqa: E731
    rows = max(B, sum(max(0, n) for n in new))
    qkv = torch.randn((rows, H + 2 * Hk, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    w = torch.ones(d, dtype=dt, device="cuda")
    env = dict(pod=pod, block_table=torch.zeros((B, 9), dtype=torch.int32, device="cuda"), kv_lens=dev([0] * B),
               new_lens=dev(new), free_pages=dev(np.random.RandomState(1).permutation(pages)), free_count=dev([pages]),
               page_size=page_size, batch=B, qkv=qkv, H=H, Hk=Hk, kv_cache=kv, wq=w, wk=w,
               bounds=torch.zeros((pages, Hk, 2, d), dtype=dt, device="cuda"))
    first = pod.pod_step_tables(env["block_table"], env["kv_lens"], dev(lens), env["free_pages"], env["free_count"], page_size,
                                max_rows=sum(lens))
    pod.pod_page_bounds(kv, env["bounds"], first.slots)
    exec(code, env)
    now = [max(0, a + b) for a, b in zip(lens, new)]
    assert env["kv_lens"].tolist() == now
    table = env["block_table"].cpu().numpy()
    qn, _ = pod.pod_qk_norm_rope(qkv[:, :H], None, env["t"].positions, q_weight=w)
    x = values64(kv, None, "NHD", "16bit")
    row = 0
    for r, n in enumerate(new):
        if n <= 0:
            continue
        row += n
        want = attend64(qn[row - 1].double().cpu().numpy(), x, dense_keys(table[r], now[r], page_size, Hk, -1), 1 / math.sqrt(d),
                        None)
        check(env["out"][r:r + 1], env["lse"][r:r + 1], *(y[None] for y in want), d, dt)


# ------------------------------------------------------------------ step tables
@gpu
def test_step_tables_of_the_largest_stack():
    """2^31 - 1 places for 2^31 pages that are given back: indices end at the last place of 31 bits."""
    batch, width = 1024, 1 << 21
    total = batch * width
    table = torch.arange(total, dtype=torch.int32, device="cuda").view(batch, width)
    stack = torch.full((total + 63,), -9, dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), width, dtype=torch.int32, device="cuda")
    count, status = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    t = pod.pod_step_tables(table, lens, -lens, stack[32:32 + total - 1], count, 1, max_rows=1, status=status)
    assert count.item() == total - 1 and status.item() == 8 and t.kv_lens.tolist() == [0] * batch
    assert (stack[:32] == -9).all() and (stack[32 + total - 1:] == -9).all()
    assert torch.equal(stack[32:32 + total - 1], table.view(-1)[:-1])
    # a step with room for one row leaves them all there
    new = torch.full((batch,), width, dtype=torch.int32, device="cuda")
    t = pod.pod_step_tables(table, lens, new, stack[32:32 + total - 1], count, 1, max_rows=1, status=status)
    assert count.item() == total - 1 and t.kv_lens.tolist() == [0] * batch and t.requests.tolist() == [-1]


# ------------------------------------------------------------------ refusals
def test_pages_of_more_than_2_30_slots_are_refused():
    """By all calls that read a pool (two refuse them for their tables already). Nothing is launched."""
    lib = pod.load_library()
    for name in ("pod_page_bounds", "pod_select_pages", "pod_paged_decode"):
        for ps in ((1 << 30) + 1, (1 << 31) - 1):
            code = c_call(getattr(lib, name), DEC, pod._DECODE_ARGS, ps=ps, num_pages=1, Hk=1, rows=0, batch=0, width=1)
            assert code == 1 and pod.pod_last_error(), (name, ps)
    assert c_call(lib.pod_page_bounds, DEC, pod._DECODE_ARGS, ps=1 << 30, num_pages=1, Hk=1, rows=0) == 0
