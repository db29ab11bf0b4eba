"""Decode steps whose tables live on the device: step tables, page bounds, page
selection and paged decode against 64-bit definitions on the GPU, a captured
step that serves later ones, and the refusals on the CPU.

Tolerances, fixed before the first run. A logit s q.k is a sum of d products in
fp32 (exact products; an addition of the matrix unit is off by 2^-23 at most):
d 2^-23 A, with A = s sum |q_j k_j|, so a weight is off by that much of itself, by
2^-17 for its two 16-bit parts (2^-12 for the one fp16 part that bf16 results over FP8
caches take), by 2^-21 for the exponential and the scales of the joins; the output by twice the sum (numerator and denominator) of B = sum p |v|, and
then by its rounding, eps / 2. The base-2 LSE: the same relative error times log2(e),
and 2^-22 of itself. Weights below 2^-24 of the largest fp16 operand are off by up to
2^-39 of the largest weight each, which 2^20 keys leave below 2^-19.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import prefill_decode_paged_pod_gb300 as pod

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
K_SCALE, V_SCALE = 0.034375, 0.0125


@pytest.fixture(scope="module", autouse=True)
def built():
    from prefill_decode_paged_pod_gb300 import _build
    _build.build()
    pod.load_library()


# ------------------------------------------------------------------ inputs and definitions
def make_cache(pages, ps, hk, d, layout, fmt, dtype, seed, scale_lo=117, scale_hi=124):
    g = torch.Generator().manual_seed(seed)
    inner = (ps, hk) if layout == "NHD" else (hk, ps)
    x = torch.randn((pages, 2) + inner + (d,), generator=g)
    if fmt == "16bit":
        return x.to(dtype).cuda(), None
    if fmt == "scaled":
        x[:, 0] /= K_SCALE
        x[:, 1] /= V_SCALE
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).cuda(), None
    sc = torch.randint(scale_lo, scale_hi, (pages, 2) + inner, generator=g, dtype=torch.uint8)
    return (x * 120).clamp(-448, 448).to(torch.float8_e4m3fn).cuda(), sc.cuda()


def values64(kv, scales, layout, fmt):
    """[pages, 2, ps, hk, d] in 64 bits."""
    x = kv.cpu().float().double()
    if fmt == "scaled":
        x[:, 0] *= float(np.float32(K_SCALE))
        x[:, 1] *= float(np.float32(V_SCALE))
    elif fmt == "block":
        x = x * torch.exp2(scales.cpu().double() - 127)[..., None]
    return x if layout == "NHD" else x.transpose(2, 3)


def fmt_args(fmt, scales):
    if fmt == "scaled":
        return dict(k_scale=K_SCALE, v_scale=V_SCALE)
    return dict(kv_scales=scales) if fmt == "block" else {}


def table_of(lens, ps, seed, spare=2, pad=0):
    """A block table [batch, width] with random pages, garbage behind a request's pages."""
    r = np.random.RandomState(seed)
    n = [-(-x // ps) for x in lens]
    total = max(1, sum(n)) + spare
    perm = r.permutation(total)
    width = max(1, max(n)) + pad
    t = r.choice([-1, -(1 << 31), (1 << 31) - 1, total], size=(len(lens), width)).astype(np.int64)
    at = 0
    for i, k in enumerate(n):
        t[i, :k] = perm[at:at + k]
        at += k
    return t.astype(np.int32), total


def attend64(q, x, keys, scale, sinks):
    """q [H, d] over keys [per KV head: (page, slot) arrays]; (out, lse, A, B)."""
    H, d = q.shape
    hk = x.shape[3]
    G = H // hk
    out, lse = np.zeros((H, d)), np.full(H, -np.inf)
    A, B = np.zeros(H), np.zeros((H, d))
    for h in range(hk):
        page, slot = keys[h]
        if len(page) == 0:
            continue
        k, v = x[page, 0, slot, h].numpy(), x[page, 1, slot, h].numpy()
        for g in range(h * G, (h + 1) * G):
            s = k @ q[g] * scale
            m = s.max()
            p = np.exp(s - m)
            z = p.sum()
            lse[g] = (m + np.log(z)) / np.log(2)
            den = z + (np.exp(sinks[g] - m) if sinks is not None else 0.0)
            out[g] = p @ v / den
            A[g] = scale * (np.abs(k) @ np.abs(q[g])).max()
            B[g] = p @ np.abs(v) / den
    return out, lse, A, B


def check(got, lse, want, wlse, A, B, d, dtype, fmt="16bit"):
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    rel = d * 2.0 ** -23 * A + 2.0 ** -16
    part = 2.0 ** -12 if fmt != "16bit" and dtype == torch.bfloat16 else 0.0       # (not in the sum of the weights)
    tol = np.abs(want) * torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -7) + (2 * rel[..., None] + part) * B \
        + torch.finfo(dtype).tiny
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], tol[bad][:4])
    none = np.isneginf(wlse)
    assert (np.isneginf(lse) == none).all()
    err = np.abs(lse[~none] - wlse[~none])
    ltol = (rel * 1.4427 + 2.0 ** -22 * np.abs(wlse))[~none]
    assert (err <= ltol).all(), (err.max(), ltol.min())


def dense_keys(table, n, ps, hk, window):
    t = np.arange(max(0, n - 1 - window) if window >= 0 else 0, n)
    return [(table[t // ps].astype(np.int64), t % ps)] * hk


DECODES = [
    # H, Hk, d, ps, fmt, layout, dtype, lens, window, sinks
    (32, 8, 128, 16, "16bit", "NHD", "bf16", [1, 15, 16, 17, 600, 0, 63, 64, 65], -1, False),
    (64, 8, 128, 16, "16bit", "HND", "fp16", [2049, 3, 777], -1, True),
    (4, 1, 64, 16, "16bit", "NHD", "fp16", [17, 29, 5, 48], -1, False),
    (8, 8, 128, 1, "16bit", "NHD", "bf16", [257, 31, 1], -1, False),
    (6, 2, 128, 3, "16bit", "HND", "bf16", [100, 0, 7, 1000], 40, True),
    (12, 1, 128, 16, "16bit", "NHD", "bf16", [333, 64], -1, False),
    (40, 2, 64, 32, "16bit", "HND", "fp16", [333, 1], -1, True),
    (16, 2, 256, 16, "16bit", "NHD", "bf16", [130, 9], -1, False),
    (9, 1, 256, 64, "16bit", "HND", "fp16", [500, 63], 100, False),
    (5, 1, 128, 16, "16bit", "NHD", "fp16", [90, 3000], 0, True),
    (32, 8, 128, 16, "scaled", "NHD", "bf16", [1, 31, 32, 33, 1000, 0], -1, False),
    (28, 4, 128, 5, "scaled", "HND", "fp16", [300, 129], 64, True),
    (16, 2, 64, 16, "scaled", "NHD", "fp16", [63, 64, 65, 511], -1, False),
    (20, 2, 64, 16, "scaled", "HND", "bf16", [257], -1, True),
    (8, 2, 256, 16, "scaled", "NHD", "bf16", [200, 16], -1, False),
    (64, 8, 128, 16, "block", "NHD", "bf16", [4097, 1, 0, 33], -1, False),
    (24, 2, 128, 16, "block", "HND", "fp16", [300, 65], -1, True),
    (8, 1, 64, 3, "block", "NHD", "fp16", [300, 2], 128, False),
    (9, 1, 64, 16, "block", "HND", "bf16", [700, 70], -1, False),
    (7, 1, 256, 32, "block", "NHD", "fp16", [100, 1], -1, True),
    (130, 2, 64, 16, "16bit", "NHD", "bf16", [70, 200, 1], -1, True),        # 65 heads a KV head
    (66, 1, 256, 16, "scaled", "HND", "fp16", [50], 20, True),
]


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,hk,d,ps,fmt,layout,dtype,lens,window,sinks", DECODES)
def test_decode(H, hk, d, ps, fmt, layout, dtype, lens, window, sinks, wide):
    """Rows under a narrow table go to a CTA or a cluster each, under a wide one to the split kernel."""
    dt = DT[dtype]
    tab, pages = table_of(lens, ps, 1, pad=33000 // ps if wide else 2)
    kv, sc = make_cache(pages, ps, hk, d, layout, fmt, dt, 2)
    # slots behind a request's keys hold NaN (the code 0x7f, or an exponent byte of 255)
    raw = kv.view(torch.uint8) if fmt != "16bit" else kv
    for i, n in enumerate(lens):
        if n % ps:
            p = int(tab[i, n // ps])
            at = (p, slice(None), slice(n % ps, None)) if layout == "NHD" else (p, slice(None), slice(None), slice(n % ps, None))
            raw[at] = float("nan") if fmt == "16bit" else 0x7f
            if fmt == "block":
                sc[at] = 255
    g = torch.Generator().manual_seed(3)
    wide = torch.randn((len(lens), H + 3, d), generator=g).to(dt).cuda()       # rows of a fused projection
    q = wide[:, :H]
    snk = torch.randn(H, generator=g).cuda() if sinks else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = torch.from_numpy(tab).cuda()
    out, lse = pod.pod_paged_decode(q, kv, t, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    window_left=window, sinks=snk, kv_layout=layout, status=status,
                                    **fmt_args(fmt, sc))
    x = values64(kv, sc, layout, fmt)
    scale = 1 / math.sqrt(d)
    ref = [attend64(q[i].double().cpu().numpy(), x, dense_keys(tab[i], n, ps, hk, window), scale,
                    None if snk is None else snk.double().cpu().numpy()) for i, n in enumerate(lens)]
    check(out, lse, *(np.stack(y) for y in zip(*ref)), d, dt, fmt)
    assert status.item() == 0
    for i, n in enumerate(lens):
        if n == 0:
            assert (out[i] == 0).all() and torch.isneginf(lse[i]).all()


@gpu
@pytest.mark.parametrize("hk", [1, 8])
@pytest.mark.parametrize("batch", [1, 5, 9, 17, 40, 130])
def test_decode_widths(batch, hk):
    """One batch under tables of every width: one to eight CTAs a row, and the split kernel."""
    dt, d, ps, H = torch.bfloat16, 128, 16, 4 * hk
    r = np.random.RandomState(batch)
    lens = [int(x) for x in r.randint(0, 400, batch)]
    lens[0], lens[-1] = 0, 5
    tab, pages = table_of(lens, ps, batch + 1)
    kv, _ = make_cache(pages, ps, hk, d, "NHD", "16bit", dt, 3)
    q = torch.from_numpy(r.standard_normal((batch, H, d))).to(dt).cuda()
    x = values64(kv, None, "NHD", "16bit")
    scale = 1 / math.sqrt(d)
    ref = [attend64(q[i].double().cpu().numpy(), x, dense_keys(tab[i], n, ps, hk, -1), scale, None)
           for i, n in enumerate(lens)]
    ref = [np.stack(y) for y in zip(*ref)]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for keys in (0, 500, 1000, 2000, 4000, 9000):
        t = np.concatenate([tab, np.full((batch, keys // ps), -1, np.int32)], 1)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(t).cuda(), n, status=status)
        check(out, lse, *ref, d, dt)
        assert status.item() == 0


@gpu
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("ps,fmt,layout,dtype,d", [(16, "16bit", "NHD", "bf16", 128), (1, "scaled", "HND", "fp16", 128),
                                                   (3, "block", "NHD", "bf16", 64), (64, "16bit", "HND", "fp16", 256)])
def test_decode_of_listed_pages(ps, fmt, layout, dtype, d, wide):
    """Pages per KV head in any order, a page twice, entries that are skipped."""
    dt, hk, G = DT[dtype], 2, 4
    lens = [10 * ps, 7 * ps - min(2, ps - 1), ps, 0, 4 * ps]
    more = 33000 // ps if wide else 0
    tab, pages = table_of(lens, ps, 5, pad=more)
    kv, sc = make_cache(pages, ps, hk, d, layout, fmt, dt, 6)
    sel = np.array([[[3, 1, 9, -1, 0], [2, 2, 8, 5, 10]],        # 10: past the request's pages
                    [[6, 0, -1, -1, -1], [5, 6, 4, 3, 2]],
                    [[0, -1, -1, -1, -1], [-1, 0, 0, 0, 0]],     # one page: only one entry is read
                    [[0, 1, 2, 3, 4], [-1, -1, -1, -1, -1]],
                    [[1 << 30, -7, 2, 1, 0], [99, 4, -1, 77, 0]]], dtype=np.int32)
    sel = np.concatenate([sel, np.full((5, hk, more), -1, np.int32)], -1)
    q = torch.randn((5, hk * G, d), generator=torch.Generator().manual_seed(7)).to(dt).cuda()
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    pages=torch.from_numpy(sel).cuda(), sm_scale=0.1, kv_layout=layout,
                                    **fmt_args(fmt, sc))
    x = values64(kv, sc, layout, fmt)
    ref = []
    for i, n in enumerate(lens):
        keys = []
        for h in range(hk):
            t = [np.arange(p * ps, min(n, (p + 1) * ps)) for p in sel[i, h, :-(-n // ps)].tolist() if 0 <= p * ps < n]
            t = np.concatenate(t + [np.zeros(0, int)]).astype(int)
            keys.append((tab[i][t // ps].astype(np.int64), t % ps))
        ref.append(attend64(q[i].double().cpu().numpy(), x, keys, 0.1, None))
    check(out, lse, *(np.stack(y) for y in zip(*ref)), d, dt, fmt)


@gpu
@pytest.mark.parametrize("width", [5, 2200])
def test_bad_pages_and_lengths_are_masked_and_reported(width):
    """A page outside the pool in front of a request's end, a negative length and
    one past the table: nothing outside is read."""
    ps, hk, H, d, dt = 16, 2, 4, 128, torch.bfloat16
    lens = [80, -5, width * ps + 920, 33]
    tab = np.array([[0, 7, 2, 3, 4], [1, 1, 1, 1, 1], [5, 6, 0, 1, 2], [3, -1, 1 << 30, 0, 0]], dtype=np.int32)
    tab = np.concatenate([tab, np.random.RandomState(4).randint(-1, 8, (4, width - 5)).astype(np.int32)], 1)
    kv, _ = make_cache(7, ps, hk, d, "NHD", "16bit", dt, 1)
    q = torch.randn((4, H, d), generator=torch.Generator().manual_seed(2)).to(dt).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    status=status)
    x = values64(kv, None, "NHD", "16bit")
    ref = []
    for i, n in enumerate(lens):
        t = np.arange(min(max(n, 0), width * ps))
        t = t[(tab[i][t // ps] >= 0) & (tab[i][t // ps] < 7)]
        ref.append(attend64(q[i].double().cpu().numpy(), x, [(tab[i][t // ps].astype(np.int64), t % ps)] * hk,
                            1 / math.sqrt(d), None))
    check(out, lse, *(np.stack(y) for y in zip(*ref)), d, dt)
    assert status.item() == 4


@gpu
@pytest.mark.parametrize("pad", [0, 2100])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_block_scales_far_apart(dtype, pad):
    """K and V exponents over many binades; the largest V scale under a small weight."""
    dt, hk, H, d, ps, n = DT[dtype], 1, 4, 128, 16, 400
    tab, pages = table_of([n], ps, 1, pad=pad)
    kv, sc = make_cache(pages, ps, hk, d, "NHD", "block", dt, 4, 112, 121)
    g = torch.Generator().manual_seed(9)
    sc[:, 1] = torch.randint(100, 126, sc[:, 1].shape, generator=g, dtype=torch.uint8).cuda()
    sc[int(tab[0, 3]), 1, 2] = 0
    q = torch.randn((1, H, d), generator=g).to(dt).cuda()
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"),
                                    kv_scales=sc)
    ref = [attend64(q[0].double().cpu().numpy(), values64(kv, sc, "NHD", "block"), dense_keys(tab[0], n, ps, hk, -1),
                    1 / math.sqrt(d), None)]
    check(out, lse, *(np.stack(y) for y in zip(*ref)), d, dt, "block")


@gpu
def test_large_logits_and_infinite_values():
    """Logits of some thousands, an infinite key (NaN out, for its heads only), large V."""
    ps, hk, H, d, dt, n = 16, 2, 4, 64, torch.bfloat16, 300
    tab, pages = table_of([n, n], ps, 1)
    kv, _ = make_cache(pages, ps, hk, d, "NHD", "16bit", dt, 4)
    kv[:, 0] *= 40
    kv[:, 1] *= 2.0 ** 100
    q = (torch.randn((2, H, d), generator=torch.Generator().manual_seed(3)) * 40).to(dt).cuda()
    lens = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    run = lambda: pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), lens)    # noqa: E731
    out, lse = run()
    x = values64(kv, None, "NHD", "16bit")
    ref = [attend64(q[i].double().cpu().numpy(), x, dense_keys(tab[i], n, ps, hk, -1), 1 / 8, None) for i in range(2)]
    check(out, lse, *(np.stack(y) for y in zip(*ref)), d, dt)
    kv[int(tab[1, 4]), 0, 5, 1] = float("nan")
    again, lse2 = run()
    assert torch.equal(again[0], out[0]) and torch.equal(again[1, :2], out[1, :2])
    assert again[1, 2:].isnan().all() and lse2[1, 2:].isnan().all()


@gpu
def test_decode_repeats_its_bits_and_leaves_other_memory():
    ps, hk, H, d, dt = 16, 8, 32, 128, torch.bfloat16
    lens = [5000, 1, 900, 0, 12000, 3]
    tab, pages = table_of(lens, ps, 1)
    kv, _ = make_cache(pages, ps, hk, d, "NHD", "16bit", dt, 4)
    q = torch.randn((6, H, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    t, ln = torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    need = pod.pod_paged_decode_workspace_size(6, H, hk, d)
    outs = []
    for fill in (0, 255):
        ws = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        big = torch.full((6, H + 2, d), 7.0, dtype=dt, device="cuda")
        out, lse = pod.pod_paged_decode(q, kv, t, ln, workspace=ws[256:256 + need], out=big[:, :H])
        assert (ws[:256] == fill).all() and (ws[256 + need:] == fill).all() and (big[:, H:] == 7).all()
        outs.append((out.clone(), lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@gpu
def test_many_requests_and_many_heads():
    """More requests than a block has threads, most of them empty, and a merge of many rows."""
    ps, hk, H, d, dt = 16, 2, 16, 64, torch.float16
    r = np.random.RandomState(0)
    lens = [int(x) if r.rand() < 0.5 else 0 for x in r.randint(1, 90, 700)]
    lens[650] = 7000
    tab, pages = table_of(lens, ps, 1)
    kv, _ = make_cache(pages, ps, hk, d, "HND", "16bit", dt, 4)
    q = torch.randn((700, H, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    kv_layout="HND")
    x = values64(kv, None, "HND", "16bit")
    at = [0, 1, 2, 650, 651, 699] + list(range(100, 130))
    ref = [attend64(q[i].double().cpu().numpy(), x, dense_keys(tab[i], lens[i], ps, hk, -1), 1 / 8, None) for i in at]
    check(out[at], lse[at], *(np.stack(y) for y in zip(*ref)), d, dt)
    empty = [i for i, n in enumerate(lens) if n == 0]
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()


@gpu
@pytest.mark.parametrize("H,hk,d,ps,fmt,dtype", [(16, 8, 128, 1, "16bit", "bf16"), (48, 4, 64, 3, "block", "fp16"),
                                                 (8, 4, 256, 1, "scaled", "bf16"), (96, 8, 128, 2, "16bit", "fp16")])
def test_small_pages_of_many_requests(H, hk, d, ps, fmt, dtype):
    """Four KV heads a CTA: one warp a head, requests cut between CTAs and empty ones among them."""
    dt, B = DT[dtype], 120
    r = np.random.RandomState(4)
    lens = [int(x) for x in r.choice([0, 1, 5, 63, 64, 65, 200], B)]
    lens[7], lens[60] = 3000, 1111
    tab, pages = table_of(lens, ps, 1, pad=9000 // ps)
    kv, sc = make_cache(pages, ps, hk, d, "NHD", fmt, dt, 2)
    q = torch.randn((B, H, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    snk = torch.randn(H, generator=torch.Generator().manual_seed(8)).cuda()
    out, lse = pod.pod_paged_decode(q, kv, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                    sinks=snk, **fmt_args(fmt, sc))
    x = values64(kv, sc, "NHD", fmt)
    at = [7, 60] + list(range(20, 50)) + [B - 1]
    ref = [attend64(q[i].double().cpu().numpy(), x, dense_keys(tab[i], lens[i], ps, hk, -1), 1 / math.sqrt(d),
                    snk.double().cpu().numpy()) for i in at]
    check(out[at], lse[at], *(np.stack(y) for y in zip(*ref)), d, dt, fmt)


@gpu
def test_two_calls_at_once():
    """Two streams, each with a workspace of its own (given, and made by the call)."""
    ps, hk, H, d, dt = 16, 8, 32, 128, torch.bfloat16
    lens = [3000 + 17 * i for i in range(24)]
    tab, pages = table_of(lens, ps, 1)
    kv, _ = make_cache(pages, ps, hk, d, "NHD", "16bit", dt, 4)
    g = torch.Generator().manual_seed(3)
    qs = [torch.randn((24, H, d), generator=g).to(dt).cuda() for _ in range(2)]
    bounds = make_bounds(pages, hk, d, dt, 5)
    t, ln = torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")

    def step(q, ws=None):
        sel = pod.pod_select_pages(q, bounds, t, ln, 20, ps)
        return (sel,) + pod.pod_paged_decode(q, kv, t, ln, workspace=ws) + pod.pod_paged_decode(q, kv, t, ln, pages=sel)

    want = [step(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    ws = torch.empty(pod.pod_paged_decode_workspace_size(24, H, hk, d), dtype=torch.uint8, device="cuda")
    got = []
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, step(qs[i], ws if i == 0 else None)))
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


@gpu
def test_pool_past_4_gb():
    """Pages whose offsets pass 32 bits, in every call that reads them."""
    ps, hk, H, d, dt = 16, 8, 8, 128, torch.bfloat16
    pages = 80000                                                   # 64 KB each
    kv = torch.empty((pages, 2, ps, hk, d), dtype=dt, device="cuda")
    bounds = torch.empty((pages, hk, 2, d), dtype=dt, device="cuda")
    tab = np.array([[79999, 70000, 3, 66000]], dtype=np.int32)
    small, _ = make_cache(4, ps, hk, d, "NHD", "16bit", dt, 4)
    kv[tab[0].tolist()] = small
    n = 60
    slots = torch.from_numpy((tab[0].astype(np.int64)[np.arange(n) // ps] * ps + np.arange(n) % ps)).cuda()
    pod.pod_page_bounds(kv, bounds, slots)
    k = small[:, 0].clone()
    k[3, n % ps:] = k[3, 0]
    assert torch.equal(bounds[tab[0].tolist()], torch.stack([k.amin(1), k.amax(1)], 2))
    q = torch.randn((1, H, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    t, ln = torch.from_numpy(tab).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda")
    got = pod.pod_select_pages(q, bounds, t, ln, 2, ps)
    assert torch.equal(got.cpu(), select64(q, bounds, tab, [n], ps, 2, 0, 1))
    out, lse = pod.pod_paged_decode(q, kv, t, ln)
    x = values64(small, None, "NHD", "16bit")
    ref = [attend64(q[0].double().cpu().numpy(), x, dense_keys(np.arange(4), n, ps, hk, -1), 1 / math.sqrt(d), None)]
    check(out, lse, *(np.stack(y) for y in zip(*ref)), d, dt)


# ------------------------------------------------------------------ selection
def select64(q, bounds, table, lens, ps, k, first, last):
    b, q = bounds.double().cpu().numpy(), q.double().cpu().numpy()
    hk = b.shape[1]
    G = q.shape[1] // hk
    out = np.full((q.shape[0], hk, k), -1, dtype=np.int32)
    for r, length in enumerate(lens):
        n = -(-min(max(length, 0), table.shape[1] * ps) // ps)
        for h in range(hk):
            pages = table[r, :n].astype(np.int64)
            known = (pages >= 0) & (pages < b.shape[0])
            x = q[r, h * G:(h + 1) * G]
            with np.errstate(invalid="ignore"):
                up, down = np.where(x < 0, 0, x).sum(0), np.where(x > 0, 0, x).sum(0)
                at = b[np.where(known, pages, 0), h]
                score = np.where(known, (at[:, 0] * down + at[:, 1] * up).sum(-1), -np.inf)
            rank = np.where(np.isnan(score), np.inf, score)
            must = set(range(min(first, n))) | set(range(max(0, n - last), n))
            rest = [i for i in np.lexsort((np.arange(n), ~np.isnan(score), -rank)).tolist() if i not in must]
            got = sorted((sorted(must) + rest)[:k])
            out[r, h, :len(got)] = got
    return torch.from_numpy(out)


def make_bounds(pages, hk, d, dt, seed):
    x = torch.randn((2, pages, hk, d), generator=torch.Generator().manual_seed(seed))
    return torch.stack([torch.minimum(x[0], x[1]), torch.maximum(x[0], x[1])], 2).to(dt).cuda()


@gpu
@pytest.mark.parametrize("H,hk,d,ps,dtype,lens,k,first,last", [
    (32, 8, 128, 16, "bf16", [1, 0, 100, 2000, 4096, 511], 16, 1, 2),
    (4, 4, 64, 8, "fp16", [3000, 40, 8], 5, 0, 1),
    (24, 2, 256, 16, "bf16", [700, 1600], 33, 2, 4),
    (7, 1, 128, 1, "fp16", [500, 77], 64, 0, 0),
    (5, 1, 64, 3, "bf16", [1000, 17, 6], 6, 3, 3),
    (16, 1, 128, 64, "bf16", [9000], 1, 0, 0),
    (2, 1, 64, 1, "bf16", [9500, 8192, 8193], 300, 1, 1),
])
def test_select(H, hk, d, ps, dtype, lens, k, first, last):
    dt = DT[dtype]
    tab, pages = table_of(lens, ps, 3, pad=1)
    bounds = make_bounds(pages, hk, d, dt, 4)
    wide = torch.randn((len(lens), H + 1, d), generator=torch.Generator().manual_seed(5)).to(dt).cuda()
    got = pod.pod_select_pages(wide[:, 1:], bounds, torch.from_numpy(tab).cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), k, ps, keep_first=first,
                               keep_last=last)
    assert torch.equal(got.cpu(), select64(wide[:, 1:], bounds, tab, lens, ps, k, first, last))


@gpu
@pytest.mark.parametrize("width,dtype", [(90, "bf16"), (2100, "fp16"), (4200, "bf16")])
def test_select_of_many_rows(width, dtype):
    """More choices than SMs, rows of every length, pages that requests share (so many
    scores of a row are equal)."""
    dt, B, hk, d, k = DT[dtype], 160, 2, 64, 40
    r = np.random.RandomState(width)
    tab = r.randint(0, 300, (B, width)).astype(np.int32)
    tab[::2] = r.permutation(300)[:min(width, 300)][np.arange(width) % min(width, 300)]
    lens = r.randint(0, width * 4 + 1, B).tolist()
    bounds = make_bounds(300, hk, d, dt, 4)
    q = torch.randn((B, 8, d), generator=torch.Generator().manual_seed(5)).to(dt).cuda()
    got = pod.pod_select_pages(q, bounds, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               k, 4, keep_first=2, keep_last=3)
    assert torch.equal(got.cpu(), select64(q, bounds, tab, lens, 4, k, 2, 3))


@gpu
def test_select_ties_and_scores_that_fp32_cannot_tell_apart():
    ps, hk, d, dt, n = 16, 1, 128, torch.bfloat16, 300
    tab, pages = table_of([n * ps] * 4, ps, 3)
    t = torch.from_numpy(tab).cuda()
    lens = torch.tensor([n * ps] * 4, dtype=torch.int32, device="cuda")
    r = np.random.RandomState(1)
    bounds = torch.zeros((pages, hk, 2, d))
    # every page scores 2^20, but for one part of it 2^-10 .. 2^-4 in a channel of its own: less
    # than an fp32 sum of this size can hold
    bounds[:, 0, 1, 0] = 1024.0
    for row in range(4):
        for p in range(n):
            bounds[int(tab[row, p]), 0, 1, 1 + p % 100] = 2.0 ** -float(r.randint(4, 11))
    bounds = bounds.to(dt).cuda()
    q = torch.ones((4, 2, d))
    q[:, :, 0] = 512.0
    q[2] = 0.0                                             # all equal: the lowest positions
    q[3, :, 0] = 0.0                                       # many equal scores
    q = q.to(dt).cuda()
    for k in (1, 7, 150, 299):
        got = pod.pod_select_pages(q, bounds, t, lens, k, ps, keep_last=0)
        assert torch.equal(got.cpu(), select64(q, bounds, tab, [n * ps] * 4, ps, k, 0, 0))
    assert got[2, 0, :].tolist() == list(range(299))


@gpu
def test_select_with_infinite_and_nan_bounds_and_bad_pages():
    ps, hk, d, dt = 16, 2, 64, torch.float16
    lens = [100 * ps, 50 * ps, 100 * ps, 2000 * ps]
    tab, pages = table_of([100 * ps] * 3, ps, 3)
    bounds = make_bounds(pages, hk, d, dt, 4)
    bounds[int(tab[0, 40]), 0, 1, 3] = float("nan")
    bounds[int(tab[0, 50]), 1, 1, 3] = float("inf")
    bounds[int(tab[1, 20]), 0, 0, 5] = float("-inf")
    tab = np.concatenate([tab, tab[:1]])
    tab[2, 10], tab[2, 11] = -1, pages
    q = torch.randn((4, 4, d), generator=torch.Generator().manual_seed(5)).to(dt).cuda()
    q[1, 3, 5] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = pod.pod_select_pages(q, bounds, torch.from_numpy(tab).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               99, ps, status=status)
    assert torch.equal(got.cpu(), select64(q, bounds, tab, lens, ps, 99, 0, 1)) and status.item() == 4
    assert 40 in got[0, 0].tolist()


# ------------------------------------------------------------------ bounds
def outward(lo, hi, dt):
    big = torch.finfo(dt).max
    out = []
    for x, up in ((lo, False), (hi, True)):
        x = x.double().clamp(-big, big)
        y = x.to(dt)
        off = y.double() < x if up else y.double() > x
        inf = torch.full_like(y.float(), math.inf if up else -math.inf).to(dt)
        out.append(torch.where(off, step_toward(y, inf), y))
    return torch.stack(out, -2)


def step_toward(y, inf):
    b = y.view(torch.int16).int()
    up = inf.float() > 0
    s = torch.where(y == 0, torch.where(up, 1, -32767), b + torch.where((b >= 0) == up, 1, -1))
    return s.to(torch.int16).view(y.dtype)


@gpu
@pytest.mark.parametrize("hk,d,ps,fmt,layout,dtype,runs", [
    (8, 128, 16, "16bit", "NHD", "bf16", [(0, 1), (5, 1), (15, 1), (16, 1), (31, 40)]),
    (2, 64, 8, "16bit", "HND", "fp16", [(0, 200), (3, 5)]),
    (1, 256, 3, "16bit", "NHD", "bf16", [(1, 1), (2, 7)]),
    (4, 128, 32, "scaled", "HND", "bf16", [(0, 33), (40, 1), (63, 2)]),
    (3, 64, 1, "scaled", "NHD", "fp16", [(0, 9)]),
    (2, 256, 64, "scaled", "NHD", "fp16", [(10, 130)]),
    (8, 128, 16, "block", "NHD", "fp16", [(0, 50), (7, 9), (31, 1)]),
    (1, 64, 5, "block", "HND", "bf16", [(4, 11)]),
    (2, 256, 100, "block", "HND", "bf16", [(0, 250)]),
])
def test_bounds(hk, d, ps, fmt, layout, dtype, runs):
    dt = DT[dtype]
    need = [(a + n - 1) // ps - a // ps + 1 for a, n in runs]
    pages = sum(need) + 3
    kv, sc = make_cache(pages, ps, hk, d, layout, fmt, dt, 2)
    perm = np.random.RandomState(1).permutation(pages)
    slots, at, last = [], 0, {}
    for (a, n), m in zip(runs, need):
        t = np.arange(a, a + n)
        page = perm[at + t // ps - a // ps]
        at += m
        slots += (page * ps + t % ps).tolist() + [-1] * (len(slots) % 3)
        for p, i in zip(page.tolist(), (t % ps).tolist()):
            last[p] = i
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = torch.tensor(slots + [pages * ps], device="cuda")
    bounds = torch.full((pages, hk, 2, d), 5.0, dtype=dt, device="cuda")
    want = bounds.cpu().clone()
    x = kv.cpu().float()
    if fmt == "scaled":
        x *= np.float32(K_SCALE)
    elif fmt == "block":
        x = x * torch.exp2(sc.cpu().float() - 127)[..., None]
    x = (x if layout == "NHD" else x.transpose(2, 3))[:, 0]
    for p, i in last.items():
        want[p] = outward(x[p, :i + 1].amin(0), x[p, :i + 1].amax(0), dt)
    a = dict(k_scale=K_SCALE) if fmt == "scaled" else dict(kv_scales=sc) if fmt == "block" else {}
    for _ in range(2):                                     # (again: the same)
        got = pod.pod_page_bounds(kv, bounds, sl, kv_layout=layout, status=status, **a)
        assert got is bounds and torch.equal(bounds.cpu(), want)
    assert status.item() == 4


@gpu
@pytest.mark.parametrize("hk,d,ps,layout,dtype", [(2, 128, 16, "NHD", "bf16"), (1, 64, 40, "HND", "fp16"),
                                                  (3, 256, 70, "NHD", "bf16"), (1, 128, 5, "HND", "fp16")])
def test_bounds_of_scales_far_apart(hk, d, ps, layout, dtype):
    """Exponents of a page within 15 binades, at 16, and over the whole range; results past fp16's."""
    dt, pages = DT[dtype], 5
    kv, sc = make_cache(pages, ps, hk, d, layout, "block", dt, 2)
    g = torch.Generator().manual_seed(7)
    half = sc[:, 0]
    for p, (lo, hi) in enumerate([(110, 126), (110, 127), (0, 255), (0, 16), (120, 160)]):
        half[p] = torch.randint(lo, hi, half[p].shape, generator=g, dtype=torch.int64).to(torch.uint8).cuda()
        half[p].view(-1)[0], half[p].view(-1)[-1] = lo, hi - 1
    slots = torch.arange(pages * ps, device="cuda")
    bounds = torch.zeros((pages, hk, 2, d), dtype=dt, device="cuda")
    pod.pod_page_bounds(kv, bounds, slots, kv_scales=sc, kv_layout=layout)
    x = kv.cpu().float() * torch.exp2(sc.cpu().double() - 127).float()[..., None]
    x = (x if layout == "NHD" else x.transpose(2, 3))[:, 0]
    want = torch.stack([outward(x[p].amin(0), x[p].amax(0), dt) for p in range(pages)])
    assert torch.equal(bounds.cpu(), want)


@gpu
def test_bounds_of_odd_values():
    """Infinities end at the largest number, NaN does not count, fp16 bounds of small codes."""
    kv = torch.zeros((1, 2, 4, 1, 64), dtype=torch.float16, device="cuda")
    kv[0, 0, :, 0, 0] = torch.tensor([1.0, math.inf, 2.0, -3.0])
    kv[0, 0, :, 0, 1] = torch.tensor([math.nan, 7.0, math.nan, 8.0])
    kv[0, 0, :, 0, 2] = torch.tensor([-math.inf, 7.0, 5.0, 6e-8])
    bounds = torch.empty((1, 1, 2, 64), dtype=torch.float16, device="cuda")
    pod.pod_page_bounds(kv, bounds, torch.arange(4, device="cuda"))
    assert bounds[0, 0, :, :3].T.tolist() == [[-3.0, 65504.0], [7.0, 8.0], [-65504.0, 7.0]]
    codes = torch.zeros((1, 2, 4, 1, 64), dtype=torch.float8_e4m3fn, device="cuda")
    codes[0, 0, 0, 0, 0] = 1.0
    codes[0, 0, 1, 0, 1] = -1.0
    sc = torch.full((1, 2, 4, 1), 90, dtype=torch.uint8, device="cuda")      # 2^-37: below fp16
    pod.pod_page_bounds(codes, bounds, torch.arange(4, device="cuda"), kv_scales=sc)
    tiny = 2.0 ** -24
    assert bounds[0, 0, :, :2].T.tolist() == [[0.0, tiny], [-tiny, 0.0]]


# ------------------------------------------------------------------ step tables
def step_ref(table, lens, new, free, count, ps, max_rows, max_pages):
    """The step as a loop over the requests, on the host."""
    table, free = table.copy(), free.copy()
    B, W = table.shape
    status, now, old = 0, [], []
    count = min(max(count, 0), len(free))
    for n in lens:
        old.append(min(max(n, 0), W * ps))
        status |= 4 if old[-1] != n else 0
    pages = lambda x: -(-x // ps)                          # noqa: E731
    for r in range(B):
        now.append(old[r] if new[r] >= 0 else max(0, old[r] + new[r]))
        for p in range(pages(now[r]), pages(old[r])):
            if count < len(free):
                free[count] = table[r, p]
                count += 1
            else:
                status |= 8
    rows, closed, indptr = [], False, [0]
    want_pages = want_rows = 0
    top = count
    for r in range(B):
        if new[r] > 0 and old[r] + new[r] > W * ps:
            status |= 8
        elif new[r] > 0:
            need = pages(old[r] + new[r]) - pages(old[r])
            want_pages, want_rows = want_pages + need, want_rows + new[r]
            closed |= want_pages > top or want_rows > max_rows
            if closed:
                status |= 8
            else:
                now[r] = old[r] + new[r]
                for p in range(pages(old[r]), pages(now[r])):
                    count -= 1
                    table[r, p] = free[count]
                for t in range(old[r], now[r]):
                    page = int(table[r, t // ps])
                    rows.append((r, t, page * ps + t % ps if page >= 0 else -1))
        indptr.append(len(rows))
    rows += [(-1, 0, -1)] * (max_rows - len(rows))
    kv_indptr = np.concatenate([[0], np.cumsum([pages(x) for x in now])])
    flat = [int(x) for r in range(B) for x in table[r, :pages(now[r])]]
    if len(flat) > max_pages and max_pages:
        status |= 8
    flat = (flat + [-1] * max_pages)[:max_pages]
    cols = list(zip(*rows)) if rows else [[], [], []]
    return dict(table=table, free=free, free_count=[count], kv_lens=now, q_indptr=indptr, requests=cols[0],
                positions=cols[1], slots=cols[2], kv_indptr=kv_indptr, kv_indices=flat,
                last_page_len=[(x - 1) % ps + 1 if x else 0 for x in now]), status


def run_step(table, lens, new, free, count, ps, max_rows, max_pages=0, in_place=True, stride=0):
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")    # noqa: E731
    B, W = table.shape
    wide = torch.full((B, W + stride), -9, dtype=torch.int32, device="cuda")
    wide[:, :W] = torch.from_numpy(table).cuda()
    lens_t, free_t, count_t, status = dev(lens), dev(free), dev([count]), dev([0])
    kw = {} if in_place else dict(kv_lens_out=torch.empty_like(lens_t), free_count_out=torch.empty_like(count_t))
    t = pod.pod_step_tables(wide[:, :W], lens_t, dev(new), free_t, count_t, ps, max_rows=max_rows, max_pages=max_pages,
                            status=status, **kw)
    assert (wide[:, W:] == -9).all()
    got = dict(table=wide[:, :W], free=free_t, free_count=count_t if in_place else kw["free_count_out"],
               kv_lens=t.kv_lens, q_indptr=t.q_indptr, requests=t.requests, positions=t.positions, slots=t.slots)
    if max_pages:
        got.update(kv_indptr=t.kv_indptr, kv_indices=t.kv_indices, last_page_len=t.last_page_len)
    if not in_place:
        assert lens_t.tolist() == list(lens) and count_t.item() == count
    return got, status.item()


def compare_step(*a, **k):
    got, status = run_step(*a, **k)
    want, wstatus = step_ref(*a[:7], a[7] if len(a) > 7 else k.get("max_pages", 0))
    for name, x in got.items():
        assert np.array_equal(x.cpu().numpy(), np.asarray(want[name])), name
    assert status == wstatus
    return got, status


@gpu
@pytest.mark.parametrize("B,W,ps,rows,pages,seed", [(1, 4, 16, 8, 0, 1), (64, 40, 16, 64, 0, 2), (5, 9, 3, 500, 60, 3),
                                                    (130, 30, 1, 3000, 0, 4), (1030, 12, 16, 4000, 9000, 5),
                                                    (2100, 6, 16, 2100, 0, 6)])
def test_step_tables(B, W, ps, rows, pages, seed):
    r = np.random.RandomState(seed)
    perm = r.permutation(B * W + 5).astype(np.int32)
    table = perm[:B * W].reshape(B, W).copy()
    lens = r.randint(0, W * ps + 1, B)
    kind = r.rand(B)
    new = np.where(kind < 0.5, 1, np.where(kind < 0.6, r.randint(1, 2 * ps + 2, B), np.where(kind < 0.8, 0, -r.randint(1, 3 * ps + 1, B))))
    free = np.concatenate([perm[B * W:], perm[:B]]).astype(np.int32)
    free = np.concatenate([free, np.full(B * W, -3, np.int32)])
    for count in (B + 5, 3, 0):
        compare_step(table, lens, new, free, count, ps, rows, pages, in_place=count != 3, stride=count % 4)


@gpu
def test_step_tables_at_their_limits():
    table = np.arange(12, dtype=np.int32).reshape(3, 4) + 50
    free = np.arange(100, 110, dtype=np.int32)
    for lens, new, count, rows in [
            ([0, 0, 0], [0, 0, 0], 10, 4),                 # nothing to do
            ([64, 63, 1], [1, 1, 1], 10, 4),               # the first is at the end of its table row
            ([16, 16, 16], [1, 1, 1], 2, 4),               # pages for two
            ([16, 5, 16], [17, 1, 1], 2, 4),               # rows run out at once: nobody behind grows either
            ([16, 5, 16], [1, 3, 1], 9, 4),                # rows for the first two
            ([70, -3, 64], [1, 2, -64], 10, 4),            # lengths out of range
            ([3, 3, 3], [-10, -3, -2], 0, 1),              # down to nothing
            ([64, 64, 64], [-64, -64, -64], 3, 1),         # a full stack: ten of twelve and three
            ([0, 0, 0], [2 ** 31 - 1] * 3, 10, 4),
            ([64, 0, 64], [-(2 ** 31), 64, -17], 0, 64),   # pages given back serve at once
            ([20, 33, 7], [1, 1, 1], -4, 4),               # a count out of range
            ([20, 33, 7], [12, 1, 1], 400, 64)]:
        compare_step(table, lens, new, free, count, 16, rows, 8)
        compare_step(table, lens, new, free, count, 16, rows)


@gpu
def test_step_tables_into_kept_arrays():
    """The arrays of an earlier step, with and without the page table; other memory stays."""
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")    # noqa: E731
    table = torch.arange(24, dtype=torch.int32, device="cuda").view(4, 6) + 100
    free, count = dev(list(range(60))), dev([50])
    lens = dev([15, 0, 33, 96])
    first = pod.pod_step_tables(table, lens, dev([1, 5, -3, 0]), free, count, 16, max_rows=9, max_pages=30)
    kept = [x.clone() for x in first]
    again = pod.pod_step_tables(table, lens, dev([2, 1, 1, -96]), free, count, 16, max_rows=9, max_pages=30, out=first)
    assert all(a is b for a, b in zip(again, first)) and again.kv_lens is lens
    assert again.kv_lens.tolist() == [18, 6, 31, 0] and again.q_indptr.tolist() == [0, 2, 3, 4, 4]
    assert again.positions.tolist() == [16, 17, 5, 30, 0, 0, 0, 0, 0] and again.slots.tolist()[4:] == [-1] * 5
    assert again.last_page_len.tolist() == [2, 6, 15, 0] and kept[1].tolist() == [0, 1, 6, 6, 6]
    plain = pod.pod_step_tables(table, lens, dev([1, 1, 1, 1]), free, count, 16, max_rows=9, out=first)
    assert plain.kv_indptr is None and plain.slots is first.slots and first.kv_indptr.tolist() == [0, 2, 3, 5, 5]
    for bad in (first._replace(slots=first.slots[:8]), first._replace(requests=first.slots), first._replace(kv_indices=None)):
        with pytest.raises(pod.PodError):
            pod.pod_step_tables(table, lens, dev([1, 1, 1, 1]), free, count, 16, max_rows=9, max_pages=30, out=bad)


@gpu
def test_step_tables_of_nothing():
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    count = torch.tensor([2], dtype=torch.int32, device="cuda")
    t = pod.pod_step_tables(torch.empty((0, 3), dtype=torch.int32, device="cuda"), empty, empty,
                            torch.zeros(4, dtype=torch.int32, device="cuda"), count, 16, max_rows=3, max_pages=2)
    assert t.q_indptr.tolist() == [0] and t.requests.tolist() == [-1] * 3 and t.slots.tolist() == [-1] * 3
    assert t.kv_indptr.tolist() == [0] and t.kv_indices.tolist() == [-1, -1] and count.item() == 2
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device="cuda")
    kv = torch.zeros((2, 2, 16, 2, 64), dtype=torch.float16, device="cuda")
    tab = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    out, lse = pod.pod_paged_decode(q, kv, tab, empty)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    b = torch.zeros((2, 2, 2, 64), dtype=torch.float16, device="cuda")
    assert pod.pod_select_pages(q, b, tab, empty, 2, 16).shape == (0, 2, 2)
    pod.pod_page_bounds(kv, b, torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert (b == 0).all()


# ------------------------------------------------------------------ the step as a whole
@gpu
@pytest.mark.parametrize("fmt,layout,dtype", [("16bit", "NHD", "bf16"), ("block", "HND", "fp16"), ("scaled", "NHD", "bf16")])
def test_one_captured_step_serves_the_later_ones(fmt, layout, dtype):
    """Tables, norm and rotation with the cache write, bounds, selection, attention:
    captured once, replayed while requests grow over page borders, pause, give
    tokens back and start over; the dense attention and the sparse one share a workspace."""
    dt, H, hk, d, ps, B, W, k = DT[dtype], 8, 2, 64, 4, 5, 40, 6
    pages = 60
    kv, sc = make_cache(pages, ps, hk, d, layout, fmt, dt, 1)
    bounds = torch.zeros((pages, hk, 2, d), dtype=dt, device="cuda")
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")    # noqa: E731
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    lens, new, free, count, status = dev([0] * B), dev([0] * B), dev(list(range(pages))), dev([pages]), dev([0])
    R = 64
    qkv = torch.zeros((R, H + 2 * hk, d), dtype=dt, device="cuda")
    w = (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(2))).to(dt).cuda()
    ws = torch.empty(max(pod.pod_paged_decode_workspace_size(B, H, hk, d), pod.pod_select_pages_workspace_size(B, hk, W)),
                     dtype=torch.uint8, device="cuda")
    fa = fmt_args(fmt, sc)
    fb = {x: y for x, y in fa.items() if x != "v_scale"}
    last = torch.zeros((B, H, d), dtype=dt, device="cuda")

    def step():
        t = pod.pod_step_tables(table, lens, new, free, count, ps, max_rows=R, status=status)
        q = pod.pod_norm_rope_append(qkv[:, :H], qkv[:, H:H + hk], qkv[:, H + hk:], t.positions, kv, t.slots,
                                     q_weight=w, k_weight=w, kv_layout=layout, status=status, **fa)
        pod.pod_page_bounds(kv, bounds, t.slots, kv_layout=layout, status=status, **fb)
        # the last row of every request that has one, its query of before otherwise
        at = (t.q_indptr[1:] - 1).long()
        has = (t.q_indptr[1:] > t.q_indptr[:-1])[:, None, None]
        last.copy_(torch.where(has, q[at.clamp(min=0)], last))
        sel = pod.pod_select_pages(last, bounds, table, lens, k, ps, keep_first=1, keep_last=1, workspace=ws, status=status)
        return (t, sel) + pod.pod_paged_decode(last, kv, table, lens, pages=sel, kv_layout=layout, workspace=ws,
                                               status=status, **fa) + \
            pod.pod_paged_decode(last, kv, table, lens, kv_layout=layout, workspace=ws, status=status, **fa)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()                                             # (nothing grows: a warm-up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t, sel, out_s, lse_s, out_d, lse_d = step()
    host = [0] * B
    r = np.random.RandomState(3)
    plan = [[9, 1, 30, 0, 2], [1, 1, 1, 1, 1], [1, 0, 1, 3, 1], [1, 1, -7, 1, 1], [1, 3, 1, 1, 1], [1, 1, 1, 1, -4],
            [-100, 1, 1, 1, 1], [5, 1, 1, 1, 1]] + [[1] * B] * 6
    for i, n in enumerate(plan):
        qkv.copy_(torch.from_numpy(r.randn(*qkv.shape)).to(dt))
        new.copy_(dev(n))
        graph.replay()
        torch.cuda.synchronize()
        host = [max(0, a + b) for a, b in zip(host, n)]
        assert lens.tolist() == host and status.item() == 0
        tab = table.cpu().numpy()
        held = [int(x) for q_, m in enumerate(host) for x in tab[q_, :-(-m // ps)]]
        assert len(set(held)) == len(held) and set(held) | set(free[:count.item()].tolist()) == set(range(pages))
        x = values64(kv, sc, layout, fmt)
        for q_, m in enumerate(host):                      # bounds hold every key of the page
            for p in range(-(-m // ps)):
                keys = x[int(tab[q_, p]), 0, :min(ps, m - p * ps)]
                b = bounds[int(tab[q_, p])].double().cpu()
                # (a product code * k_scale has 28 bits and is rounded to fp32's 24 before it is
                # rounded outward: 2^-24 of it; the other formats' values are exact)
                slack = keys.abs().amax(0) * (2.0 ** -24 if fmt == "scaled" else 0.0)
                assert (b[:, 0] <= keys.amin(0) + slack).all() and (b[:, 1] >= keys.amax(0) - slack).all()
        assert torch.equal(sel.cpu(), select64(last, bounds, tab, host, ps, k, 1, 1))
        for out, lse, sparse in ((out_s, lse_s, True), (out_d, lse_d, False)):
            ref = []
            for q_, m in enumerate(host):
                keys = dense_keys(tab[q_], m, ps, hk, -1)
                if sparse:
                    keys = []
                    for h in range(hk):
                        c = [np.arange(p * ps, min(m, p * ps + ps)) for p in sel[q_, h].tolist() if p >= 0]
                        c = np.concatenate(c + [np.zeros(0, int)]).astype(int)
                        keys.append((tab[q_][c // ps].astype(np.int64), c % ps))
                ref.append(attend64(last[q_].double().cpu().numpy(), x, keys, 1 / 8, None))
            check(out, lse, *(np.stack(y) for y in zip(*ref)), d, dt, fmt)


@gpu
def test_step_tables_feed_the_host_planner():
    """The device's page table, copied to the host, is what pod_plan reads; the decode
    halves agree."""
    H, hk, d, ps, dt = 32, 8, 128, 16, torch.bfloat16
    lens = [40, 200, 1, 64]
    tab, pages = table_of([x + 16 for x in lens], ps, 1)
    kv, _ = make_cache(pages, ps, hk, d, "NHD", "16bit", dt, 4)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")    # noqa: E731
    table = torch.from_numpy(tab).cuda()
    t = pod.pod_step_tables(table, dev(lens), dev([1] * 4), dev([0, 1, 2, 3]), dev([4]), ps, max_rows=4, max_pages=64)
    n = t.kv_indptr[-1].item()
    h = pod.pod_plan(None, None, None, None, np.arange(5, dtype=np.int32), t.kv_indptr.cpu(), t.kv_indices[:n].cpu(),
                     t.last_page_len.cpu(), H, hk, d, ps, dtype=dt, p_num_pages=0, d_num_pages=pages)
    ws = torch.empty(pod.pod_workspace_size(h), dtype=torch.uint8, device="cuda")
    pod.pod_bind_workspace(h, ws)
    q = torch.randn((4, H, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    _, _, want, wlse = pod.pod_run(h, None, None, q, kv, ws)
    out, lse = pod.pod_paged_decode(q, kv, table, t.kv_lens)
    # (pod_run rounds each weight once to bf16: 2^-8 of it)
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -8 * 3 * kv[:, 1].abs().max()
    assert (lse - wlse).abs().max() <= 1e-3


@gpu
def test_other_streams_and_kept_outputs():
    ps, hk, H, d, dt, n = 16, 2, 8, 128, torch.float16, 500
    tab, pages = table_of([n, n], ps, 1)
    kv, _ = make_cache(pages, ps, hk, d, "NHD", "16bit", dt, 4)
    q = torch.randn((2, H, d), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    t, ln = torch.from_numpy(tab).cuda(), torch.tensor([n, n], dtype=torch.int32, device="cuda")
    want, wl = pod.pod_paged_decode(q, kv, t, ln)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        out, lse = pod.pod_paged_decode(q, kv, t, ln, stream=stream)
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    keep, kl = torch.empty_like(want), torch.empty_like(wl)
    out, lse = pod.pod_paged_decode(q, kv, t, ln, out=keep, lse=kl)
    assert out is keep and lse is kl and torch.equal(keep, want) and torch.equal(kl, wl)


# ------------------------------------------------------------------ refusals
@gpu
def test_refusals_of_the_binding():
    ps, hk, H, d = 16, 2, 8, 128
    kv = torch.zeros((4, 2, ps, hk, d), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, H, d), dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    tab, ln = torch.zeros((2, 3), **i32), torch.zeros(2, **i32)
    b = torch.zeros((4, hk, 2, d), dtype=torch.bfloat16, device="cuda")
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    calls = [
        lambda: pod.pod_paged_decode(q.cpu(), kv, tab, ln),
        lambda: pod.pod_paged_decode(q.float(), kv, tab, ln),
        lambda: pod.pod_paged_decode(q.half(), kv, tab, ln),
        lambda: pod.pod_paged_decode(q, kv, tab.long(), ln),
        lambda: pod.pod_paged_decode(q, kv, tab[:1], ln),
        lambda: pod.pod_paged_decode(q, kv, tab.T.contiguous().T, ln),
        lambda: pod.pod_paged_decode(q, kv, tab, ln[:1]),
        lambda: pod.pod_paged_decode(q, kv, tab, ln, pages=torch.zeros((2, 3, 4), **i32)),
        lambda: pod.pod_paged_decode(q, kv, tab, ln, pages=torch.zeros((2, 2, 4), **i32), window_left=3),
        lambda: pod.pod_paged_decode(q, kv, tab, ln, pages=torch.zeros((2, 2, 0), **i32)),
        lambda: pod.pod_paged_decode(q, kv, tab, ln, sinks=torch.zeros(3, device="cuda")),
        lambda: pod.pod_paged_decode(q, kv, tab, ln, workspace=small),
        lambda: pod.pod_paged_decode(q, kv, tab, ln, sm_scale=math.inf),
        lambda: pod.pod_paged_decode(q, kv, tab, ln, window_left=-2),
        lambda: pod.pod_paged_decode(q[:, :7], kv, tab, ln),
        lambda: pod.pod_paged_decode(q, kv, tab, ln, kv_layout="DHN"),
        lambda: pod.pod_paged_decode(q, kv, tab, ln, kv_scales=small),
        lambda: pod.pod_paged_decode(q, kv, tab, ln, out=q.new_empty((2, H, 64))),
        lambda: pod.pod_select_pages(q, b, tab, ln, 0, ps),
        lambda: pod.pod_select_pages(q, b, tab, ln, 2, ps, keep_first=2, keep_last=1),
        lambda: pod.pod_select_pages(q, b, tab, ln, 2, ps, keep_first=-1),
        lambda: pod.pod_select_pages(q, b[..., :64], tab, ln, 2, ps),
        lambda: pod.pod_select_pages(q, b.half(), tab, ln, 2, ps),
        lambda: pod.pod_select_pages(q, b, tab, ln, 2, ps, workspace=small),
        lambda: pod.pod_select_pages(q, b, tab, ln, 2, 1 << 30),
        lambda: pod.pod_page_bounds(kv, b[:3], ln.long()),
        lambda: pod.pod_page_bounds(kv, b.float(), ln.long()),
        lambda: pod.pod_page_bounds(kv, b, ln),
        lambda: pod.pod_page_bounds(kv.half(), b, ln.long()),
        lambda: pod.pod_step_tables(tab, ln, ln[:1], ln, ln[:1], ps, max_rows=2),
        lambda: pod.pod_step_tables(tab, ln, ln, ln, ln, ps, max_rows=2),
        lambda: pod.pod_step_tables(tab, ln, ln, ln, ln[:1], 0, max_rows=2),
        lambda: pod.pod_step_tables(tab, ln, ln, ln, ln[:1], ps, max_rows=-1),
        lambda: pod.pod_step_tables(tab, ln, ln.long(), ln, ln[:1], ps, max_rows=1),
        lambda: pod.pod_step_tables(tab, ln, ln, ln, ln[:1], ps, max_rows=2, max_pages=2,
                                    out=pod.PodStep(None, ln.new_zeros(3), ln, ln, ln.long())),
    ]
    for i, c in enumerate(calls):
        with pytest.raises(pod.PodError):
            c()
            pytest.fail(f"call {i}")


# (fields of the two structs, in order)
STEP = "table lens new lens_out free count count_out q_indptr requests positions slots kv_indptr kv_indices last status " \
       "stride batch width ps capacity max_rows max_pages".split()
DEC = "q cache scales bounds table lens pages slots sinks out lse ws status q_stride out_stride stride num_pages rows " \
      "ws_bytes batch width ps H Hk d layout fmt dtype k first last window sm k_scale v_scale".split()


def c_call(fn, names, packer, **over):
    base = dict(table=256, lens=256, new=256, lens_out=256, free=256, count=256, count_out=256, q_indptr=256, requests=256,
                positions=256, slots=256, kv_indptr=0, kv_indices=0, last=0 if names is STEP else 1, status=0, stride=8,
                batch=2, width=8, ps=16, capacity=8, max_rows=4, max_pages=0, q=256, cache=256, scales=0, bounds=256,
                pages=256, sinks=0, out=256, lse=256, ws=256, q_stride=1024, out_stride=1024, num_pages=8, rows=4,
                ws_bytes=1 << 30, H=8, Hk=2, d=128, layout=0, fmt=0, dtype=1, k=4, first=0, window=-1, sm=0.0,
                k_scale=1.0, v_scale=1.0)
    base.update(over)
    return fn(packer.pack(*(base[n] for n in names)), None)


def test_refusals_of_the_c_calls():
    """Checked before anything is launched: no GPU is needed. (All pointers are made up.)"""
    lib = pod.load_library()
    bad = {
        "pod_step_tables": [dict(table=0), dict(lens=0), dict(new=0), dict(lens_out=0), dict(free=0), dict(count=0),
                            dict(count_out=0), dict(q_indptr=0), dict(requests=0), dict(positions=0), dict(slots=0),
                            dict(kv_indptr=256), dict(kv_indptr=256, last=256, max_pages=3), dict(batch=-1), dict(ps=0),
                            dict(width=0), dict(width=1 << 27), dict(stride=7), dict(max_rows=-1), dict(max_pages=-1),
                            dict(capacity=-1)],
        "pod_page_bounds": [dict(cache=0), dict(cache=8), dict(cache=272), dict(bounds=0), dict(bounds=8), dict(slots=0), dict(rows=-1),
                            dict(rows=1 << 31), dict(d=96), dict(dtype=2), dict(fmt=3), dict(fmt=2), dict(scales=256),
                            dict(layout=2), dict(Hk=0), dict(ps=0), dict(num_pages=0), dict(num_pages=1 << 40),
                            dict(fmt=1, k_scale=0.0), dict(fmt=1, k_scale=math.inf)],
        "pod_select_pages": [dict(q=0), dict(q=8), dict(q_stride=1023), dict(q_stride=1025), dict(bounds=0), dict(bounds=8),
                             dict(table=0), dict(lens=0), dict(pages=0), dict(ws=0), dict(ws=264), dict(ws_bytes=100),
                             dict(k=0), dict(first=-1), dict(first=4), dict(last=-1), dict(batch=-1), dict(H=7), dict(H=0),
                             dict(width=0), dict(stride=7), dict(d=32), dict(dtype=5)],
        "pod_paged_decode": [dict(q=0), dict(q=8), dict(q_stride=1000), dict(cache=0), dict(out=0), dict(out=8),
                             dict(out_stride=1000), dict(out_stride=1028), dict(table=0), dict(lens=0), dict(ws=0),
                             dict(ws_bytes=1000), dict(ws=128), dict(window=-2), dict(window=5), dict(k=0),
                             dict(sm=math.nan), dict(fmt=1, v_scale=-1.0), dict(fmt=2), dict(d=100), dict(H=9),
                             dict(ps=0), dict(num_pages=1 << 33), dict(batch=-3), dict(width=1 << 30)],
    }
    for name, cases in bad.items():
        fn = getattr(lib, name)
        names, packer = (STEP, pod._STEP_ARGS) if name == "pod_step_tables" else (DEC, pod._DECODE_ARGS)
        assert fn(None, None) == 1
        for over in cases:
            code = c_call(fn, names, packer, **over)
            assert code in (1, 2, 3), (name, over, code)
            assert pod.pod_last_error(), (name, over)
    # nothing to do: accepted without a launch
    assert c_call(lib.pod_page_bounds, DEC, pod._DECODE_ARGS, rows=0, slots=0) == 0
    assert c_call(lib.pod_select_pages, DEC, pod._DECODE_ARGS, batch=0, q=0) == 0
    assert c_call(lib.pod_paged_decode, DEC, pod._DECODE_ARGS, batch=0, q=0) == 0


def test_workspace_sizes():
    """Sizes that a call refuses give 0; others do not shrink with the batch."""
    assert pod.pod_select_pages_workspace_size(-1, 8, 10) == 0 and pod.pod_select_pages_workspace_size(4, 0, 10) == 0
    assert pod.pod_select_pages_workspace_size(4, 8, 100) >= 4 * 8 * 100 * 12
    assert pod.pod_paged_decode_workspace_size(4, 7, 2, 128) == 0 and pod.pod_paged_decode_workspace_size(4, 8, 2, 96) == 0
    a, b = (pod.pod_paged_decode_workspace_size(n, 8, 2, 128) for n in (1, 1000))
    assert 0 < a <= b and a % 256 == 0 and b % 256 == 0


def test_struct_sizes_are_those_of_the_header(tmp_path):
    import os
    import subprocess
    src = tmp_path / "s.c"
    src.write_text('#include "pod.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu", sizeof(pod_step_args), '
                   'sizeof(pod_decode_args)); return 0; }\n')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    sizes = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout
    assert sizes == f"{pod._STEP_ARGS.size} {pod._DECODE_ARGS.size}"
    assert ctypes.sizeof(ctypes.c_void_p) == 8
