"""Norm, rotation, cache write and cache read: against 64-bit definitions on
the GPU, and their refusals through the C ABI on the CPU.

Tolerances, fixed before the first run. A 16-bit result is the fp32 one rounded
once: eps/2 of the value. The fp32 part: d squares summed in fp32 (relative
d/2 * 2^-24 on the norm's factor, so at most 2^-18 for d = 256), two products,
rsqrtf (2 ulp), and cos / sin from an angle that is off by at most 2^-25 half
turns (float) + pos * 2^-53 turns, under 2^-21 radians at |pos| < 2^31. Together
below 2^-17 of the row's largest value.
"""
import math
import struct

import numpy as np
import pytest
import torch

import prefill_decode_paged_pod_gb300 as pod

ATOL = 2.0 ** -17          # of the row's largest value


@pytest.fixture(scope="module", autouse=True)
def built():
    from prefill_decode_paged_pod_gb300 import _build
    _build.build()
    pod.load_library()


# ------------------------------------------------------------------ 64-bit definitions
def norm_rope_64(x, w, pos, R, inter, scale=1.0, theta=1e4, eps=1e-6):
    y = x.double().numpy().copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w.double().numpy()
    out = y.copy()
    for j in range(R // 2):
        a, b = (2 * j, 2 * j + 1) if inter else (j, j + R // 2)
        ang = np.asarray(pos, dtype=np.float64) / scale * theta ** (-2.0 * j / R)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def check16(got, want, dtype):
    got = got.double().cpu().numpy()
    tol = np.abs(want) * (torch.finfo(dtype).eps / 2) * (1 + 2.0 ** -7) \
        + ATOL * np.abs(want).max(-1, keepdims=True) + torch.finfo(dtype).tiny
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.abs(got - want)[bad].max(), np.argwhere(bad)[0])


def codes_of(x32):
    """E4M3 codes of fp32 values: saturating, NaN kept (through torch's own cast)."""
    c = x32.clamp(-448, 448)
    c = torch.where(torch.isnan(x32), x32, c)
    return c.to(torch.float8_e4m3fn).view(torch.uint8)


def block_byte(x32):
    amax = torch.nan_to_num(x32.abs(), nan=0.0, posinf=math.inf).amax(-1)
    out = torch.zeros(amax.shape, dtype=torch.uint8)
    for i, a in enumerate(amax.flatten().tolist()):
        e = -127
        if a == math.inf:
            e = 120
        elif a > 0:
            m, x = math.frexp(a)               # a = m 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9
            e = max(-127, x - 9 + (1 if m > 0.875 else 0))
        out.view(-1)[i] = e + 127
    return out


def write_64(cache, scales, slots, k, v, layout, fmt, ks, vs):
    """The cache after a write of fp32 rows, on the CPU: bytes for FP8."""
    for half, x, s in ((0, k, ks), (1, v, vs)):
        for r, slot in enumerate(slots.tolist()):
            ps = cache.shape[2] if layout == "NHD" else cache.shape[3]
            if slot < 0 or slot >= cache.shape[0] * ps:
                continue
            p, i = slot // ps, slot % ps
            at = (p, half, i) if layout == "NHD" else (p, half, slice(None), i)
            if fmt == "16bit":
                cache[at] = x[r].to(cache.dtype)
            elif fmt == "scaled":
                cache[at] = codes_of(x[r].float() / torch.full_like(x[r].float(), s))
            else:
                b = block_byte(x[r].float())
                f = torch.tensor([2.0 ** (127 - int(t)) for t in b.flatten()]).view(-1, 1)
                cache[at] = codes_of(x[r].float() * f)
                scales[at] = b


def empty_cache(pages, ps, hk, d, layout, fmt, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    inner = (ps, hk) if layout == "NHD" else (hk, ps)
    shape = (pages, 2) + inner
    if fmt == "16bit":
        return torch.randn(shape + (d,), generator=g).to(dtype), None
    c = torch.randint(0, 120, shape + (d,), generator=g, dtype=torch.uint8)
    return c, torch.randint(100, 140, shape, generator=g, dtype=torch.uint8) if fmt == "block" else None


def as_cache(c, fmt):
    c = c.cuda()
    return c if fmt == "16bit" else c.view(torch.float8_e4m3fn)


def rows_of(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


# ------------------------------------------------------------------ norm and rotation
NORM_CASES = [
    # rows, H, Hk, d, rotary, interleaved, dtype, norm, rope_scale, theta, positions
    (1, 32, 8, 128, 128, False, torch.bfloat16, True, 1.0, 1e4, "low"),
    (7, 5, 1, 64, 64, False, torch.float16, True, 1.0, 1e4, "low"),
    (33, 6, 2, 256, 256, False, torch.bfloat16, True, 4.0, 5e5, "far"),
    (300, 28, 4, 128, 64, False, torch.float16, True, 1.0, 1e4, "far"),
    (65, 3, 3, 128, 48, False, torch.bfloat16, True, 1.0, 1e4, "negative"),
    (19, 7, 1, 128, 128, True, torch.float16, True, 1.0, 1e6, "far"),
    (40, 9, 3, 64, 16, True, torch.bfloat16, False, 1.0, 1e4, "edge"),
    (11, 4, 4, 256, 0, False, torch.float16, True, 1.0, 1e4, None),
    (130, 64, 8, 128, 128, False, torch.bfloat16, False, 0.5, 1e4, "edge"),
    (3, 300, 20, 64, 32, False, torch.float16, True, 1.0, 0.5, "low"),
]


def positions_of(kind, rows, seed):
    r = np.random.RandomState(seed)
    if kind == "low":
        p = np.arange(rows)
    elif kind == "far":
        p = r.randint(0, 1 << 20, rows)
    elif kind == "negative":
        p = r.randint(-5000, 5000, rows)
    else:
        p = r.randint(-(2 ** 31), 2 ** 31, rows, dtype=np.int64)
        p[:2] = [2 ** 31 - 1, -(2 ** 31)]
    return p.astype(np.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("case", NORM_CASES, ids=[f"{c[0]}x{c[1]}+{c[2]}x{c[3]}r{c[4]}" for c in NORM_CASES])
def test_norm_rope(case):
    rows, H, Hk, d, R, inter, dt, norm, scale, theta, kind = case
    qkv = rows_of((rows, H + 2 * Hk, d), dt, rows + d) * 3
    wq, wk = (1 + 0.3 * rows_of((2, d), dt, 5)).unbind(0) if norm else (None, None)
    pos = positions_of(kind, rows, 1) if kind else None
    x = qkv.cuda()
    dev = [None if t is None else t.contiguous().cuda() for t in (wq, wk)]
    p = None if pos is None else torch.from_numpy(pos).cuda()
    q, k = x[:, :H], x[:, H:H + Hk]
    qo, ko = pod.pod_qk_norm_rope(q, k, p, q_weight=dev[0], k_weight=dev[1], eps=1e-5, rotary_dim=R,
                                  interleaved=inter, rope_scale=scale, rope_theta=theta)
    check16(qo, norm_rope_64(qkv[:, :H], wq, pos, R, inter, scale, theta, 1e-5), dt)
    check16(ko, norm_rope_64(qkv[:, H:H + Hk], wk, pos, R, inter, scale, theta, 1e-5), dt)
    assert torch.equal(x.cpu(), qkv), "inputs are only read"
    # one tensor alone, and in place inside the fused buffer: the same bits, v untouched
    q1, none = pod.pod_qk_norm_rope(q, None, p, q_weight=dev[0], eps=1e-5, rotary_dim=R, interleaved=inter,
                                    rope_scale=scale, rope_theta=theta)
    assert none is None and torch.equal(q1, qo)
    _, k1 = pod.pod_qk_norm_rope(None, k, p, k_weight=dev[1], eps=1e-5, rotary_dim=R, interleaved=inter,
                                 rope_scale=scale, rope_theta=theta)
    assert torch.equal(k1, ko)
    pod.pod_qk_norm_rope(q, k, p, q_weight=dev[0], k_weight=dev[1], eps=1e-5, rotary_dim=R,
                         interleaved=inter, rope_scale=scale, rope_theta=theta, q_out=q, k_out=k)
    assert torch.equal(x[:, :H], qo) and torch.equal(x[:, H:H + Hk], ko)
    assert torch.equal(x[:, H + Hk:].cpu(), qkv[:, H + Hk:])


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_cos_and_sin_are_fp32_ones(interleaved):
    """Pairs (1, 0) turn into (cos, sin): the nearest fp16 value, unless the true one
    is that near to a tie. The angle left of the nearest quarter turn is at most 1/4
    half turn, so its rounding is off by 2^-27 of a half turn, 2^-25.3 radians; cos
    and sin of it by an ulp below 1, 2^-24: together 2^-23.4."""
    d, rows = 64, 3000
    r = np.random.RandomState(3)
    pos = r.randint(-131072, 131073, rows).astype(np.int32)
    pos[:2] = [0, 1]
    k = torch.zeros((rows, 1, d), dtype=torch.float16)
    first = np.arange(0, d, 2) if interleaved else np.arange(d // 2)
    second = first + (1 if interleaved else d // 2)
    k[:, :, torch.from_numpy(first)] = 1
    out = pod.pod_qk_norm_rope(None, k.cuda(), torch.from_numpy(pos).cuda(), interleaved=interleaved)[1]
    out = out[:, 0].double().cpu().numpy()
    angle = pos.astype(np.float64)[:, None] * 1e4 ** (-2.0 * np.arange(d // 2) / d)
    for got, want in ((out[:, first], np.cos(angle)), (out[:, second], np.sin(angle))):
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -14))) - 10)
        assert (np.abs(got - want) <= step / 2 + 2.0 ** -23.4).all(), np.abs(got - want).max()


@pytest.mark.gpu
def test_norm_special_values():
    """Zeros stay zeros, a NaN stays in its head, no rows launch nothing."""
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    x[1, 0, 3] = math.nan
    x[2] = 1e30
    w = torch.ones(64, dtype=torch.bfloat16).cuda()
    pos = torch.arange(4, dtype=torch.int32).cuda()
    q, k = pod.pod_qk_norm_rope(x.cuda(), x.cuda(), pos, q_weight=w)
    q, k = q.cpu(), k.cpu()
    assert (q[0] == 0).all() and (q[3] == 0).all()
    assert q[1, 0].isnan().all() and (q[1, 1] == 0).all()
    assert k[1, 0].isnan().sum() in (1, 2) and torch.isfinite(k[2]).all()
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16).cuda()
    q, k = pod.pod_qk_norm_rope(e, e, torch.empty(0, dtype=torch.int32).cuda(), q_weight=w)
    assert q.shape == e.shape and k.shape == e.shape


# ------------------------------------------------------------------ write and read
WRITE_CASES = [
    # rows, Hk, d, ps, layout, fmt, dtype
    (1, 1, 64, 16, "NHD", "16bit", torch.float16),
    (37, 8, 128, 16, "NHD", "scaled", torch.bfloat16),
    (37, 8, 128, 16, "HND", "scaled", torch.float16),
    (50, 3, 128, 3, "NHD", "block", torch.bfloat16),
    (50, 5, 64, 1, "HND", "block", torch.float16),
    (129, 2, 256, 64, "NHD", "block", torch.float16),
    (129, 2, 256, 5, "HND", "scaled", torch.bfloat16),
    (700, 8, 128, 16, "HND", "16bit", torch.bfloat16),
    (700, 40, 64, 16, "NHD", "block", torch.bfloat16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", WRITE_CASES, ids=["-".join(map(str, c[:6])) for c in WRITE_CASES])
def test_write_and_read(case):
    rows, hk, d, ps, layout, fmt, dt = case
    pages = rows // ps + 5
    cache, scales = empty_cache(pages, ps, hk, d, layout, fmt, dt, 3)
    kv = rows_of((rows, 3 * hk, d), dt, rows)
    # magnitudes over many binades; a zero head row, negative zeros, NaN and infinities
    g = torch.Generator().manual_seed(rows + d)
    kv = (kv.float() * torch.exp2(torch.randint(-12, 6, (rows, 3 * hk, 1), generator=g).float())).to(dt)
    kv[0, 0] = 0
    kv[0, hk, 1::2] = -0.0                     # (its sign is kept)
    if fmt != "16bit" and rows > 3:
        kv[1, 0, 5], kv[2, hk, 0], kv[3, 0, 1] = math.nan, math.inf, -math.inf
    k, v = kv[:, :hk], kv[:, hk:2 * hk]
    r = np.random.RandomState(rows)
    slots = torch.from_numpy(r.permutation(pages * ps)[:rows].astype(np.int64))
    if rows > 10:
        slots[4], slots[9] = -1, -(2 ** 40)
    ks, vs = (0.037, 0.011) if fmt == "scaled" else (1.0, 1.0)
    want_c, want_s = cache.clone(), None if scales is None else scales.clone()
    write_64(want_c, want_s, slots, k.float(), v.float(), layout, fmt, ks, vs)
    dc, ds = as_cache(cache, fmt), None if scales is None else scales.cuda()
    x = kv.cuda()
    scale = dict(k_scale=ks, v_scale=vs, kv_scales=ds, kv_layout=layout)
    pod.pod_append_kv(x[:, :hk], x[:, hk:2 * hk], dc, slots.cuda(), **scale)
    got = dc.cpu() if fmt == "16bit" else dc.view(torch.uint8).cpu()
    if fmt == "16bit":
        assert torch.equal(got, want_c)
    else:                      # any NaN code stands for NaN
        nan = (want_c & 0x7F) == 0x7F
        assert torch.equal((got & 0x7F) == 0x7F, nan)
        assert torch.equal(got[~nan], want_c[~nan])
    if ds is not None:
        assert torch.equal(ds.cpu(), want_s)

    # read back: every row of the write, and padding rows as zeros
    out = pod.pod_gather_kv(dc, slots.cuda(), dtype=dt, **scale).cpu()
    for i in range(rows):
        s = int(slots[i])
        if s < 0:
            assert (out[i] == 0).all()
            continue
        p, o = s // ps, s % ps
        for half in (0, 1):
            at = (p, half, o) if layout == "NHD" else (p, half, slice(None), o)
            if fmt == "16bit":
                want = want_c[at]
            else:
                f = want_c[at].view(torch.float8_e4m3fn).double()
                sc = (vs if half else ks) if fmt == "scaled" else torch.exp2(want_s[at].double() - 127)[:, None]
                sc = float(np.float32(sc)) if fmt == "scaled" else sc
                big = torch.finfo(dt).max
                want = (f * sc).float().clamp(-big, big).to(dt)   # (fp32 product, then one rounding)
            assert torch.equal(out[i, half].nan_to_num(123.0), want.nan_to_num(123.0)), (i, half)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["16bit", "scaled", "block"])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_fused_write(fmt, layout):
    """Norm, rotation and write in one pass: q as pod_qk_norm_rope gives it, K
    within half an E4M3 step (2^-4, and the subnormal step below 2^-6) of the
    64-bit value, V as pod_append_kv writes it."""
    rows, H, hk, d, ps, R, dt = 83, 12, 4, 128, 16, 96, torch.bfloat16
    qkv = rows_of((rows, H + 2 * hk, d), dt, 9)
    wq, wk = (1 + 0.3 * rows_of((2, d), dt, 5)).unbind(0)
    pos = positions_of("far", rows, 2)
    pages = 8
    cache, scales = empty_cache(pages, ps, hk, d, layout, fmt, dt, 3)
    slots = torch.from_numpy(np.random.RandomState(1).permutation(pages * ps)[:rows].astype(np.int64))
    slots[7] = -1
    ks, vs = (0.037, 0.011) if fmt == "scaled" else (1.0, 1.0)
    want_c, want_s = cache.clone(), None if scales is None else scales.clone()
    write_64(want_c, want_s, slots, qkv[:, H:H + hk].float(), qkv[:, H + hk:].float(), layout, fmt, ks, vs)
    dc, ds = as_cache(cache, fmt), None if scales is None else scales.cuda()
    x, p = qkv.cuda(), torch.from_numpy(pos).cuda()
    kw = dict(q_weight=wq.cuda(), k_weight=wk.cuda(), rotary_dim=R)
    scale = dict(k_scale=ks, v_scale=vs, kv_scales=ds, kv_layout=layout)
    q = pod.pod_norm_rope_append(x[:, :H], x[:, H:H + hk], x[:, H + hk:], p, dc, slots.cuda(), **kw, **scale)
    assert torch.equal(q, pod.pod_qk_norm_rope(x[:, :H], x[:, H:H + hk], p, **kw)[0])
    k64 = norm_rope_64(qkv[:, H:H + hk], wk, pos, R, False)
    got = (dc if fmt == "16bit" else dc.view(torch.uint8)).cpu()
    used = torch.zeros(pages * ps, dtype=torch.bool)
    for i, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        used[s] = True
        at_k = (s // ps, 0, s % ps) if layout == "NHD" else (s // ps, 0, slice(None), s % ps)
        at_v = (s // ps, 1, s % ps) if layout == "NHD" else (s // ps, 1, slice(None), s % ps)
        assert torch.equal(got[at_v], want_c[at_v])
        if ds is not None:
            assert torch.equal(ds.cpu()[at_v], want_s[at_v])
        if fmt == "16bit":
            check16(got[at_k], k64[i], dt)
            continue
        f = got[at_k].view(torch.float8_e4m3fn).double().numpy()
        if fmt == "scaled":
            sc = float(np.float32(ks))
            y = np.clip(k64[i] / sc, -448, 448)
        else:
            b = ds.cpu()[at_k].double().numpy()[:, None]
            sc = 2.0 ** (b - 127)
            y = k64[i] / sc
            amax = np.abs(k64[i]).max(-1, keepdims=True)
            assert (amax <= 448 * sc * (1 + ATOL)).all() and (amax > 224 * sc * (1 - ATOL)).all()
        tol = np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10) + ATOL * np.abs(y).max(-1, keepdims=True) * 2
        assert (np.abs(f - y) <= tol).all()
    # slots that no row names keep their bytes
    flat = got if layout == "NHD" else got.transpose(2, 3)
    before = cache if layout == "NHD" else cache.transpose(2, 3)
    keep = ~used.view(pages, ps)
    for half in (0, 1):
        assert torch.equal(flat[:, half][keep], before[:, half][keep])
    # without q: the same cache
    d2, s2 = as_cache(cache, fmt), None if scales is None else scales.cuda()
    assert pod.pod_norm_rope_append(None, x[:, H:H + hk], x[:, H + hk:], p, d2, slots.cuda(),
                                    k_weight=kw["k_weight"], rotary_dim=R, k_scale=ks, v_scale=vs,
                                    kv_scales=s2, kv_layout=layout) is None
    assert torch.equal(d2.view(torch.uint8), dc.view(torch.uint8))


@pytest.mark.gpu
def test_slots_outside_the_pool():
    """Reported in the status word, nothing written, zeros read."""
    k = torch.ones((3, 2, 64), dtype=torch.float16).cuda()
    kv = torch.zeros((2, 2, 4, 2, 64), dtype=torch.float16).cuda()
    st = torch.zeros(1, dtype=torch.int32).cuda()
    pod.pod_append_kv(k, k, kv, torch.tensor([0, -1, 7]).cuda(), status=st)
    assert st.item() == 0 and kv.sum().item() == 2 * 2 * 2 * 64
    pod.pod_append_kv(2 * k, k, kv, torch.tensor([8, 2 ** 62, -1]).cuda(), status=st)
    assert st.item() == 4 and kv.sum().item() == 2 * 2 * 2 * 64
    st.zero_()
    out = pod.pod_gather_kv(kv, torch.tensor([0, 8, -3]).cuda(), dtype=torch.float16, status=st)
    assert st.item() == 4 and (out[0] == 1).all() and (out[1:] == 0).all()


@pytest.mark.gpu
def test_large_offsets():
    """Slots whose byte offset passes 32 bits."""
    pages, ps, hk, d = 70000, 16, 8, 128
    kv = torch.zeros((pages, 2, ps, hk, d), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.zeros((pages, 2, ps, hk), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([pages * ps - 1, 0, 66000 * ps + 5]).cuda()
    k, v = rows_of((3, hk, d), torch.bfloat16, 1).cuda(), rows_of((3, hk, d), torch.bfloat16, 2).cuda()
    pod.pod_append_kv(k, v, kv, slots, kv_scales=sc)
    out = pod.pod_gather_kv(kv, slots, dtype=torch.bfloat16, kv_scales=sc)
    assert (out[:, 0] - k).abs().max() <= 2.0 ** -4 * k.abs().max()
    assert (out[:, 1] - v).abs().max() <= 2.0 ** -4 * v.abs().max()
    assert int((sc != 0).sum()) == 3 * 2 * hk


@pytest.mark.gpu
def test_graph_and_stream():
    """Captured on a side stream and replayed on new data: the eager result."""
    rows, H, hk, d, ps = 9, 8, 2, 128, 16
    x = rows_of((rows, H + 2 * hk, d), torch.bfloat16, 1).cuda()
    kv = torch.zeros((4, 2, ps, hk, d), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.zeros((4, 2, ps, hk), dtype=torch.uint8, device="cuda")
    pos = torch.arange(rows, dtype=torch.int32).cuda()
    slots = torch.arange(rows).cuda() + 5
    qo = torch.empty((rows, H, d), dtype=torch.bfloat16, device="cuda")
    back = torch.empty((rows, 2, hk, d), dtype=torch.bfloat16, device="cuda")

    def step():
        pod.pod_norm_rope_append(x[:, :H], x[:, H:H + hk], x[:, H + hk:], pos, kv, slots, kv_scales=sc, q_out=qo)
        pod.pod_gather_kv(kv, slots, dtype=torch.bfloat16, kv_scales=sc, out=back)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        step()
    x.copy_(rows_of((rows, H + 2 * hk, d), torch.bfloat16, 2))
    pos += 1000
    slots += 7
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (qo, back)]
    kv.view(torch.uint8).zero_()
    step()
    torch.cuda.synchronize()
    assert torch.equal(got[0], qo) and torch.equal(got[1], back)


@pytest.mark.gpu
@pytest.mark.parametrize("as_int", [False, True])
def test_a_stream_of_the_callers(as_int):
    """Given streams are launched on, and own the outputs made for them."""
    x = rows_of((50, 6, 64), torch.float16, 1).cuda()
    pos = torch.arange(50, dtype=torch.int32).cuda()
    want = pod.pod_qk_norm_rope(x[:, :4], x[:, 4:], pos)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side.cuda_stream if as_int else side
    hold = torch.zeros(1 << 24, device="cuda")
    for _ in range(3):
        got = pod.pod_qk_norm_rope(x[:, :4], x[:, 4:], pos, stream=s)
        junk = [torch.full((50, 4, 64), 9.0, dtype=torch.float16, device="cuda") for _ in range(4)]
        hold.add_(1)
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del junk, got
    with torch.cuda.stream(side):
        got = pod.pod_qk_norm_rope(x[:, :4], x[:, 4:], pos)
    side.synchronize()
    assert torch.equal(got[0], want[0])


@pytest.mark.gpu
def test_serving_step_over_a_written_cache():
    """Rows written with per-tensor scales are what the FP8 decode half reads,
    and the same cache read back runs in the 16-bit prefill half."""
    import oracle
    from podtest_util import LSE_ATOL, OUT_ATOL, OUT_RTOL
    H, hk, d, ps, dt = 16, 2, 128, 16, torch.bfloat16
    lens = [70, 33, 128]
    npg = [(n + ps - 1) // ps for n in lens]
    indptr = np.concatenate([[0], np.cumsum(npg)]).astype(np.int32)
    last = np.array([(n - 1) % ps + 1 for n in lens], dtype=np.int32)
    pages = int(indptr[-1]) + 2
    indices = np.random.RandomState(0).permutation(pages)[:indptr[-1]].astype(np.int32)
    req = np.concatenate([np.full(n, i) for i, n in enumerate(lens)])
    at = np.concatenate([np.arange(n) for n in lens])
    slots = torch.from_numpy(pod.pod_kv_slots(indptr, indices, ps, req, at)).cuda()
    total = sum(lens)
    k, v = rows_of((total, hk, d), dt, 1).cuda(), rows_of((total, hk, d), dt, 2).cuda()
    ks, vs = 0.02, 0.013
    kv = torch.zeros((pages, 2, ps, hk, d), dtype=torch.float8_e4m3fn, device="cuda")
    pod.pod_append_kv(k, v, kv, slots, k_scale=ks, v_scale=vs)
    # decode half over the FP8 cache
    q = rows_of((3, H, d), dt, 3).cuda()
    h = pod.pod_plan(None, None, None, None, np.arange(4, dtype=np.int32), indptr, indices, last, H, hk, d,
                     ps, True, -1, None, dtype=dt, p_num_pages=0, d_num_pages=pages)
    pod.pod_plan_set_decode_fp8(h, ks, vs)
    ws = torch.empty(pod.pod_workspace_size(h), dtype=torch.uint8, device="cuda")
    pod.pod_bind_workspace(h, ws)
    _, _, od, ld = pod.pod_run(h, None, None, q, kv, ws)
    # prefill half over the cache read back
    back = pod.pod_gather_kv(kv, slots, dtype=dt, k_scale=ks, v_scale=vs)
    qi = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    qp = rows_of((total, H, d), dt, 4).cuda()
    h2 = pod.pod_plan(qi, qi, np.arange(total, dtype=np.int32), np.ones(3, dtype=np.int32),
                      None, None, None, None, H, hk, d, 1, True, -1, None, dtype=dt,
                      p_num_pages=total, d_num_pages=0)
    ws2 = torch.empty(pod.pod_workspace_size(h2), dtype=torch.uint8, device="cuda")
    pod.pod_bind_workspace(h2, ws2)
    op, lp, _, _ = pod.pod_run(h2, qp, back.view(total, 2, 1, hk, d), None, None, ws2)
    torch.cuda.synchronize()
    codes = kv.cpu().double()
    for r, n in enumerate(lens):
        pg = indices[indptr[r]:indptr[r + 1]]
        kk = codes[pg, 0].reshape(-1, hk, d)[:n].numpy() * ks
        vv = codes[pg, 1].reshape(-1, hk, d)[:n].numpy() * vs
        bb = back[qi[r]:qi[r + 1]].cpu().double().numpy()
        for g in range(H):
            x = kk[:, g // 8] @ q[r, g].cpu().double().numpy() / math.sqrt(d)
            w = np.exp(x - x.max())
            ref = (w / w.sum()) @ vv[:, g // 8]
            err = np.abs(od[r, g].cpu().double().numpy() - ref)
            assert (err <= OUT_ATOL + OUT_RTOL * np.abs(ref)).all()
            assert abs(ld[r, g].item() - (x.max() + math.log(w.sum())) / math.log(2)) <= LSE_ATOL
            x = bb[:, 0, g // 8] @ qp[qi[r] + n - 1, g].cpu().double().numpy() / math.sqrt(d)
            w = np.exp(x - x.max())
            ref = (w / w.sum()) @ bb[:, 1, g // 8]
            err = np.abs(op[qi[r] + n - 1, g].cpu().double().numpy() - ref)
            assert (err <= OUT_ATOL + OUT_RTOL * np.abs(ref)).all()


# ------------------------------------------------------------------ refusals (host only)
P = 1 << 20          # a 16-byte aligned address that is never read: every call below is refused


def _err(code, want, text):
    assert code == want and text in pod.pod_last_error(), (code, pod.pod_last_error())


FIELDS = ("q", "k", "v", "qw", "kw", "pos", "slots", "qo", "ko", "kv", "sc", "st", "qs", "ks", "vs", "qos", "kos",
          "rows", "pages", "ps", "H", "Hk", "d", "lay", "fmt", "dt", "R", "il", "eps", "rs", "th", "k_scale", "v_scale")


def io_call(name, a, kw):
    """The C entry point with pod_io_args packed field by field (its documented order)."""
    a = {**dict.fromkeys(FIELDS, 0), "dt": 1, "rs": 1.0, "th": 1e4, "k_scale": 1.0, "v_scale": 1.0, **a, **kw}
    assert len(a) == len(FIELDS)
    kinds = "Q" * 12 + "q" * 7 + "i" * 9 + "f" * 5
    packed = struct.pack("@" + kinds, *[0 if a[f] is None else a[f] for f in FIELDS])
    return getattr(pod.load_library(), name)(packed, None)


def norm_call(**kw):
    return io_call("pod_qk_norm_rope", dict(q=P, k=P, qs=1024, ks=256, rows=4, H=8, Hk=2, d=128, qw=P, kw=P, eps=1e-6,
                                            pos=P, R=128, qo=P, ko=P, qos=1024, kos=256), kw)


@pytest.mark.parametrize("kw,code,text", [
    (dict(q=None), 1, "q is NULL"), (dict(k=P + 8), 1, "k must be 16-byte"), (dict(ko=None), 1, "k_out is NULL"),
    (dict(qs=1020), 1, "multiple of 8"), (dict(ks=128), 1, "row stride"), (dict(qos=-1024), 1, "row stride"),
    (dict(d=96), 2, "head_dim"), (dict(dt=2), 2, "dtype"), (dict(H=0, Hk=0), 1, "no heads"),
    (dict(H=-1), 1, "no heads"), (dict(R=130), 1, "rotary_dim"), (dict(R=24), 1, "rotary_dim"),
    (dict(R=-16), 1, "rotary_dim"), (dict(pos=None), 1, "positions"), (dict(eps=-1.0), 1, "eps"),
    (dict(eps=math.nan), 1, "eps"), (dict(rs=0.0), 1, "rope_scale"), (dict(th=math.inf), 1, "rope_theta"),
    (dict(rows=-1), 1, "rows"), (dict(rows=2 ** 31), 1, "rows"), (dict(qw=P + 2), 1, "weights"),
])
def test_norm_refusals(kw, code, text):
    _err(norm_call(**kw), code, text)


def test_no_rows_need_no_tensors():
    assert norm_call(rows=0, q=None, k=None, qo=None, ko=None, pos=None) == 0


CACHE = dict(kv=P, pages=10, ps=16, Hk=2, d=128, slots=P, rows=4)


def append_call(**kw):
    return io_call("pod_append_kv", dict(CACHE, k=P, v=P, ks=256, vs=256), kw)


def fused_call(**kw):
    return io_call("pod_norm_rope_append", dict(CACHE, k=P, v=P, ks=256, vs=256, q=P, qo=P, qs=1024, qos=1024, H=8,
                                                pos=P, R=128, eps=1e-6), kw)


def gather_call(**kw):
    return io_call("pod_gather_kv", dict(CACHE, ko=P), kw)


CACHE_REFUSALS = [
    (dict(kv=None), 1, "cache"), (dict(kv=P + 8), 1, "cache"), (dict(fmt=3), 1, "format"),
    (dict(fmt=2), 1, "needs its scales"), (dict(fmt=1, sc=P), 1, "scales given"), (dict(sc=P), 1, "scales given"),
    (dict(fmt=1, k_scale=0.0), 1, "k_scale"), (dict(fmt=1, v_scale=math.nan), 1, "v_scale"),
    (dict(lay=2), 1, "kv_layout"), (dict(Hk=0), 1, "num_kv_heads"), (dict(pages=0), 1, "empty"),
    (dict(ps=0), 1, "empty"), (dict(pages=2 ** 60), 1, "too large"), (dict(slots=None), 1, "slots"),
    (dict(d=32), 2, "head_dim"), (dict(dt=7), 2, "dtype"),
]


@pytest.mark.parametrize("kw,code,text", CACHE_REFUSALS)
def test_cache_refusals(kw, code, text):
    _err(append_call(**kw), code, text)
    _err(fused_call(**kw), code, text)
    _err(gather_call(**kw), code, text)


@pytest.mark.parametrize("kw,text", [
    (dict(k=None), "k is NULL"), (dict(v=P + 4), "v must be"), (dict(ks=128), "row stride")])
def test_append_refusals(kw, text):
    _err(append_call(**kw), 1, text)
    _err(fused_call(**kw), 1, text)


@pytest.mark.parametrize("kw,text", [
    (dict(q=None), "q is NULL"), (dict(qo=P + 8), "q_out must"), (dict(R=40), "rotary_dim"), (dict(pos=None), "positions"),
    (dict(kw=P + 2), "weights"), (dict(H=-1), "heads"), (dict(eps=math.inf), "eps")])
def test_fused_refusals(kw, text):
    _err(fused_call(**kw), 1, text)


def test_no_arguments():
    for name in ("pod_qk_norm_rope", "pod_append_kv", "pod_norm_rope_append", "pod_gather_kv"):
        _err(getattr(pod.load_library(), name)(None, None), 1, "args is NULL")


def test_gather_refuses_a_missing_output():
    _err(gather_call(ko=None), 1, "k_out is NULL")
    assert gather_call(rows=0, ko=None, slots=None) == 0 and append_call(rows=0, k=None, v=None, slots=None) == 0


def test_binding_refuses_host_tensors():
    k = torch.zeros((2, 2, 64), dtype=torch.float16)
    with pytest.raises(pod.PodError, match="CUDA"):
        pod.pod_qk_norm_rope(k, k, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(pod.PodError, match="CUDA"):
        pod.pod_append_kv(k, k, torch.zeros((1, 2, 4, 2, 64), dtype=torch.float16), torch.zeros(2).long())


@pytest.mark.gpu
def test_binding_refusals():
    k = torch.zeros((2, 2, 64), dtype=torch.float16).cuda()
    kv = torch.zeros((1, 2, 4, 2, 64), dtype=torch.float16).cuda()
    s = torch.zeros(2).long().cuda()
    pos = torch.zeros(2, dtype=torch.int32).cuda()
    bad = [
        lambda: pod.pod_qk_norm_rope(k, k, None),
        lambda: pod.pod_qk_norm_rope(k, k, pos.long()),
        lambda: pod.pod_qk_norm_rope(k, k[:1], pos),
        lambda: pod.pod_qk_norm_rope(k, k.bfloat16(), pos),
        lambda: pod.pod_qk_norm_rope(k[..., ::2], k, pos),
        lambda: pod.pod_qk_norm_rope(k, k, pos, q_weight=torch.ones(63).half().cuda()),
        lambda: pod.pod_append_kv(k, k, kv, s[:1]),
        lambda: pod.pod_append_kv(k, k, kv, s.int()),
        lambda: pod.pod_append_kv(k, k, kv.bfloat16(), s),
        lambda: pod.pod_append_kv(k, k, kv, s, kv_layout="HND"),
        lambda: pod.pod_append_kv(k, k, kv, s, kv_scales=torch.zeros((1, 2, 4, 2)).byte().cuda()),
        lambda: pod.pod_append_kv(k.float(), k.float(), kv, s),
        lambda: pod.pod_append_kv(k, k[:, :1], kv, s),
        lambda: pod.pod_gather_kv(kv, s, dtype=torch.float16, out=torch.zeros((2, 2, 2, 32)).half().cuda()),
        lambda: pod.pod_gather_kv(kv[:, :1], s, dtype=torch.float16),
    ]
    for f in bad:
        with pytest.raises(pod.PodError):
            f()


def test_slots_of_a_page_table():
    indptr, indices = np.array([0, 2, 5], np.int32), np.array([7, 3, 9, 0, 4], np.int32)
    s = pod.pod_kv_slots(indptr, indices, 4, np.array([0, 0, 1, 1]), np.array([3, 4, 0, 9]))
    assert s.tolist() == [31, 12, 36, 17] and s.dtype == np.int64
    t = pod.pod_kv_slots(torch.from_numpy(indptr), torch.from_numpy(indices), 4,
                         torch.tensor([0, 0, 1, 1]), torch.tensor([3, 4, 0, 9]))
    assert t.tolist() == [31, 12, 36, 17] and t.dtype == torch.int64
