"""The operators around the cache at the edges of what their calls allow: slots
of positions that no page holds, rows of any magnitude, angles of far positions,
caches past 4 GB, and kernels that start beside the one before.
"""
import os
import subprocess
from decimal import Decimal, localcontext
from fractions import Fraction

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


# ------------------------------------------------------------------ norm of any magnitude
BF = torch.bfloat16


def magnitudes(rows, heads, d, seed):
    """bf16 rows from the smallest numbers to the largest, and ordinary ones between."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, heads, d), generator=g, dtype=torch.float64).clamp(-4, 4)
    e = torch.tensor([-130, -126, -110, -80, -65, -63, -33, -31, 0, 3, 31, 40, 63, 66, 100, 125])
    at = torch.randint(0, len(e), (rows, heads, 1), generator=g)
    at.view(-1)[:len(e)] = torch.arange(len(e))
    return (x * torch.exp2(e[at].double())).to(BF)


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30, 1e-41, 1e3])
@pytest.mark.parametrize("w_exp", [0, 90, -90, 124])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_norm_of_rows_of_any_magnitude(eps, w_exp, d):
    """Squares, and products with the weights, that leave fp32's range on the way
    to values that do not. fp32's own subnormal results carry their step."""
    from test_cache_io import ATOL, norm_rope_64
    rows, H, Hk, R = 37, 3, 2, 32
    x = magnitudes(rows, H + Hk, d, d)
    g = torch.Generator().manual_seed(1)
    w = (torch.exp2(torch.full((d,), w_exp).double()) * (1 + 0.3 * torch.randn(d, generator=g).double())).to(BF)
    w[3] = 0
    pos = np.arange(rows, dtype=np.int32)
    q, k = pod.pod_qk_norm_rope(x[:, :H].cuda(), x[:, H:].cuda(), torch.from_numpy(pos).cuda(), q_weight=w.cuda(),
                                k_weight=w.cuda(), eps=eps, rotary_dim=R)
    eps32 = float(np.float32(eps))
    for got, part in ((q, x[:, :H]), (k, x[:, H:])):
        want = norm_rope_64(part, w, pos, R, False, eps=eps32)
        got = got.double().cpu().numpy()
        over = np.abs(want) > torch.finfo(BF).max * (1 - 2.0 ** -9)
        tol = np.abs(want) * 2.0 ** -8 * (1 + 2.0 ** -7) + ATOL * np.abs(want).max(-1, keepdims=True) + 2.0 ** -126
        bad = ~over & ~(np.abs(got - want) <= tol)
        assert not bad.any(), (np.argwhere(bad)[0], got[bad][0], want[bad][0])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["16bit", "block"])
def test_fused_write_of_rows_of_any_magnitude(fmt):
    """The same through the write: K rows of 2^-80 to 2^100 come out near the weights,
    and rows without a value, infinities and NaN stay what they were."""
    from test_cache_io import norm_rope_64
    rows, hk, d = 40, 2, 128
    x = magnitudes(rows, hk, d, 7)
    x[20], x[21, 0, 5], x[22, 1, 9] = 0, torch.inf, torch.nan
    w = torch.ones(d, dtype=BF)
    kv = torch.zeros((rows, 2, 1, hk, d), dtype=BF if fmt == "16bit" else torch.float8_e4m3fn, device="cuda")
    sc = None if fmt == "16bit" else torch.zeros((rows, 2, 1, hk), dtype=torch.uint8, device="cuda")
    slots = torch.arange(rows).cuda()
    pod.pod_norm_rope_append(None, x.cuda(), x.cuda(), None, kv, slots, k_weight=w.cuda(), eps=1e-30, rotary_dim=0,
                             kv_scales=sc)
    got = pod.pod_gather_kv(kv, slots, dtype=BF, kv_scales=sc)[:, 0].double().cpu().numpy()
    want = norm_rope_64(x, w, None, 0, False, eps=1e-30)
    plain = np.ones(rows, dtype=bool)
    plain[20:23] = False
    step = 2.0 ** -8 if fmt == "16bit" else 2.0 ** -4 + 2.0 ** -8
    tol = np.abs(want) * step * (1 + 2.0 ** -7) + (2.0 ** -16 if fmt == "16bit" else 2.0 ** -9) * np.abs(want).max(-1, keepdims=True)
    assert (np.abs(got - want)[plain] <= tol[plain]).all()
    assert (got[20] == 0).all()
    assert (np.delete(got[21, 0], 5) == 0).all() and np.isnan(got[21, 0, 5])
    assert np.isnan(got[22, 1]).all() and np.isfinite(got[22, 0]).all()


# ------------------------------------------------------------------ frequencies of the rotation
def exact_turns(R, scale, theta, j):
    """theta^(-2j/R) / (2 pi scale) as a Decimal of 60 digits."""
    def arctan_inv(n):
        x = s = Decimal(1) / n
        k = 1
        while abs(x) > Decimal(10) ** -70:
            x, k = -x / (n * n), k + 2
            s += x / k
        return s
    with localcontext() as c:
        c.prec = 75
        pi = 4 * (4 * arctan_inv(5) - arctan_inv(239))
        th, sc = Decimal(float(np.float32(theta))), Decimal(float(np.float32(scale)))
        return (th.ln() * Decimal(-2 * j) / R).exp() / (2 * pi * sc)


@pytest.fixture(scope="module")
def turns_client(tmp_path_factory):
    from prefill_decode_paged_pod_gb300 import _build
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path_factory.mktemp("turns") / "turns_client")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", _build.CSRC, os.path.join(here, "csrc", "turns_client.cpp"),
                    "-o", exe], check=True)

    def call(mode, *settings):
        args = [repr(x) if isinstance(x, float) else str(x) for s in settings for x in s]
        return [int(x) for x in subprocess.run([exe, mode] + args, check=True, capture_output=True,
                                               text=True).stdout.split()]
    return call


@pytest.mark.parametrize("R,scale,theta", [(128, 1.0, 1e4), (64, 1.0, 5e5), (256, 32.0, 1e6), (48, 1.0, 1e4),
                                           (96, 0.5, 1.5), (16, 4.0, 0.5), (128, 1e-3, 1e4), (256, 1.0, 1e30),
                                           (80, 1.0, 1.0), (112, 3.0, 7.7), (32, 1.0, 1e-6)])
def test_frequencies_to_a_unit_of_64_bits(turns_client, R, scale, theta):
    got = turns_client("F", (R, scale, theta))
    assert len(got) == R // 2
    for j, f in enumerate(got):
        t = exact_turns(R, scale, theta, j)
        with localcontext() as c:
            c.prec = 75
            assert t < 2 ** 30
            off = (f - t * 2 ** 64) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, (j, off)


def test_kept_tables(turns_client):
    """A layer's calls, a write among them (R = 0), and a model's few settings make
    each table once; the fifth setting takes the place of the first."""
    a, b, c, d, e = (128, 1.0, 1e4), (128, 1.0, 1e6), (64, 1.0, 1e4), (128, 2.0, 1e4), (32, 1.0, 1e4)
    write = (0, 1.0, 1.0)
    assert turns_client("N", *[a, write] * 5) == [1]
    assert turns_client("N", *[a, b, write, c, d] * 3) == [4]
    assert turns_client("N", a, b, c, d, e, b, c, d, e, a) == [6]
    assert turns_client("N", write, write) == [0]
    assert turns_client("F", a, b, write)[64:] == turns_client("F", b)


@pytest.mark.gpu
@pytest.mark.parametrize("scale,theta", [(1.0, 1e4), (1.0, 1e6), (0.25, 500.0)])
def test_cos_and_sin_of_far_positions(scale, theta):
    """As near to the true ones at +-2^31 as at 0: pairs (1, 0) turn into (cos, sin),
    rounded to fp16 once, within 2^-23.4 before that (a turn's fraction to 2^-34, fp32
    afterwards)."""
    d, rows = 64, 2000
    r = np.random.RandomState(4)
    pos = np.concatenate([2 ** 31 - 1 - np.arange(rows), -(2 ** 31) + np.arange(rows),
                          r.randint(-(2 ** 31), 2 ** 31, rows)]).astype(np.int32)
    k = torch.zeros((len(pos), 1, d), dtype=torch.float16)
    k[:, :, :d // 2] = 1
    out = pod.pod_qk_norm_rope(None, k.cuda(), torch.from_numpy(pos).cuda(), rope_scale=scale, rope_theta=theta)[1]
    out = out[:, 0].double().cpu().numpy()
    for j in range(d // 2):
        with localcontext() as c:
            c.prec = 75
            f = int(exact_turns(d, scale, theta, j) * 2 ** 120)
        turn = np.array([float(Fraction(int(p) * f % 2 ** 120, 2 ** 120)) for p in pos])
        turn = 2 * np.pi * (turn - np.round(turn))
        for got, want in ((out[:, j], np.cos(turn)), (out[:, j + d // 2], np.sin(turn))):
            step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -14))) - 10)
            off = np.abs(got - want) - step / 2
            assert (off <= 2.0 ** -23.4).all(), (j, off.max())


# ------------------------------------------------------------------ caches past 4 GB
@pytest.mark.gpu
@pytest.mark.parametrize("fmt,layout", [("block", "NHD"), ("block", "HND"), ("16bit", "NHD"), ("scaled", "HND")])
def test_byte_offsets_past_32_bits(fmt, layout):
    """Rows behind the first 2^32 bytes, and at its end, lie where they should: a
    short pool's bytes, and nothing else in the long one."""
    from test_cache_io import rows_of
    ps, hk, d = 16, 8, 128
    page = 2 * ps * hk * d * (2 if fmt == "16bit" else 1)
    pages = 2 ** 32 // page + 4001
    inner = (ps, hk) if layout == "NHD" else (hk, ps)
    kind = BF if fmt == "16bit" else torch.float8_e4m3fn
    edge = 2 ** 32 // page                       # the page that begins at 2^32 bytes
    at = torch.tensor([pages - 1, 0, edge, edge - 1, edge + 1, edge + 3000])
    kw = dict(kv_layout=layout, **(dict(k_scale=0.02, v_scale=0.03) if fmt == "scaled" else {}))
    k, v = rows_of((len(at), hk, d), BF, 1).cuda(), rows_of((len(at), hk, d), BF, 2).cuda()
    pools = []
    for n, where in ((pages, at), (len(at), torch.arange(len(at)))):
        kv = torch.zeros((n, 2) + inner + (d,), dtype=kind, device="cuda")
        sc = torch.zeros((n, 2) + inner, dtype=torch.uint8, device="cuda") if fmt == "block" else None
        slots = (where * ps + torch.arange(len(at)) % ps).cuda()
        pod.pod_append_kv(k, v, kv, slots, kv_scales=sc, **kw)
        pools.append((kv.view(torch.uint8), sc, pod.pod_gather_kv(kv, slots, dtype=BF, kv_scales=sc, **kw)))
    (long, long_s, long_r), (short, short_s, short_r) = pools
    assert torch.equal(long_r, short_r) and torch.equal(long[at.cuda()], short)
    assert sum(int(torch.count_nonzero(x)) for x in long.split(4096)) == int(torch.count_nonzero(short))
    if fmt == "block":
        assert torch.equal(long_s[at.cuda()], short_s) and int(torch.count_nonzero(long_s)) == int(torch.count_nonzero(short_s))


# ------------------------------------------------------------------ behind pod_run
@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[9000, 400, 7000], [700] * 300], ids=["merged", "many"])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_write_right_behind_pod_run(lens, fp8):
    """The write may start while pod_run's kernel still reads the cache that it
    writes into: it may not touch it before. Nothing waits between the two."""
    H, hk, d, ps = 16, 2, 128, 16
    npg = [(n + ps - 1) // ps for n in lens]
    indptr = np.concatenate([[0], np.cumsum(npg)]).astype(np.int32)
    pages = int(indptr[-1])
    last = np.array([(n - 1) % ps + 1 for n in lens], dtype=np.int32)
    g = torch.Generator(device="cuda").manual_seed(3)
    old = torch.randn((pages, 2, ps, hk, d), generator=g, device="cuda")
    old = (old * 20).to(torch.float8_e4m3fn) if fp8 else old.to(BF)
    q = torch.randn((len(lens), H, d), generator=g, device="cuda").to(BF)
    h = pod.pod_plan(None, None, None, None, np.arange(len(lens) + 1, dtype=np.int32), indptr,
                     np.arange(pages, dtype=np.int32), last, H, hk, d, ps, True, -1, None, dtype=BF, p_num_pages=0,
                     d_num_pages=pages)
    kw = dict(k_scale=0.05, v_scale=0.05) if fp8 else {}
    if fp8:
        pod.pod_plan_set_decode_fp8(h, 0.05, 0.05)
    ws = torch.empty(pod.pod_workspace_size(h), dtype=torch.uint8, device="cuda")
    pod.pod_bind_workspace(h, ws)
    slots = torch.arange(pages * ps, device="cuda")
    new = torch.full((pages * ps, hk, d), 3.0, dtype=BF, device="cuda")
    kv = old.clone()
    want = pod.pod_run(h, None, None, q, kv, ws)[2:]
    torch.cuda.synchronize()
    for _ in range(4):
        kv = old.clone()
        torch.cuda.synchronize()
        got = pod.pod_run(h, None, None, q, kv, ws)[2:]
        pod.pod_append_kv(new, new, kv, slots, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (kv.float() * (0.05 if fp8 else 1) - 3).abs().max() < 0.2


@pytest.mark.gpu
def test_slots_of_device_tables():
    """The host's slots, nothing read outside the table (an index out of range would end
    the process), also in a graph."""
    req = np.array([0, 0, 0, 1, 2, 2, 2, -1, 3, 2, 0])
    pos = np.array([-1, 7, 8, 0, -4, 11, 12, 0, 0, 1 << 40, 0])
    want = pod.pod_kv_slots(INDPTR, INDICES, 4, req, pos).tolist()
    args = [torch.from_numpy(x).cuda() for x in (INDPTR, INDICES, req, pos)]
    call = lambda: pod.pod_kv_slots(args[0], args[1], 4, args[2], args[3])   # noqa: E731
    assert call().tolist() == want
    none = torch.zeros(0, dtype=torch.int32).cuda()
    assert pod.pod_kv_slots(torch.zeros(3, dtype=torch.int32).cuda(), none, 4, args[2], args[3]).tolist() == [-1] * 11
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        out = call()
    args[3] -= 4
    g.replay()
    torch.cuda.synchronize()
    assert out.tolist() == pod.pod_kv_slots(INDPTR, INDICES, 4, req, pos - 4).tolist()
