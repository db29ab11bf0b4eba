"""Attention of drafted token trees over a paged cache: against the 64-bit
definition on the GPU; the planner's tables and the refusals on the CPU.

Tolerances, fixed before the first run. An output is sum_t p_t v_t / l:
  - rounded once to its type: eps/2 of the value;
  - each weight is rounded to the operand type of P V: bf16 2^-8 of itself;
    fp16 2^-11, or 2^-25 of the largest weight below its normal range. For FP8
    caches it is two E4M3 parts of P, the largest P at least 2^6: x rounded to 4
    significant bits leaves at most 2^-4 of x's binade 2^e, 4 bits of that leave
    2^-9 * 2^e, and the remainder is taken from x in fp16, off by 2^-11 * 2^e: so
    2^-9 + 2^-11 of x; below E4M3's normal range (2^-6) the parts are
    multiples of 2^-9, at most 2^-10 off each, together 2^-9, which is 2^-15 of
    the largest weight. With fp16 results the remainder is two E5M2 parts of 3
    bits instead: 3 bits of at most 2^-4 * 2^e leave 2^-8 * 2^e, 3 bits of that
    2^-12 * 2^e; E5M2 ends at multiples of 2^-16, 2^-17 off, 2^-23 of the largest
    weight (2^-22 for the two). With
    block scales the weights are relative to the largest V scale. So at most
    u * sum p |v| / l + floor * sum |v in those units| / l;
  - the logits: products are exact in fp32, their sum of d terms is off by at
    most 2^-19 of sum |q k| (d <= 256 terms, 2^-23 each with partial sums), in
    base-2 units dx = 2^-19 * s * log2(e) * max_t sum_j |q_j k_tj| + 2^-19 (the
    exponential and the scaling); a weight is off by 2 dx relatively. With FP8
    caches q is scaled to a largest value of at least 2^7 and split into E4M3
    parts that end at multiples of 2^-9: off by 2^-10, so 2^-17 of the row's
    largest |q| times sum |k|, which joins dx;
  - fp32 sums over the keys: 2^-16 of sum p |v| / l covers 2^8 sequential
    sums a block accumulator takes.
The LSE is off by dx + 2^-20 * |lse| + 2^-18.
"""
import math

import numpy as np
import pytest
import torch

import prefill_decode_paged_pod_gb300 as pod


@pytest.fixture(scope="module", autouse=True)
def built():
    from prefill_decode_paged_pod_gb300 import _build
    _build.build()
    pod.load_library()


# ------------------------------------------------------------------ inputs and definition
class Case:
    def __init__(self, n, kv_len, H, Hk, d, ps, fmt="16bit", layout="NHD", dtype=torch.bfloat16, seed=0, spread=0,
                 mask="tree", sinks=False, q_mul=1.0):
        self.n, self.kv_len, self.H, self.Hk, self.d, self.ps = n, kv_len, H, Hk, d, ps
        self.fmt, self.layout, self.dtype, self.q_mul = fmt, layout, dtype, q_mul
        g = torch.Generator().manual_seed(seed + 17 * sum(kv_len) + d)
        r = np.random.RandomState(seed + sum(n))
        npg = [(x + ps - 1) // ps for x in kv_len]
        self.q_indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.kv_indptr = np.concatenate([[0], np.cumsum(npg)]).astype(np.int32)
        total = int(self.kv_indptr[-1])
        self.pages = total + 3
        self.kv_indices = r.permutation(self.pages)[:total].astype(np.int32)
        self.last = np.array([(x - 1) % ps + 1 if x else 1 for x in kv_len], dtype=np.int32)
        inner = (ps, Hk) if layout == "NHD" else (Hk, ps)
        shape = (self.pages, 2) + inner
        self.q = (torch.randn((sum(n), H, d), generator=g) * q_mul).to(dtype)
        self.scales, self.ks, self.vs = None, 1.0, 1.0
        x = torch.randn(shape + (d,), generator=g)
        if fmt == "16bit":
            self.kv = x.to(dtype)
        else:
            if fmt == "scaled":
                self.ks, self.vs = 0.017, 0.6
                x[:, 0] *= 1 / 0.017 * 0.7
                x[:, 1] *= 1 / 0.6
            else:
                x *= 100
                # exponents of K near 2^-7, of V spread over `spread` binades
                self.scales = torch.randint(118, 123, shape, generator=g, dtype=torch.uint8)
                if spread:
                    self.scales[:, 1] = torch.randint(120 - spread, 121, shape, generator=g, dtype=torch.uint8)[:, 1]
            self.kv = x.clamp(-448, 448).to(torch.float8_e4m3fn)
        # unused slots hold NaN
        flat = self.kv.view(torch.uint8) if fmt != "16bit" else self.kv
        used = torch.zeros((self.pages, ps), dtype=torch.bool)
        for i, kl in enumerate(kv_len):
            for t in range(kl):
                used[int(self.kv_indices[self.kv_indptr[i] + t // ps]), t % ps] = True
        sel = ~used[:, None, :, None].expand(-1, 2, -1, Hk) if layout == "NHD" else \
            ~used[:, None, None, :].expand(-1, 2, Hk, -1)
        flat[sel] = math.nan if fmt == "16bit" else 0x7F
        if self.scales is not None:
            self.scales[sel] = 0xFF
        # masks
        self.bits = []
        for x in n:
            m = np.zeros((x, x), dtype=np.uint8)
            if mask == "tree":
                for i in range(x):
                    m[i, i] = 1
                    p = r.randint(-1, i) if i else -1
                    if p >= 0:
                        m[i] |= m[p]
            elif mask == "random":
                m[:] = r.rand(x, x) < 0.5
                m[: (x + 2) // 3] = 0             # rows without tree keys
            elif mask is None:
                m[:] = np.tril(np.ones((x, x), dtype=np.uint8))
            self.bits.append(m)
        self.packed = None if mask is None else \
            torch.from_numpy(np.packbits(np.concatenate([b.reshape(-1) for b in self.bits]), bitorder="little"))
        self.sinks = torch.randn(H, generator=g) if sinks else None
        self.scale = 1 / math.sqrt(d)

    def rows64(self, r):
        t = np.arange(self.kv_len[r])
        pg = self.kv_indices[self.kv_indptr[r]:self.kv_indptr[r + 1]].astype(np.int64)[t // self.ps]
        x = self.kv.float()
        at = [(pg, h, t % self.ps) if self.layout == "NHD" else (pg, h, slice(None), t % self.ps) for h in (0, 1)]
        code = [x[torch.from_numpy(a[0]), a[1], torch.from_numpy(a[2])] if self.layout == "NHD" else
                x[torch.from_numpy(a[0]), a[1], :, torch.from_numpy(a[3])] for a in at]
        code = [c.double().numpy() for c in code]
        unit = [np.ones(c.shape[:2]), np.ones(c.shape[:2])] if (c := code[0]) is not None else None
        if self.fmt == "scaled":
            unit = [unit[0] * float(np.float32(self.ks)), unit[1] * float(np.float32(self.vs))]
        elif self.fmt == "block":
            s = self.scales.double()
            unit = [np.exp2((s[torch.from_numpy(a[0]), a[1], torch.from_numpy(a[2])] if self.layout == "NHD" else
                             s[torch.from_numpy(a[0]), a[1], :, torch.from_numpy(a[3])]).numpy() - 127) for a in at]
        return code[0] * unit[0][..., None], code[1], unit[1]

    def check(self, out, lse, seen_top=False):
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        G = self.H // self.Hk
        bf = self.dtype == torch.bfloat16
        if self.fmt == "16bit":
            u_p, tiny = (2.0 ** -8, 0.0) if bf else (2.0 ** -11, 2.0 ** -25)
        else:
            u_p, tiny = (2.0 ** -9 + 2.0 ** -11, 2.0 ** -15) if bf else (2.0 ** -12, 2.0 ** -22)
        eps = torch.finfo(self.dtype).eps / 2
        for r in range(len(self.n)):
            n, L = self.n[r], self.kv_len[r]
            if n == 0:
                continue
            k, vcode, vunit = self.rows64(r)
            see = np.ones((n, L), dtype=bool)
            see[:, L - n:] = self.bits[r] != 0
            q = self.q[self.q_indptr[r]:self.q_indptr[r] + n].double().numpy()
            for h in range(self.H):
                g = h // G
                kk, vv = k[:, g], vcode[:, g] * vunit[:, g][:, None]
                x = q[:, h] @ kk.T * (self.scale / math.log(2))
                x[~see] = -np.inf
                m = x.max(-1)
                some = np.isfinite(m)
                p = np.exp2(x - np.where(some, m, 0.0)[:, None])
                l = p.sum(-1)
                sink = np.exp2(float(self.sinks[h]) / math.log(2) - np.where(some, m, 0.0)) if self.sinks is not None else 0.0
                den = np.where(l + sink > 0, l + sink, 1.0)
                ref = p @ vv / den[:, None]
                dx = 2.0 ** -19 * (np.abs(q[:, h]) @ np.abs(kk).T).max(-1) * self.scale / math.log(2) + 2.0 ** -19
                if self.fmt != "16bit":
                    dx = dx + 2.0 ** -17 * np.abs(q[:, h]).max(-1) * np.abs(kk).sum(-1).max() * self.scale / math.log(2)
                pv = p @ np.abs(vv) / den[:, None]
                top = vunit[:, g].max()
                low = tiny * (see @ np.abs(vcode[:, g])) * top / den[:, None]
                if seen_top:
                    wu = (p * vunit[:, g]).max(-1)
                    low = 8 * tiny * (see @ np.abs(vcode[:, g])) * (wu / den)[:, None]
                tol = eps * np.abs(ref) * (1 + 2.0 ** -7) + (u_p * (1 + 2.0 ** -7) + 2 * dx[:, None] + 2.0 ** -16) * pv \
                    + low + torch.finfo(self.dtype).tiny
                a, b = int(self.q_indptr[r]), int(self.q_indptr[r]) + n
                got, most = out[a:b, h], float(torch.finfo(self.dtype).max)
                over = np.abs(ref) - tol > most * (1 + eps)          # rounds to infinity (fp16)
                assert (np.isinf(got[over]) & (np.sign(got[over]) == np.sign(ref[over]))).all(), (r, h)
                edge = (np.abs(ref) + tol >= most) & np.isinf(got)
                err = np.where(over | edge, 0.0, np.abs(np.where(over | edge, 0.0, got) - ref))
                assert np.isfinite(got[~(over | edge)]).all(), (r, h)
                bad = (err > tol) & ~(over | edge)
                assert not bad.any(), (r, h, np.argwhere(bad)[0], err[bad][0], tol[bad][0], err.max())
                want = np.where(some, m + np.log2(np.where(some, l, 1.0)), -np.inf)
                got = lse[a:b, h]
                assert np.array_equal(np.isneginf(got), ~some), (r, h)
                le = np.abs(got[some] - want[some])
                lt = dx[some] + 2.0 ** -20 * np.abs(want[some]) + 2.0 ** -18
                assert (le <= lt).all(), (r, h, le.max(), lt[le.argmax()])

    def plan(self, **kw):
        return pod.pod_tree_plan(self.q_indptr, self.kv_indptr, self.kv_indices, self.last, self.H, self.Hk, self.d,
                                 self.ps, dtype=self.dtype, num_pages=self.pages, kv_format=self.fmt,
                                 k_scale=self.ks, v_scale=self.vs, kv_layout=self.layout,
                                 has_sinks=self.sinks is not None, **kw)

    def args(self):
        c = lambda t: None if t is None else t.cuda()   # noqa: E731
        return c(self.q), c(self.kv), dict(tree_mask=c(self.packed), kv_scales=c(self.scales), sinks=c(self.sinks))

    def run(self, num_sms=0):
        h = self.plan(num_sms=num_sms)
        ws = torch.empty(max(256, pod.pod_tree_workspace_size(h)), dtype=torch.uint8, device="cuda")
        pod.pod_tree_bind_workspace(h, ws)
        q, kv, more = self.args()
        res = pod.pod_tree_run(h, q, kv, ws, **more)
        torch.cuda.synchronize()
        assert pod.pod_tree_read_device_status(h, ws) == 0
        again = pod.pod_tree_run(h, q, kv, ws, **more)
        assert torch.equal(res[0], again[0]) and torch.equal(res[1], again[1]), "two runs differ"
        return res


def run_once(c):
    h = c.plan()
    ws = torch.empty(max(256, pod.pod_tree_workspace_size(h)), dtype=torch.uint8, device="cuda")
    pod.pod_tree_bind_workspace(h, ws)
    q, kv, more = c.args()
    return pod.pod_tree_run(h, q, kv, ws, **more)


BF, HF = torch.bfloat16, torch.float16
CASES = {
    # smallest: one token and one key; a chain without a mask; keys at a block's edge
    "one": dict(n=[1], kv_len=[1], H=1, Hk=1, d=64, ps=16, dtype=HF),
    "edge": dict(n=[1, 2, 3, 4], kv_len=[64, 65, 63, 128], H=4, Hk=2, d=128, ps=16, mask=None),
    # tile fill: 32, 33, 64, 65, 128, 129 packed rows
    "rows32": dict(n=[8], kv_len=[200], H=4, Hk=1, d=128, ps=16),
    "rows33": dict(n=[11], kv_len=[200], H=3, Hk=1, d=128, ps=16, dtype=HF),
    "rows64": dict(n=[16, 1], kv_len=[200, 77], H=8, Hk=2, d=128, ps=32),
    "rows65": dict(n=[13], kv_len=[300], H=5, Hk=1, d=64, ps=8, dtype=HF),
    "rows128": dict(n=[16], kv_len=[1000], H=16, Hk=2, d=128, ps=64),
    "rows129": dict(n=[43], kv_len=[130], H=3, Hk=1, d=128, ps=128),
    "wide": dict(n=[64, 70], kv_len=[500, 70], H=16, Hk=2, d=128, ps=16, dtype=HF),
    "many_heads": dict(n=[3], kv_len=[90], H=150, Hk=1, d=64, ps=16),
    # trees over more than one mask word, masks with empty rows, nothing but the tree
    "long_tree": dict(n=[200], kv_len=[333], H=2, Hk=1, d=64, ps=16, mask="random"),
    "no_context": dict(n=[5, 40], kv_len=[5, 40], H=4, Hk=4, d=128, ps=16, mask="random", sinks=True),
    "chain_long": dict(n=[130], kv_len=[190], H=4, Hk=2, d=64, ps=16, mask=None, dtype=HF),
    # ragged batch with requests that have no tokens, sinks
    "ragged": dict(n=[0, 7, 1, 0, 19, 4], kv_len=[30, 700, 1, 0, 129, 1500], H=28, Hk=4, d=128, ps=16, sinks=True),
    # gathered page sizes
    "page1": dict(n=[6, 2], kv_len=[150, 64], H=8, Hk=2, d=128, ps=1),
    "page3_hnd": dict(n=[6, 2], kv_len=[150, 64], H=8, Hk=2, d=64, ps=3, layout="HND", dtype=HF),
    "page24": dict(n=[20], kv_len=[250], H=8, Hk=2, d=256, ps=24),
    "page4": dict(n=[9], kv_len=[100], H=8, Hk=8, d=128, ps=4, sinks=True),
    # TMA, head-major; head_dim 256
    "hnd": dict(n=[6, 2, 30], kv_len=[150, 64, 31], H=12, Hk=2, d=128, ps=16, layout="HND"),
    "d256": dict(n=[6, 50], kv_len=[350, 164], H=12, Hk=2, d=256, ps=16, dtype=HF, sinks=True),
    "d256_hnd": dict(n=[3], kv_len=[129], H=2, Hk=2, d=256, ps=8, layout="HND"),
    # FP8
    "f8": dict(n=[8, 1, 30], kv_len=[300, 17, 64], H=8, Hk=2, d=128, ps=16, fmt="scaled"),
    "f8_fp16": dict(n=[5, 33], kv_len=[500, 129], H=16, Hk=4, d=64, ps=32, fmt="scaled", dtype=HF, layout="HND"),
    "f8_page3": dict(n=[7], kv_len=[200], H=6, Hk=2, d=128, ps=3, fmt="scaled", sinks=True),
    "f8_256": dict(n=[7, 60], kv_len=[200, 90], H=4, Hk=2, d=256, ps=64, fmt="scaled"),
    "b8": dict(n=[8, 1, 30], kv_len=[300, 17, 64], H=8, Hk=2, d=128, ps=16, fmt="block"),
    "b8_fp16": dict(n=[5, 33], kv_len=[500, 129], H=16, Hk=4, d=64, ps=32, fmt="block", dtype=HF, layout="HND"),
    "b8_wide": dict(n=[40], kv_len=[1000], H=8, Hk=1, d=128, ps=16, fmt="block", spread=20),
    "b8_page1": dict(n=[7, 12], kv_len=[200, 65], H=6, Hk=2, d=128, ps=1, fmt="block", spread=12, sinks=True),
    "b8_256": dict(n=[7, 60], kv_len=[200, 90], H=4, Hk=2, d=256, ps=8, fmt="block", spread=6, dtype=HF),
    "b8_mask": dict(n=[20], kv_len=[20], H=7, Hk=1, d=128, ps=16, fmt="block", mask="random"),
    # large logits: the running maximum moves by far more than 8 and the weights are near one-hot
    "sharp": dict(n=[9], kv_len=[2000], H=8, Hk=1, d=128, ps=16, q_mul=12.0, dtype=HF),
    "sharp_b8": dict(n=[3], kv_len=[2000], H=8, Hk=1, d=128, ps=16, q_mul=12.0, fmt="block", spread=9),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_tree(name):
    c = Case(**CASES[name], seed=3)
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["ragged", "wide", "rows32", "rows64", "b8", "b8_wide", "f8_page3", "d256", "long_tree"])
@pytest.mark.parametrize("sms", [1, 3, 13])
def test_tree_cut_anywhere(name, sms):
    """Plans for other SM counts cut the units elsewhere; the result stays."""
    c = Case(**CASES[name], seed=4)
    c.check(*c.run(num_sms=sms))


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    dict(n=[8] * 6, kv_len=[3000, 17, 12000, 600, 9000, 64], H=32, Hk=8, d=128, ps=16),
    dict(n=[24, 5], kv_len=[6000, 9001], H=16, Hk=2, d=128, ps=16, fmt="block", spread=3),
    dict(n=[64], kv_len=[5000], H=32, Hk=4, d=128, ps=16, dtype=HF),
    dict(n=[4], kv_len=[40000], H=4, Hk=1, d=64, ps=16, fmt="scaled"),
], ids=["ragged", "block", "wide", "one_long"])
def test_tree_long(kw):
    c = Case(**kw, seed=9)
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["16bit", "block"])
def test_masked_keys_may_hold_anything_in_k(fmt):
    """K of a key that a row does not see may be infinite or NaN: that row is unchanged."""
    c = Case(n=[6], kv_len=[100], H=4, Hk=1, d=128, ps=16, fmt=fmt, seed=1)
    c.bits[0][:, 3] = 0
    c.packed = torch.from_numpy(np.packbits(c.bits[0].reshape(-1), bitorder="little"))
    want = c.run()
    t = 100 - 6 + 3
    pg = int(c.kv_indices[t // 16])
    raw = c.kv.view(torch.uint8) if fmt == "block" else c.kv
    raw[pg, 0, t % 16, 0, ::2] = 0x7F if fmt == "block" else math.inf
    raw[pg, 0, t % 16, 0, 1::2] = 0xFF if fmt == "block" else math.nan
    got = c.run()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    dict(n=[8, 3], kv_len=[700, 260], H=8, Hk=2, d=128, ps=16),
    dict(n=[16], kv_len=[300], H=4, Hk=1, d=64, ps=16, dtype=HF, layout="HND"),
    dict(n=[40], kv_len=[500], H=4, Hk=1, d=128, ps=64, dtype=HF),
    dict(n=[30], kv_len=[290], H=8, Hk=1, d=128, ps=3),
    dict(n=[20], kv_len=[300], H=4, Hk=1, d=256, ps=16),
], ids=["copies4", "copies2_fp16", "fp16", "gather", "d256"])
@pytest.mark.parametrize("sms", [0, 1])
def test_block_scales_of_keys_that_count_for_nothing(kw, sms):
    """V scales over dozens of binades: a row's accuracy is that of the keys it
    sees, with their weights. The weights times V scale are carried relative to
    the row's own largest (within 2^3: the reference moves lazily)."""
    c = Case(**kw, fmt="block", mask="random", seed=11)
    g = torch.Generator().manual_seed(5)
    s = c.scales[:, 1]
    s.copy_(torch.randint(100, 124, s.shape, generator=g, dtype=torch.uint8))
    for r in range(len(c.n)):                         # and huge drafted keys, seen by some rows
        L, n = c.kv_len[r], c.n[r]
        for t, b in [(L - 1, 190), (L - n, 150)]:
            pg, at = int(c.kv_indices[c.kv_indptr[r] + t // c.ps]), t % c.ps
            (s[pg, at] if c.layout == "NHD" else s[pg, :, at]).fill_(b)
    c.check(*c.run(num_sms=sms), seen_top=True)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["16bit", "scaled", "block"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_query_stays_in_its_row(fmt, bad):
    c = Case(n=[6], kv_len=[300], H=4, Hk=1, d=128, ps=16, fmt=fmt, seed=1)
    want = c.run()
    c.q[2, 1, 7] = bad
    got = run_once(c)
    assert got[0][2, 1].isnan().all()
    keep = torch.ones((6, 4), dtype=torch.bool)
    keep[2, 1] = False
    assert torch.equal(got[0].cpu()[keep], want[0].cpu()[keep]) and torch.equal(got[1].cpu()[keep], want[1].cpu()[keep])


@pytest.mark.gpu
def test_rows_outside_stay_and_optional_lse():
    """Only the planned rows are written; lse may be given or not."""
    import ctypes
    c = Case(**CASES["rows64"], seed=2)
    h = c.plan()
    ws = torch.empty(pod.pod_tree_workspace_size(h), dtype=torch.uint8, device="cuda")
    pod.pod_tree_bind_workspace(h, ws)
    q, kv, more = c.args()
    big = torch.full((h.rows + 4, c.H, c.d), 7.0, dtype=c.dtype, device="cuda")
    out, lse = pod.pod_tree_run(h, q, kv, ws, out=big[2:2 + h.rows], **more)
    c.check(out, lse)
    assert (big[:2] == 7).all() and (big[2 + h.rows:] == 7).all()
    lib = pod.load_library()
    out2 = torch.empty_like(out)
    code = lib.pod_tree_run(ctypes.c_void_p(h.ptr), q.data_ptr(), kv.data_ptr(), None, more["tree_mask"].data_ptr(),
                            more["tree_mask"].numel(), None, ws.data_ptr(), out2.data_ptr(), None,
                            torch.cuda.current_stream().cuda_stream)
    assert code == 0 and torch.equal(out2, out)


@pytest.mark.gpu
def test_graph_replay_and_two_plans():
    """Captured on a side stream and replayed on new tensors, next to a second
    plan with its own workspace on another stream."""
    a, b = Case(**CASES["ragged"], seed=5), Case(**CASES["b8"], seed=6)
    runs = []
    for c in (a, b):
        h = c.plan()
        ws = torch.empty(pod.pod_tree_workspace_size(h), dtype=torch.uint8, device="cuda")
        pod.pod_tree_bind_workspace(h, ws)
        q, kv, more = c.args()
        out = torch.empty((h.rows, c.H, c.d), dtype=c.dtype, device="cuda")
        lse = torch.empty((h.rows, c.H), dtype=torch.float32, device="cuda")
        pod.pod_tree_run(h, q, kv, ws, out=out, lse=lse, **more)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            pod.pod_tree_run(h, q, kv, ws, out=out, lse=lse, **more)
        runs.append((g, q, out, lse, h, ws, kv, more))
    a2 = Case(**CASES["ragged"], seed=5)
    a2.q = torch.randn(a2.q.shape, generator=torch.Generator().manual_seed(1)).to(a2.dtype)
    runs[0][1].copy_(a2.q)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            runs[0][0].replay()
        with torch.cuda.stream(s2):
            runs[1][0].replay()
    torch.cuda.synchronize()
    a2.check(runs[0][2], runs[0][3])
    b.check(runs[1][2], runs[1][3])
    assert all(pod.pod_tree_read_device_status(r[4], r[5]) == 0 for r in runs)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["16bit", "scaled", "block"])
def test_verification_step(fmt):
    """The operators as a serving step uses them: drafted tokens normed, rotated
    at their depth and written into the cache, then attended as a tree."""
    H, Hk, d, ps, dt = 8, 2, 128, 16, BF
    n, ctx = [6, 3], [100, 37]
    kv_len = [a + b for a, b in zip(n, ctx)]
    c = Case(n=n, kv_len=kv_len, H=H, Hk=Hk, d=d, ps=ps, fmt=fmt, seed=8)
    g = torch.Generator().manual_seed(0)
    qkv = torch.randn((sum(n), H + 2 * Hk, d), generator=g).to(dt).cuda()
    w = (1 + 0.1 * torch.randn((2, d), generator=g)).to(dt).cuda()
    depth = [c.bits[r].sum(1) - 1 for r in range(2)]
    pos = torch.from_numpy(np.concatenate([ctx[r] + depth[r] for r in range(2)]).astype(np.int32)).cuda()
    req = np.repeat([0, 1], n)
    at = np.concatenate([np.arange(ctx[r], kv_len[r]) for r in range(2)])
    slots = torch.from_numpy(pod.pod_kv_slots(c.kv_indptr, c.kv_indices, ps, req, at)).cuda()
    kv, sc = c.kv.cuda(), None if c.scales is None else c.scales.cuda()
    q = pod.pod_norm_rope_append(qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], pos, kv, slots, q_weight=w[0],
                                 k_weight=w[1], kv_scales=sc, k_scale=c.ks, v_scale=c.vs)
    h = c.plan()
    ws = torch.empty(pod.pod_tree_workspace_size(h), dtype=torch.uint8, device="cuda")
    pod.pod_tree_bind_workspace(h, ws)
    out, lse = pod.pod_tree_run(h, q, kv, ws, tree_mask=c.packed.cuda(), kv_scales=sc)
    c.q, c.kv, c.scales = q.cpu(), kv.cpu(), None if sc is None else sc.cpu()
    c.check(out, lse)
    # the written rows are the rotated keys: read back, and compared with the pass alone
    k = pod.pod_qk_norm_rope(None, qkv[:, H:H + Hk], pos, k_weight=w[1])[1].float()
    back = pod.pod_gather_kv(kv, slots, dtype=dt, kv_scales=sc, k_scale=c.ks, v_scale=c.vs)
    step = 2.0 ** -4 if fmt != "16bit" else 0.0
    assert ((back[:, 0].float() - k).abs() <= (step + 2.0 ** -7) * k.abs() + 0.01 * (fmt != "16bit")).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["16bit", "scaled", "block"])
def test_calls_right_behind_each_other(fmt):
    """Layers on one stream: each call's queries are the last one's output, its
    new keys are written by the call before; nothing waits on the host. The
    kernels may overlap, the results may not differ from waiting for each."""
    c = Case(n=[9, 30, 4], kv_len=[2500, 700, 40], H=8, Hk=2, d=128, ps=16, fmt=fmt, seed=2)
    h = c.plan(num_sms=20)                            # (few CTAs: cut units, a merge a call)
    assert len(pod.pod_tree_plan_table(h, 2)) > 0
    ws = torch.empty(pod.pod_tree_workspace_size(h), dtype=torch.uint8, device="cuda")
    pod.pod_tree_bind_workspace(h, ws)
    rows = sum(c.n)
    req = np.repeat(np.arange(3), c.n)
    at = np.concatenate([np.arange(a - b, a) for a, b in zip(c.kv_len, c.n)])
    slots = torch.from_numpy(pod.pod_kv_slots(c.kv_indptr, c.kv_indices, c.ps, req, at)).cuda()

    def layers(wait):
        q, kv, more = c.args()
        for _ in range(8):
            new = q[:, :2].contiguous()
            pod.pod_append_kv(new, new, kv, slots, kv_scales=more["kv_scales"], k_scale=c.ks, v_scale=c.vs)
            if wait:
                torch.cuda.synchronize()
            q, lse = pod.pod_tree_run(h, q, kv, ws, **more)
            if wait:
                torch.cuda.synchronize()
        return q, lse
    want, got = layers(True), layers(False)
    assert rows == len(got[0]) and torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert got[0].isfinite().all()


# ------------------------------------------------------------------ planner (host)
def tables(c, sms):
    h = c.plan(num_sms=sms)
    return (pod.pod_tree_plan_table(h, 0).reshape(-1, 16), pod.pod_tree_plan_table(h, 1),
            pod.pod_tree_plan_table(h, 2).reshape(-1, 8), h)


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("sms", [1, 5, 152])
def test_plan_covers_every_block_once(name, sms):
    c = Case(**CASES[name])
    segs, ctas, groups, h = tables(c, sms)
    G = c.H // c.Hk
    seen = {}
    for s in segs.tolist():
        g, row0, nrows, b0, b1, prow, kvl, ntok, qrow, page0, npg, lo, hi, copies = s[:14]
        r = [i for i in range(len(c.n)) if c.n[i] and c.q_indptr[i] == qrow][0]
        assert (kvl, ntok, page0, npg) == (c.kv_len[r], c.n[r], c.kv_indptr[r], c.kv_indptr[r + 1] - c.kv_indptr[r])
        assert (lo & 0xffffffff) + (hi << 32) == sum(x * x for x in c.n[:r])
        assert row0 % 128 == 0 and nrows == min(128, c.n[r] * G - row0)
        assert copies == (4 if nrows <= 32 else 2 if nrows <= 64 else 1)
        assert 0 <= b0 < b1
        seen.setdefault((r, g, row0), []).append((b0, b1, prow, nrows))
    tiles = {(r, g, m) for r in range(len(c.n)) for g in range(c.Hk) for m in range(0, c.n[r] * G, 128)}
    assert set(seen) == tiles
    prows = set()
    pieces = [int(x[4]) for x in groups]
    n_big = sum(p > 4 for p in pieces)
    assert all(p > 4 for p in pieces[:n_big]) and all(2 <= p <= 4 for p in pieces[n_big:])
    for (r, g, row0), parts in seen.items():
        at = 0
        for b0, b1, prow, nrows in parts:
            assert b0 == at
            at = b1
            assert (prow < 0) == (len(parts) == 1)
            if prow >= 0 and b0 == 0:
                assert [g, row0, nrows, prow, len(parts), int(c.q_indptr[r])] in groups[:, :6].tolist()
            if prow >= 0:
                mine = set(range(prow, prow + nrows))
                assert not mine & prows
                prows |= mine
        blk = 128 if c.fmt == "block" else 64
        assert at == (c.kv_len[r] + blk - 1) // blk
    assert prows == set(range(len(prows)))
    assert ctas[0] == 0 and ctas[-1] == len(segs) and (np.diff(ctas) > 0).all()
    planes = len({s[1] for s in segs.tolist()})
    assert len(ctas) - 1 <= max(sms * (1 if c.d == 256 else 2), planes)
    assert sum(int(g[2]) for g in groups) == sum(int(p[0][3]) for p in seen.values() if len(p) > 1)
    size = pod.pod_tree_workspace_size(h)
    assert size % 256 == 0 and size >= len(prows) * (c.d + 1) * 4


def test_plan_balances_long_requests():
    """No CTA has much more than the mean; a small batch is not cut to pieces."""
    r = np.random.RandomState(0)
    kv = r.randint(512, 16384, 64).tolist()
    n = [8] * 64
    npg = [(x + 15) // 16 for x in kv]
    ind = np.concatenate([[0], np.cumsum(npg)]).astype(np.int32)
    h = pod.pod_tree_plan(np.arange(65) * 8, ind, np.arange(ind[-1]), [(x - 1) % 16 + 1 for x in kv], 32, 8, 128, 16,
                          dtype=BF, num_pages=int(ind[-1]), num_sms=152)
    segs, ctas = pod.pod_tree_plan_table(h, 0).reshape(-1, 16), pod.pod_tree_plan_table(h, 1)
    cost = [int((segs[a:b, 4] - segs[a:b, 3] + 3).sum()) for a, b in zip(ctas[:-1], ctas[1:])]
    assert len(cost) <= 304 and max(cost) <= 1.02 * sum(cost) / 304 + 4
    assert n


def test_plan_keeps_short_units_whole():
    """No merge launch where the longest unit is little more than a share."""
    c = Case(n=[5, 8, 6, 7], kv_len=[600, 17, 333, 400], H=32, Hk=8, d=128, ps=16)
    segs, ctas, groups, _ = tables(c, 152)
    assert len(groups) == 0 and (segs[:, 5] == -1).all() and len(segs) == 32
    c = Case(n=[5], kv_len=[3000], H=32, Hk=8, d=128, ps=16)
    assert len(tables(c, 152)[2]) == 8


P = 1 << 20


def plan_call(**kw):
    import ctypes
    a = dict(qi=[0, 4, 9], ki=[0, 2, 5], idx=[0, 1, 2, 3, 4], last=[3, 16], pages=5, H=8, Hk=2, d=128, ps=16,
             scale=0.0, dt=1, fmt=0, ks=1.0, vs=1.0, lay=0)
    a.update(kw)
    arr = [None if a[k] is None else np.ascontiguousarray(a[k], dtype=np.int32) for k in ("qi", "ki", "idx", "last")]
    h, req = ctypes.c_void_p(), ctypes.c_size_t()
    code = pod.load_library().pod_tree_plan(
        *[None if x is None else x.ctypes.data for x in arr], a.get("batch", 2), a["pages"], a["H"], a["Hk"], a["d"],
        a["ps"], a["scale"], a["dt"], a["fmt"], a["ks"], a["vs"], a["lay"], 0, 152, None, 0, None, ctypes.byref(h),
        ctypes.byref(req))
    assert (h.value is None) == (code != 0)
    if h.value:
        pod.load_library().pod_tree_destroy(h)
    return code


@pytest.mark.parametrize("kw,code,text", [
    (dict(H=7), 1, "multiple"), (dict(Hk=0), 1, "multiple"), (dict(d=96), 2, "head_dim"), (dict(ps=0), 1, "page_size"),
    (dict(pages=4), 1, "outside the pool"), (dict(idx=[0, 1, 2, -1, 4]), 1, "outside the pool"),
    (dict(last=[0, 16]), 1, "last_page_len"), (dict(last=[3, 17]), 1, "last_page_len"),
    (dict(qi=[0, 20, 25]), 1, "kv_len >= q_len"), (dict(qi=[1, 4, 9]), 1, "start at 0"),
    (dict(qi=[0, 4, 3]), 1, "decreases"), (dict(ki=[0, 3, 2]), 1, "decreases"), (dict(qi=None), 1, "NULL"),
    (dict(idx=None), 1, "NULL"), (dict(dt=3), 2, "dtype"), (dict(fmt=3), 1, "format"), (dict(lay=2), 1, "kv_layout"),
    (dict(fmt=1, ks=0.0), 1, "k_scale"), (dict(fmt=1, vs=math.inf), 1, "v_scale"), (dict(scale=math.nan), 1, "sm_scale"),
    (dict(ki=[0, 2, 2 ** 30 // 16 + 4], idx=[0] * (2 ** 30 // 16 + 4)), 1, "2^30 keys"), (dict(batch=-1), 1, "batch"), (dict(pages=2 ** 30), 1, "too large"),
])
def test_plan_refusals(kw, code, text):
    assert plan_call(**kw) == code and text in pod.pod_last_error(), pod.pod_last_error()


def test_plan_accepts_the_defaults_and_an_empty_batch():
    assert plan_call() == 0
    assert plan_call(batch=0, qi=None, ki=None, idx=None, last=None, pages=0) == 0


def test_run_refusals():
    """Checked on the host before anything is launched."""
    import ctypes
    lib = pod.load_library()
    c = Case(**CASES["rows64"])
    h = c.plan(num_sms=4)
    run = lambda **k: lib.pod_tree_run(*[{**dict(h=ctypes.c_void_p(h.ptr), q=P, kv=P, sc=None, m=P, mb=10 ** 6,  # noqa: E731
                                                 s=None, ws=P, o=P, l=P, st=None), **k}[x]
                                         for x in ("h", "q", "kv", "sc", "m", "mb", "s", "ws", "o", "l", "st")])
    assert run() == 3 and "no bound workspace" in pod.pod_last_error()
    assert run(h=None) == 1
    assert lib.pod_tree_bind_workspace(ctypes.c_void_p(h.ptr), P, 16, None) == 3
    assert lib.pod_tree_bind_workspace(ctypes.c_void_p(h.ptr), P + 16, 1 << 30, None) == 3
    with pytest.raises(pod.PodError, match="CUDA"):
        pod.pod_tree_run(h, c.q, c.kv, torch.empty(16, dtype=torch.uint8))
    with pytest.raises(pod.PodError, match="fit together"):
        pod.pod_tree_plan([0, 1], [0, 1], [], [1], 1, 1, 64, 16, dtype=HF, num_pages=1)
    with pytest.raises(pod.PodError, match="kv_format"):
        pod.pod_tree_plan([0, 1], [0, 1], [0], [1], 1, 1, 64, 16, dtype=HF, num_pages=1, kv_format="int8")


@pytest.mark.gpu
def test_run_refusals_of_a_bound_plan():
    c = Case(**CASES["rows64"])
    s = Case(**CASES["no_context"])
    b = Case(**CASES["b8"])
    for x, bad in (
        (c, [dict(sinks=torch.zeros(8).cuda()), dict(tree_mask=torch.zeros(3).byte().cuda()),
             dict(kv_scales=torch.zeros(3).byte().cuda()), dict(out=torch.zeros(1).cuda())]),
        (s, [dict(sinks=None)]), (b, [dict(kv_scales=None)]),
    ):
        h = x.plan()
        ws = torch.empty(pod.pod_tree_workspace_size(h), dtype=torch.uint8, device="cuda")
        q, kv, more = x.args()
        with pytest.raises(pod.PodError, match="bound"):
            pod.pod_tree_run(h, q, kv, ws, **more)
        pod.pod_tree_bind_workspace(h, ws)
        for k in bad:
            with pytest.raises(pod.PodError):
                pod.pod_tree_run(h, q, kv, ws, **{**more, **k})
        with pytest.raises(pod.PodError):
            pod.pod_tree_run(h, q[:-1], kv, ws, **more)
        with pytest.raises(pod.PodError):
            pod.pod_tree_run(h, q, kv[:-1], ws, **more)
        with pytest.raises(pod.PodError):
            pod.pod_tree_run(h, q, kv, torch.empty_like(ws), **more)
