"""Measured cases of decode steps whose tables live on the GPU.

Five kinds of call, each with a plain form in elementary torch operations
(fp32, 64 bits where pages compete for a place, rounded once at the end) and,
where ``own`` is true, the library's entry points:

  tables   request lengths to pages, slots, positions and page tables
           (pod_step_tables)
  bounds   smallest and largest key of every page that a step wrote into, per
           KV head and channel (pod_page_bounds)
  select   the pages whose bounds promise a query the largest logits
           (pod_select_pages)
  decode   attention of one token per request over its paged cache
           (pod_paged_decode)
  sparse   a layer of a long-context step: pages selected, then attended
           (pod_select_pages, pod_paged_decode)

Shapes are those of the library's own configurations (heads 64/8, 32/8 and
4/1, head_dim 128 and 64, pages of 16 and 1 slots) and neighbours of them.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
K_SCALE, V_SCALE = 0.03125 * 1.1, 0.0125     # calibration scales of the per-tensor FP8 cache
E4M3_MAX = 448.0


# ----------------------------------------------------------------- cases
def listed():
    return [
        # the start of one decode step of 64 requests: latency of a scan and some page pops
        dict(name="tables_decode", op="tables", batch=64, width=1024, ps=16, new_hi=1, mixed=False,
             csr=False, lens=11),
        # a mixed batch: prompts, decodes, idle requests, drafted tokens taken back, and the page
        # table end to end as the host planner reads it
        dict(name="tables_mixed", op="tables", batch=768, width=1024, ps=16, new_hi=2000, mixed=True,
             csr=True, lens=12),
        # the bounds after a decode step of 64 requests: one page of eight heads each
        dict(name="bounds_decode", op="bounds", batch=64, new_lo=1, new_hi=1, kv_hi=16384, Hk=8, d=128,
             ps=16, fmt="16bit", layout="NHD", dtype="bf16", lens=13),
        # the bounds of long prompts in a block-scaled FP8 cache
        dict(name="bounds_prompts", op="bounds", batch=6, new_lo=1000, new_hi=16384, kv_hi=16384, Hk=8,
             d=128, ps=16, fmt="block", layout="HND", dtype="fp16", lens=14),
        # two users with some thousand keys: launches and the selection itself
        dict(name="select_small", op="select", batch=2, kv_lo=2000, kv_hi=6000, H=32, Hk=8, d=128,
             ps=16, pages=64, first=1, last=2, dtype="bf16", lens=15),
        # 64 requests of up to 32768 keys: the bounds are read once, 128 pages stay
        dict(name="select_long", op="select", batch=64, kv_lo=8192, kv_hi=32768, H=64, Hk=8, d=128,
             ps=16, pages=128, first=1, last=4, dtype="bf16", lens=16),
        # four users, short contexts: latency
        dict(name="decode_small", op="decode", batch=4, kv_lo=17, kv_hi=600, H=32, Hk=8, d=128, ps=16,
             window=-1, fmt="16bit", layout="NHD", dtype="bf16", lens=17),
        # a decode step of 64 requests with ragged long contexts
        dict(name="decode_ragged", op="decode", batch=64, kv_lo=512, kv_hi=16384, H=32, Hk=8, d=128,
             ps=16, window=-1, fmt="16bit", layout="NHD", dtype="bf16", lens=18),
        # one long context: every SM works on the same request
        dict(name="decode_long", op="decode", batch=1, kv_lo=131000, kv_hi=131072, H=64, Hk=8, d=128,
             ps=16, window=-1, fmt="16bit", layout="HND", dtype="fp16", lens=19),
        # a decode step over a block-scaled FP8 cache, eight query heads a KV head
        dict(name="decode_block", op="decode", batch=96, kv_lo=4096, kv_hi=12288, H=64, Hk=8, d=128,
             ps=16, window=-1, fmt="block", layout="NHD", dtype="bf16", lens=20),
        # one user with a long context over per-tensor FP8, 64 pages of it attended
        dict(name="sparse_single", op="sparse", batch=1, kv_lo=65000, kv_hi=65536, H=32, Hk=8, d=128,
             ps=16, pages=64, first=1, last=2, fmt="scaled", layout="HND", dtype="fp16", lens=21),
        # a long-context batch: 2048 of up to 32768 keys attended
        dict(name="sparse_batch", op="sparse", batch=32, kv_lo=16384, kv_hi=32768, H=64, Hk=8, d=128,
             ps=16, pages=128, first=1, last=4, fmt="16bit", layout="NHD", dtype="bf16", lens=22),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "bounds", "select", "decode", "decode", "decode", "sparse", "sparse"])
    if op == "tables":
        mixed = rng.random() < 0.6
        batch = _log_int(rng, 1, 700)
        return dict(op=op, batch=batch, width=_log_int(rng, 8, 1024), ps=rng.choice([1, 3, 16, 16, 32, 64]),
                    new_hi=_log_int(rng, 1, 1500) if mixed else 1, mixed=mixed, csr=rng.random() < 0.5,
                    lens=rng.randrange(1 << 30))
    c = dict(op=op, Hk=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128, 128, 128, 256]),
             dtype=rng.choice(["bf16", "fp16"]), lens=rng.randrange(1 << 30))
    G = rng.choice([1, 3, 4, 5, 7, 8, 8, 12, 16])
    if op != "select":
        c.update(fmt=rng.choice(["16bit", "scaled", "block"]), layout=rng.choice(["NHD", "HND"]))
    if op == "bounds":
        new_hi = _log_int(rng, 1, 8000)
        return dict(c, batch=_log_int(rng, 1, max(1, min(256, 40000 // new_hi))), new_lo=rng.choice([1, new_hi]),
                    new_hi=new_hi, kv_hi=max(new_hi, _log_int(rng, 16, 16384)), ps=rng.choice([8, 16, 16, 32, 64]))
    # requests x longest context stay within the largest listed case's reading
    kv_hi = _log_int(rng, 8, 32768)
    total = 1000000 if op == "select" else 400000
    batch = _log_int(rng, 1, max(1, min(256, total * 128 // c["d"] // kv_hi)))
    c.update(batch=batch, kv_lo=rng.choice([0, kv_hi // 8, kv_hi]), kv_hi=kv_hi, H=c["Hk"] * G)
    if op == "decode":
        return dict(c, ps=rng.choice([1, 3, 16, 16, 32, 64]), window=rng.choice([-1, -1, -1, kv_hi // 3]))
    last = rng.choice([1, 2, 4])
    return dict(c, ps=rng.choice([8, 16, 16, 32, 64]), pages=_log_int(rng, 8, 300), first=rng.choice([0, 1, 2]),
                last=last)


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _cache(g, pages, case):
    """A paged cache with every slot filled, and the scale bytes of a block-scaled one."""
    ps, Hk, d, fmt = case["ps"], case["Hk"], case["d"], case["fmt"]
    inner = (ps, Hk) if case["layout"] == "NHD" else (Hk, ps)
    kv = torch.empty((pages, 2) + inner + (d,), device="cuda",
                     dtype=DTYPES[case["dtype"]] if fmt == "16bit" else torch.float8_e4m3fn)
    step = max(1, (1 << 27) // (2 * ps * Hk * d))
    for a in range(0, pages, step):
        x = torch.randn((min(step, pages - a), 2) + inner + (d,), generator=g, device="cuda")
        if fmt == "scaled":      # codes of N(0,1) values under the calibration scales
            x[:, 0] *= 1 / K_SCALE
            x[:, 1] *= 1 / V_SCALE
            x.clamp_(-E4M3_MAX, E4M3_MAX)
        elif fmt == "block":     # a head row's largest value lies in the top of the E4M3 range
            x *= 120.0
            x.clamp_(-E4M3_MAX, E4M3_MAX)
        kv[a:a + step] = x.to(kv.dtype)
    scales = None
    if fmt == "block":           # 120 * 2^-7 is about 1; other tokens are up to 8 times larger or smaller
        scales = torch.randint(117, 124, (pages, 2) + inner, generator=g, device="cuda", dtype=torch.uint8)
    return kv, scales


def _lens(case):
    """Key counts of the requests: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    return [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["batch"])]


def _table(g, kv_len, ps, extra=0):
    """Block table of requests whose pages lie anywhere in the pool, -1 behind a request's pages."""
    n = [(x + ps - 1) // ps for x in kv_len]
    total = max(1, sum(n)) + extra
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(n))
    at = torch.tensor(np.concatenate([[0], np.cumsum(n)[:-1]]), device="cuda")
    i = torch.arange(width, device="cuda")
    inside = i[None] < torch.tensor(n, device="cuda")[:, None]
    table = torch.where(inside, perm[(at[:, None] + i).clamp(max=total - 1)], -1)
    return table.to(torch.int32).contiguous(), total


def _steps(case):
    """Keys before a step and new tokens of it: prompts, single tokens, idle requests and
    requests that give tokens back. Part of the case."""
    r = random.Random(case["lens"])
    most = case["width"] * case["ps"]
    old, new = [], []
    for _ in range(case["batch"]):
        kind = r.random() if case["mixed"] else 0.5
        if kind < 0.1:                                   # a prompt, or the next chunk of one
            n = min(r.randint(1, case["new_hi"]), most)
            a = r.choice([0, r.randint(0, most - n)])
        elif kind < 0.8:
            n, a = 1, r.randint(0, most - 1)
        elif kind < 0.9:
            n, a = 0, r.randint(0, most)
        else:                                            # drafted tokens that were not accepted
            a = r.randint(0, most)
            n = -min(a, r.randint(1, 8) if kind < 0.97 else most)
        old.append(a)
        new.append(n)
    return old, new


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "tables":
        ps, W = case["ps"], case["width"]
        old, new = _steps(case)
        s["table"], total = _table(g, [W * ps] * case["batch"], ps)
        s["kv_lens"] = torch.tensor(old, dtype=torch.int32, device="cuda")
        s["new_lens"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        # what no request holds is free, in any order
        held = [(a + ps - 1) // ps for a in old]
        i = torch.arange(W, device="cuda")
        loose = s["table"][i[None] >= torch.tensor(held, device="cuda")[:, None]]
        s["free"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        order = torch.randperm(loose.numel(), generator=g, device="cuda")
        s["free"][:loose.numel()] = loose[order]
        s["free_count"] = torch.tensor([loose.numel()], dtype=torch.int32, device="cuda")
        # buffers that a program keeps over its steps: rows and pages up to the largest step
        s["max_rows"] = max(1, sum(max(0, n) for n in new)) + 5
        s["max_pages"] = sum((a + max(n, 0) + ps - 1) // ps for a, n in zip(old, new)) + 7 if case["csr"] else 0
        s["kv_lens_out"], s["free_count_out"] = torch.empty_like(s["kv_lens"]), torch.empty_like(s["free_count"])
        return s
    dt = DTYPES[case["dtype"]]
    B, Hk, d, ps = case["batch"], case["Hk"], case["d"], case["ps"]
    if case["op"] == "bounds":
        r = random.Random(case["lens"])
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
        kv = [r.randint(n, max(n, case["kv_hi"])) for n in new]
        # the pool holds the pages that the step touches; earlier ones stay out of it
        first = [(b - n) // ps for n, b in zip(new, kv)]
        touched = [(b + ps - 1) // ps - f for b, f in zip(kv, first)]
        pages = sum(touched)
        s["kv"], s["scales"] = _cache(g, pages, case)
        perm = torch.randperm(pages, generator=g, device="cuda")
        pos, at, page0 = [], [], 0
        for n, b, f, t in zip(new, kv, first, touched):
            p = np.arange(b - n, b)
            pos.append(p % ps)
            at.append(page0 + p // ps - f)
            page0 += t
        pos, at = (torch.from_numpy(np.concatenate(x)).cuda() for x in (pos, at))
        s["slots"] = perm[at] * ps + pos
        s["bounds"] = _randn(g, (pages, Hk, 2, d), dt)
        return s
    kv_len = _lens(case)
    s["kv_lens"] = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    s["table"], pages = _table(g, kv_len, ps, extra=3)
    s["q"] = _randn(g, (B, case["H"], d), dt)
    s["scale"] = 1.0 / math.sqrt(d)
    if case["op"] in ("decode", "sparse"):
        s["kv"], s["scales"] = _cache(g, pages, case)
    if case["op"] == "select":
        # smallest and largest of ps keys of N(0,1) values
        a, b = torch.randn((2, pages, Hk, d), generator=g, device="cuda") * 0.5 + math.sqrt(2 * math.log(ps)) * 0.8
        s["bounds"] = torch.stack([torch.minimum(-a, b), torch.maximum(-a, b)], 2).to(dt)
    if case["op"] == "sparse":
        s["bounds"] = torch.empty((pages, Hk, 2, d), device="cuda", dtype=dt)
        step = max(1, (1 << 26) // (ps * Hk * d))
        for a in range(0, pages, step):
            n = min(step, pages - a)
            i = torch.arange(ps, device="cuda")
            p = torch.arange(a, a + n, device="cuda")[:, None]
            k = _values(s["kv"], s["scales"], p, 0, i.expand(n, ps), case)      # [n, ps, Hk, d]
            s["bounds"][a:a + n] = _outward(k.amin(1), k.amax(1), dt)
    if own:
        import prefill_decode_paged_pod_gb300 as pod
        if case["op"] in ("select", "sparse"):
            n = pod.pod_select_pages_workspace_size(B, Hk, s["table"].shape[1])
            s["ws_select"] = torch.empty(max(256, n), dtype=torch.uint8, device="cuda")
        if case["op"] in ("decode", "sparse"):
            n = pod.pod_paged_decode_workspace_size(B, case["H"], Hk, d)
            s["ws"] = torch.empty(max(256, n), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    if case["op"] == "tables":
        return _tables(s, case)
    if case["op"] == "bounds":
        return _bounds(s, case)
    if case["op"] == "select":
        return _select(s, case)
    if case["op"] == "decode":
        return _decode(s, case)
    pages = _select(s, case)
    return (pages,) + _attend_pages(s, case, pages)


def _own(s, case):
    import prefill_decode_paged_pod_gb300 as pod
    if case["op"] == "tables":
        t = pod.pod_step_tables(s["table"], s["kv_lens"], s["new_lens"], s["free"], s["free_count"], case["ps"],
                                max_rows=s["max_rows"], max_pages=s["max_pages"], kv_lens_out=s["kv_lens_out"],
                                free_count_out=s["free_count_out"])
        out = dict(table=s["table"], free=s["free"], free_count=s["free_count_out"], kv_lens=t.kv_lens,
                   q_indptr=t.q_indptr, requests=t.requests, positions=t.positions, slots=t.slots)
        if case["csr"]:
            out.update(kv_indptr=t.kv_indptr, kv_indices=t.kv_indices, last_page_len=t.last_page_len)
        return out
    scale = dict(k_scale=K_SCALE) if case.get("fmt") == "scaled" else {}
    if case["op"] == "bounds":
        return pod.pod_page_bounds(s["kv"], s["bounds"], s["slots"], kv_scales=s["scales"],
                                   kv_layout=case["layout"], **scale)
    pages = None
    if case["op"] in ("select", "sparse"):
        pages = pod.pod_select_pages(s["q"], s["bounds"], s["table"], s["kv_lens"], case["pages"], case["ps"],
                                     keep_first=case["first"], keep_last=case["last"], workspace=s["ws_select"])
        if case["op"] == "select":
            return pages
    if scale:
        scale["v_scale"] = V_SCALE
    out, lse = pod.pod_paged_decode(s["q"], s["kv"], s["table"], s["kv_lens"], pages=pages, sm_scale=s["scale"],
                                    window_left=case.get("window", -1), kv_scales=s["scales"],
                                    kv_layout=case["layout"], workspace=s["ws"], **scale)
    return (out, lse) if pages is None else (pages, out, lse)


def _tables(s, case):
    """Pages of shrinking requests go onto the free stack in the order of the requests, then
    growing ones take theirs off its top. (Every step of these cases fits.)"""
    ps, table, free = case["ps"], s["table"], s["free"]
    old, new = s["kv_lens"].long(), s["new_lens"].long()
    length = (old + new).clamp(min=0)
    had, has = (old + ps - 1) // ps, (length + ps - 1) // ps
    i = torch.arange(table.shape[1], device="cuda")
    given = (i >= has[:, None]) & (i < had[:, None])
    taken = (i >= had[:, None]) & (i < has[:, None])
    back = table[given]
    count = s["free_count"].long() + back.numel()
    free[count - back.numel() + torch.arange(back.numel(), device="cuda")] = back
    n = int(taken.sum())
    table[taken] = free[count - 1 - torch.arange(n, device="cuda")]
    rows = new.clamp(min=0)
    q_indptr = torch.cat([rows.new_zeros(1), rows.cumsum(0)])
    r = torch.arange(s["max_rows"], device="cuda")
    live = r < q_indptr[-1]
    req = (torch.searchsorted(q_indptr, r, right=True) - 1).clamp(max=old.numel() - 1)
    pos = torch.where(live, old[req] + r - q_indptr[req], 0)
    slots = torch.where(live, table[req, pos // ps].long() * ps + pos % ps, -1)
    out = dict(table=table, free=free, free_count=(count - n).int(), kv_lens=length.int(), q_indptr=q_indptr.int(),
               requests=torch.where(live, req, -1).int(), positions=pos.int(), slots=slots)
    if case["csr"]:
        kv_indptr = torch.cat([has.new_zeros(1), has.cumsum(0)])
        indices = torch.full((s["max_pages"],), -1, dtype=torch.int32, device="cuda")
        flat = table[i < has[:, None]]
        indices[:flat.numel()] = flat
        out.update(kv_indptr=kv_indptr.int(), kv_indices=indices,
                   last_page_len=torch.where(length > 0, (length - 1) % ps + 1, 0).int())
    return out


def _pow2(e, dtype):
    """2^e exactly, from the bits of a 64-bit float."""
    return ((e.long() + 1023) << 52).view(torch.float64).to(dtype)


def _values(kv, scales, page, half, slot, case, wide=torch.float32):
    """Cache rows [..., Hk, d] of the given pages and slots in `wide`."""
    raw = kv.view(torch.uint8) if kv.dtype.itemsize == 1 else kv
    x = raw[page, half, slot] if case["layout"] == "NHD" else raw[page, half, :, slot]
    x = (x.view(kv.dtype) if kv.dtype.itemsize == 1 else x).to(wide)
    if case["fmt"] == "scaled":
        x = x * (V_SCALE if half else K_SCALE)
    elif case["fmt"] == "block":
        e = scales[page, half, slot] if case["layout"] == "NHD" else scales[page, half, :, slot]
        x = x * _pow2(e.int() - 127, wide)[..., None]
    return x


def _outward(lo, hi, dtype):
    """[..., 2, d]: lo rounded down and hi rounded up to `dtype`, within its finite values."""
    big = torch.finfo(dtype).max
    out = []
    for x, sign in ((lo, -1), (hi, 1)):
        x = x.clamp(-big, big)
        y = x.to(dtype)
        off = (y.to(x.dtype) - x) * sign < 0                 # on the wrong side: one step further
        bits = y.view(torch.int16).int()
        up = torch.where(bits >= 0, 1, -1) * sign            # magnitude grows away from zero
        moved = torch.where(y == 0, 1 if sign > 0 else -32767, bits + up).to(torch.int16).view(dtype)
        out.append(torch.where(off, moved, y))
    return torch.stack(out, -2)


def _bounds(s, case):
    ps = case["ps"]
    page, slot = s["slots"] // ps, s["slots"] % ps
    pages = s["kv"].shape[0]
    # a page is valid up to the last slot that was written
    valid = torch.zeros(pages, dtype=torch.long, device="cuda").scatter_reduce_(0, page, slot + 1, "amax")
    i = torch.arange(ps, device="cuda")
    step = max(1, (1 << 26) // (ps * case["Hk"] * case["d"]))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        p = torch.arange(a, a + n, device="cuda")
        k = _values(s["kv"], s["scales"], p[:, None], 0, i.expand(n, ps), case)
        dead = (i >= valid[p, None])[..., None, None]
        new = _outward(k.masked_fill(dead, math.inf).amin(1), k.masked_fill(dead, -math.inf).amax(1),
                       s["bounds"].dtype)
        s["bounds"][p] = torch.where((valid[p] > 0)[:, None, None, None], new, s["bounds"][p])
    return s["bounds"]


def _select(s, case):
    """Positions of the chosen pages in their request's table, ascending, -1 behind them."""
    B, H, Hk, d, ps, k = (case[x] for x in ("batch", "H", "Hk", "d", "ps", "pages"))
    n = ((s["kv_lens"].long() + ps - 1) // ps)[:, None, None]
    q = s["q"].double().view(B, Hk, H // Hk, d)
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    W = s["table"].shape[1]
    score = torch.empty((B, Hk, W), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 27) // (W * Hk * 2 * d))
    for a in range(0, B, step):
        b = s["bounds"][s["table"][a:a + step].long().clamp(min=0)].double()     # [., W, Hk, 2, d]
        score[a:a + step] = torch.einsum("bwhd,bhd->bhw", b[..., 0, :], down[a:a + step]) + \
            torch.einsum("bwhd,bhd->bhw", b[..., 1, :], up[a:a + step])
    i = torch.arange(W, device="cuda")
    score = score.masked_fill((i < case["first"]) | (i >= n - case["last"]), math.inf).masked_fill(i >= n, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    rank = torch.arange(order.shape[-1], device="cuda")
    pick = torch.where(rank < n, order, W).sort(-1).values
    out = torch.full((B, Hk, k), -1, dtype=torch.int32, device="cuda")
    out[..., :pick.shape[-1]] = torch.where(pick < W, pick, -1).int()
    return out


def _softmax_sum(x, see, v):
    """Weighted sum of v [B, Hk, L, d] under softmax(x [B, Hk, G, L]) where `see`, and the base-2 LSE."""
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgl,bhld->bhgd", p / z.clamp(min=1e-30), v)
    lse = (m + torch.log(z)) / math.log(2.0)
    return o, lse.squeeze(-1)


def _attend(s, case, page, slot, see):
    """Attention over keys [B, Hk or 1, L] of given pages and slots, a few requests at a time."""
    B, H, Hk, d = case["batch"], case["H"], case["Hk"], case["d"]
    L = slot.shape[-1]
    outs, lses = [], []
    step = max(1, (1 << 28) // (max(L, 1) * Hk * d))
    heads = torch.arange(Hk, device="cuda")[:, None]
    for a in range(0, B, step):
        pg, sl, ok = (x[a:a + step].expand(-1, Hk, -1) for x in (page, slot, see))
        kv = []
        for half, sc in ((0, K_SCALE), (1, V_SCALE)):
            raw = s["kv"].view(torch.uint8) if s["kv"].dtype.itemsize == 1 else s["kv"]
            at = (pg, half, sl, heads) if case["layout"] == "NHD" else (pg, half, heads, sl)
            x = raw[at]
            x = (x.view(s["kv"].dtype) if s["kv"].dtype.itemsize == 1 else x).float()
            if case["fmt"] == "scaled":
                x = x * sc
            elif case["fmt"] == "block":
                x = x * _pow2(s["scales"][at].int() - 127, torch.float32)[..., None]
            kv.append(x)
        q = s["q"][a:a + step].float().view(-1, Hk, H // Hk, d)
        x = torch.einsum("bhgd,bhld->bhgl", q, kv[0]) * s["scale"]
        o, lse = _softmax_sum(x, ok[:, :, None], kv[1].masked_fill(~ok[..., None], 0.0))
        outs.append(o.reshape(-1, H, d).to(s["q"].dtype))
        lses.append(lse.reshape(-1, H))
    return torch.cat(outs), torch.cat(lses)


def _decode(s, case):
    ps = case["ps"]
    kv_len = s["kv_lens"].long()[:, None, None]
    t = torch.arange(s["table"].shape[1] * ps, device="cuda")
    see = t < kv_len
    if case["window"] >= 0:
        see &= t >= kv_len - 1 - case["window"]
    page = s["table"][:, t // ps].long().clamp(min=0)[:, None]
    return _attend(s, case, page, (t % ps).expand(case["batch"], 1, -1), see)


def _attend_pages(s, case, pages):
    ps, B, Hk = case["ps"], case["batch"], case["Hk"]
    i = torch.arange(pages.shape[-1] * ps, device="cuda")
    at = pages.long()[..., i // ps]                                # [B, Hk, k * ps]
    see = (at >= 0) & (at * ps + i % ps < s["kv_lens"].long()[:, None, None])
    page = torch.gather(s["table"].long()[:, None].expand(B, Hk, -1), 2, at.clamp(min=0)).clamp(min=0)
    return _attend(s, case, page, (i % ps).expand(B, Hk, -1), see)


# ----------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "tables":
        old, new = _steps(case)
        ps = case["ps"]
        rows = sum(max(0, n) for n in new)
        now = [max(0, a + n) for a, n in zip(old, new)]
        moved = sum(abs((b + ps - 1) // ps - (a + ps - 1) // ps) for a, b in zip(old, now))
        pages = sum((b + ps - 1) // ps for b in now) if case["csr"] else 0
        # lengths in and out, q_indptr; a page id read and written; a row's request, position and slot
        return dict(bytes=16 * len(old) + 8 * moved + 16 * rows + 8 * pages + (8 * len(old) if case["csr"] else 0),
                    flops=rows * 4 + len(old) * 8)
    d, Hk, ps = case["d"], case["Hk"], case["ps"]
    code = {"16bit": 2 * d, "scaled": d, "block": d + 1}.get(case.get("fmt"), 0)
    if case["op"] == "bounds":
        r = random.Random(case["lens"])
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
        kv = [r.randint(n, max(n, case["kv_hi"])) for n in new]
        keys = sum(b - (b - n) // ps * ps for n, b in zip(new, kv))
        pages = sum((b + ps - 1) // ps - (b - n) // ps for n, b in zip(new, kv))
        return dict(bytes=keys * Hk * code + pages * Hk * 4 * d + 8 * sum(new), flops=keys * Hk * d * 2)
    H, kv = case["H"], _lens(case)
    out = dict(bytes=0, flops=0.0)
    if case["op"] in ("select", "sparse"):
        pages = sum((x + ps - 1) // ps for x in kv)
        kept = sum(min(case["pages"], (x + ps - 1) // ps) for x in kv)
        out["bytes"] += pages * (Hk * 4 * d + 4) + case["batch"] * (H * d * 2 + Hk * case["pages"] * 4)
        out["flops"] += pages * Hk * 4.0 * d
        kv = [min(x, case["pages"] * ps) for x in kv]
        if case["op"] == "select":
            return out
        out["bytes"] += kept * 4
    elif case["window"] >= 0:
        kv = [min(x, case["window"] + 1) for x in kv]
    out["bytes"] += sum(kv) * 2 * Hk * code + case["batch"] * H * (4 * d + 4) + sum(kv) // ps * 4
    out["flops"] += 4.0 * d * H * sum(kv)
    return out


# ----------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _tables_one_by_one(s, case)
    wide = torch.float64
    if case["op"] == "bounds":
        return _bounds_64(s, case)
    kv_len, ps, Hk, d, H = _lens(case), case["ps"], case["Hk"], case["d"], case["H"]
    G = H // Hk
    table = s["table"].cpu().numpy()
    if case["op"] in ("select", "sparse"):
        pages = _select_64(s, case, table, kv_len)
        if case["op"] == "select":
            return pages
    out = torch.zeros((case["batch"], H, d), dtype=wide, device="cuda")
    lse = torch.full((case["batch"], H), -math.inf, dtype=wide, device="cuda")
    for r, n in enumerate(kv_len):
        for h in range(Hk):
            if case["op"] == "sparse":
                chosen = [p for p in pages[r, h].tolist() if p >= 0]
                t = np.concatenate([np.arange(p * ps, min(n, (p + 1) * ps)) for p in chosen] or [np.zeros(0, int)])
            else:
                t = np.arange(max(0, n - 1 - case["window"]) if case["window"] >= 0 else 0, n)
            if t.size == 0:
                continue
            page = torch.from_numpy(table[r][t // ps].astype(np.int64)).cuda()
            slot = torch.from_numpy(t % ps).cuda()
            k, v = (_head_64(s, case, page, half, slot, h) for half in (0, 1))
            x = s["q"][r, h * G:(h + 1) * G].double() @ k.T * s["scale"]
            out[r, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
            lse[r, h * G:(h + 1) * G] = torch.logsumexp(x, -1) / math.log(2.0)
    return (out, lse) if case["op"] == "decode" else (pages, out, lse)


def _head_64(s, case, page, half, slot, h):
    raw = s["kv"].view(torch.uint8) if s["kv"].dtype.itemsize == 1 else s["kv"]
    at = (page, half, slot, h) if case["layout"] == "NHD" else (page, half, h, slot)
    x = raw[at]
    x = (x.view(s["kv"].dtype) if s["kv"].dtype.itemsize == 1 else x).double()
    if case["fmt"] == "scaled":
        return x * (V_SCALE if half else K_SCALE)
    return x * torch.exp2(s["scales"][at].double() - 127)[:, None] if case["fmt"] == "block" else x


def _select_64(s, case, table, kv_len):
    """Request by request, head by head: scores in 64 bits on the host, pages by (score, position)."""
    ps, Hk, k = case["ps"], case["Hk"], case["pages"]
    G = case["H"] // Hk
    out = np.full((case["batch"], Hk, k), -1, dtype=np.int32)
    for r, length in enumerate(kv_len):
        n = -(-length // ps)
        if n == 0:
            continue
        at = torch.from_numpy(table[r, :n].astype(np.int64)).cuda()
        b = s["bounds"][at].double()
        q = s["q"][r].double()
        for h in range(Hk):
            total = torch.zeros(n, dtype=torch.float64, device="cuda")
            for g in range(G):
                x = q[h * G + g]
                total += torch.maximum(x * b[:, h, 0], x * b[:, h, 1]).sum(-1)
            score = total.cpu().numpy()
            must = set(range(min(case["first"], n))) | set(range(max(0, n - case["last"]), n))
            rest = [i for i in np.lexsort((np.arange(n), -score)).tolist() if i not in must]
            got = sorted((sorted(must) + rest)[:k])
            out[r, h, :len(got)] = got
    return torch.from_numpy(out).cuda()


def _bounds_64(s, case):
    """Outward rounding as numbers: a multiple of the step at each value's binade."""
    ps, Hk, d = case["ps"], case["Hk"], case["d"]
    dt = s["bounds"].dtype
    slots = s["slots"].cpu().numpy()
    last = {}
    for x in slots.tolist():
        last[x // ps] = max(last.get(x // ps, 0), x % ps)
    out = s["bounds"].double()
    bits, low = (8, -126) if dt == torch.bfloat16 else (11, -14)

    def step_of(x):
        _, e = torch.frexp(x.abs())
        return torch.exp2((e.double() - 1).clamp(min=low) - (bits - 1))

    for count in sorted(set(last.values())):
        page = torch.tensor([p for p, c in last.items() if c == count], device="cuda")
        slot = torch.arange(count + 1, device="cuda")
        for h in range(Hk):
            k = _head_64(s, case, page.repeat_interleave(count + 1), 0, slot.repeat(page.numel()), h)
            k = k.view(page.numel(), count + 1, d)
            lo, hi = k.min(1).values, k.max(1).values
            big = torch.finfo(dt).max
            out[page, h, 0] = (torch.floor(lo / step_of(lo)) * step_of(lo)).clamp(-big, big)
            out[page, h, 1] = (torch.ceil(hi / step_of(hi)) * step_of(hi)).clamp(-big, big)
    return out


def _tables_one_by_one(s, case):
    """The step as a host loop over the requests."""
    ps = case["ps"]
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy().copy()
    old, new = _steps(case)
    top = int(s["free_count"].item())
    now = [max(0, a + n) for a, n in zip(old, new)]
    had, has = ([-(-x // ps) for x in y] for y in (old, now))
    for r in range(len(old)):
        for p in range(has[r], had[r]):
            free[top] = table[r, p]
            top += 1
    for r in range(len(old)):
        for p in range(had[r], has[r]):
            top -= 1
            table[r, p] = free[top]
    req, pos, slots, indptr = [], [], [], [0]
    for r, n in enumerate(new):
        for t in range(old[r], old[r] + max(0, n)):
            req.append(r)
            pos.append(t)
            slots.append(int(table[r, t // ps]) * ps + t % ps)
        indptr.append(len(req))
    pad = s["max_rows"] - len(req)

    def ints(x, dtype=torch.int32):
        return torch.tensor(np.asarray(x), device="cuda").to(dtype)

    out = dict(table=ints(table), free=ints(free), free_count=ints([top]), kv_lens=ints(now), q_indptr=ints(indptr),
               requests=ints(req + [-1] * pad), positions=ints(pos + [0] * pad),
               slots=ints(slots + [-1] * pad, torch.int64))
    if case["csr"]:
        flat = [int(x) for r in range(len(old)) for x in table[r, :has[r]]]
        out.update(kv_indptr=ints(np.concatenate([[0], np.cumsum(has)])),
                   kv_indices=ints(flat + [-1] * (s["max_pages"] - len(flat))),
                   last_page_len=ints([(x - 1) % ps + 1 if x else 0 for x in now]))
    return out
