"""Measured cases of the paged K/V cache operators.

A batch of sequences of different lengths keeps its keys and values in pages of
a shared pool.  Four operators serve it, in the order a program calls them:

  page_table       lengths -> block table, pages taken from a list of free ones
  slot_map         positions of the recomputed rows -> packed rows and their cache slots
  paged_write      fp32 QKV rows -> RoPE -> query rows, K and V rows in their slots
  paged_attention  packed query rows over all cached keys of their sequence
                   (one row a sequence is the single-token form)

``own`` selects the library's kernels; otherwise ``run`` computes the same
results with elementary torch operations.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
THETA = 10000.0

# (query heads, kv heads, head dim)
HEADS = [(32, 32, 128), (28, 4, 128), (4, 4, 64), (8, 2, 80), (12, 3, 48), (16, 1, 256), (6, 6, 16), (10, 2, 112)]


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a batch of four long sequences gets its pages: the smallest call, all latency
        dict(name="table 4x2048", op="page_table", batch=4, lo=2048, hi=2048, page=64, max_pages=32, pool=1.0),
        # a server admits two thousand requests of 1 .. 16384 positions in small pages
        dict(name="table 2000 ragged", op="page_table", batch=2000, lo=1, hi=16384, page=16, max_pages=1024, pool=0.9),
        # the recompute set of one layer of one sequence: 32 budgeted rows and a 33-wide window
        dict(name="slots 65 of 1024", op="slot_map", batch=1, lo=1024, hi=1024, rows_lo=65, rows_hi=65, page=64,
             given=True),
        # the recompute sets of a full server: 500 sequences, up to 160 rows each, some with none
        dict(name="slots 500 ragged", op="slot_map", batch=500, lo=200, hi=16384, rows_lo=0, rows_hi=160, page=16,
             given=True),
        # the QKV product of those 65 rows of a 32-head model into its pages
        dict(name="write 65 rows 32x128", op="paged_write", batch=1, lo=1024, hi=1024, rows_lo=65, rows_hi=65,
             page=64, heads=32, kv=32, dim=128, dtype="bf16", layout="slot"),
        # four prompts written at once, grouped heads, pages stored head by head
        dict(name="write 4x1537 rows 28/4", op="paged_write", batch=4, lo=2000, hi=2048, rows_lo=1537, rows_hi=1537,
             page=16, heads=28, kv=4, dim=128, dtype="bf16", layout="head"),
        # the small fp32 model, a few sequences
        dict(name="write f32 4x64", op="paged_write", batch=7, lo=100, hi=256, rows_lo=0, rows_hi=33, page=16,
             heads=4, kv=4, dim=64, dtype="f32", layout="slot"),
        # the small fp32 model: 33 recomputed rows over 256 keys
        dict(name="attn f32 4x64 n256", op="paged_attention", batch=1, lo=256, hi=256, rows_lo=33, rows_hi=33, page=16,
             heads=4, kv=4, dim=64, dtype="f32", layout="slot"),
        # one layer of a denoising step: 65 recomputed rows over 1024 keys
        dict(name="attn 32x128 65 rows n1024", op="paged_attention", batch=1, lo=1024, hi=1024, rows_lo=65, rows_hi=65,
             page=64, heads=32, kv=32, dim=128, dtype="bf16", layout="slot"),
        # the long-context step: 161 recomputed rows over 8192 keys
        dict(name="attn 32x128 161 rows n8192", op="paged_attention", batch=1, lo=8192, hi=8192, rows_lo=161,
             rows_hi=161, page=64, heads=32, kv=32, dim=128, dtype="bf16", layout="head"),
        # one new token over one very long cache, grouped heads
        dict(name="attn 28/4 1 row n131072", op="paged_attention", batch=1, lo=131072, hi=131072, rows_lo=1, rows_hi=1,
             page=128, heads=28, kv=4, dim=128, dtype="bf16", layout="slot"),
        # one new token for each of 64 sequences of very different lengths, one of them empty
        dict(name="attn 28/4 64 ragged tokens", op="paged_attention", batch=64, lo=0, hi=16384, rows_lo=1, rows_hi=1,
             page=16, heads=28, kv=4, dim=128, dtype="bf16", layout="slot"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["op"], {"bytes": 0, "flops": 0, "plain": 0})
        t["bytes"], t["flops"] = max(t["bytes"], w["bytes"]), max(t["flops"], w["flops"])
        t["plain"] = max(t["plain"], _plain_bytes(c))
    op = rng.choice(["page_table", "slot_map", "paged_write", "paged_attention", "paged_attention"])
    while True:
        page = rng.choice([1, 5, 16, 16, 32, 64, 128, 100, 256])
        if op == "page_table":
            hi = _log_int(rng, 1, 16384)
            c = dict(op=op, batch=_log_int(rng, 1, 4000), lo=rng.choice([0, 1, max(1, hi // 2), hi]), hi=hi, page=page,
                     max_pages=-(-hi // page) + rng.choice([0, 0, 3, 17]), pool=rng.choice([0.5, 1.0, 1.1]))
            if c["pool"] < 1.0 and c["batch"] < 8:
                c["pool"] = 1.0
        elif op == "slot_map":
            hi = _log_int(rng, 1, 16384)
            rows = min(_log_int(rng, 1, 300), hi)
            c = dict(op=op, batch=_log_int(rng, 1, 1000), lo=max(1, hi // rng.choice([1, 2, 50])), hi=hi,
                     rows_lo=rng.choice([0, 1, rows]), rows_hi=rows, page=page, given=rng.random() < 0.7)
        else:
            H, KV, D = rng.choice(HEADS)
            dtype = rng.choice(["bf16", "bf16", "f32"])
            batch = _log_int(rng, 1, 256)
            hi = _log_int(rng, 1, 131072 if batch < 4 else 16384)
            rows = 1 if rng.random() < 0.4 and op == "paged_attention" else min(_log_int(rng, 1, 400), hi)
            c = dict(op=op, batch=batch, lo=rng.choice([0 if op == "paged_attention" else 1, max(1, hi // 3), hi]),
                     hi=hi, rows_lo=rng.choice([0, 1, rows]) if rows > 1 else 1, rows_hi=rows, page=page, heads=H,
                     kv=KV, dim=D, dtype=dtype, layout=rng.choice(["slot", "head"]))
        w, t = work(c), top[op]
        if w["bytes"] <= t["bytes"] and w["flops"] <= t["flops"] and _plain_bytes(c) <= t["plain"]:
            return c


def _lens(case):
    """(lengths, rows) of the sequences: set by the case alone, so that its work is known."""
    r = random.Random("%s-%d-%d-%d" % (case["op"], case["batch"], case["lo"], case["hi"]))
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    if case["op"] == "paged_attention" and case["batch"] > 8:
        lens[case["batch"] // 3] = case["lo"]
        lens[case["batch"] // 2] = case["hi"]
    if case["op"] == "page_table":
        return lens, None
    limit = (lambda n: case["rows_hi"]) if case["op"] == "paged_attention" else (lambda n: min(n, case["rows_hi"]))
    rows = [min(r.randint(case["rows_lo"], case["rows_hi"]), limit(n)) for n in lens]
    if not any(n and k for n, k in zip(lens, rows)):
        lens[0], rows[0] = max(lens[0], 1), max(rows[0], 1)
    return lens, rows


def _pages(n, page):
    return -(-n // page)


def _plain_bytes(case):
    """Values that the plain form of a case holds at once (its rows and keys are padded to the longest)."""
    if case["op"] != "paged_attention":
        return work(case)["bytes"]
    lens, rows = _lens(case)
    n = max(1, max(lens))
    return case["batch"] * n * (2 * case["kv"] * case["dim"] + 2 * max(rows) * case["heads"])


def work(case):
    lens, rows = _lens(case)
    B, page = case["batch"], case["page"]
    if case["op"] == "page_table":
        taken = sum(_pages(n, page) for n in lens)
        return {"bytes": 4.0 * (2 * B + B * case["max_pages"] + min(1.0, case["pool"]) * taken), "flops": 0.0}
    T = sum(rows)
    if case["op"] == "slot_map":
        return {"bytes": 4.0 * (2 * B + 1 + (2 + 1 + (1 if case["given"] else 0)) * T), "flops": 0.0}
    H, KV, D, e = case["heads"], case["kv"], case["dim"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "paged_write":
        return {"bytes": float(T * (H + 2 * KV) * D * (4 + e) + T * (4 * D + 8)), "flops": float(T * (H + KV) * D * 3)}
    keys = sum(n for n, r in zip(lens, rows) if r)
    pairs = sum(n * r for n, r in zip(lens, rows))
    return {"bytes": float(2 * keys * KV * D * e + 2 * T * H * D * e + 4 * sum(_pages(n, page) for n in lens)),
            "flops": float(4 * pairs * H * D)}


# ------------------------------------------------------------------ inputs

class State:
    pass


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    lens, rows = _lens(case)
    s = State()
    s.op, s.page = case["op"], case["page"]
    B, page = case["batch"], case["page"]
    i32 = dict(dtype=torch.int32, device="cuda")
    need = [_pages(n, page) for n in lens]
    s.lens = torch.tensor(lens, **i32)
    if s.op == "page_table":
        # the free list: page ids in the order the pool gives them out; short of what is asked where pool < 1
        s.max_pages = case["max_pages"]
        n = max(1, int(case["pool"] * sum(need)))
        s.n_pages = n + 61
        s.pool = torch.randperm(s.n_pages, generator=g, device="cuda")[:n].to(torch.int32)
        s.first = torch.zeros(1, **i32)
        return s
    s.n_pages = sum(need) + 3
    s.max_pages = max(1, max(need))
    order = torch.randperm(s.n_pages, generator=g, device="cuda").to(torch.int32)
    n_t = torch.tensor(need, device="cuda")
    start = torch.cumsum(n_t, 0) - n_t
    at = torch.arange(s.max_pages, device="cuda")
    s.table = torch.where(at < n_t[:, None], order[(start[:, None] + at).clamp(max=s.n_pages - 1)],
                          torch.full((), -1, **i32)).contiguous()
    s.count = torch.tensor(rows, **i32)
    s.T, s.R = sum(rows), max(rows)
    s.row_start = torch.tensor([0] + list(np.cumsum(rows)), **i32)
    if s.op == "slot_map":
        # distinct ascending positions of each sequence, as the token selection gives them, or a first position
        s.pos, s.first = None, None
        if case["given"]:
            pos = np.zeros((B, max(lens)), np.int32)
            r = np.random.default_rng(int(seed))
            for b, (n, k) in enumerate(zip(lens, rows)):
                pos[b, :k] = np.sort(r.choice(n, k, replace=False))
            s.pos = torch.from_numpy(pos).cuda()
        else:
            s.first = ((s.lens - s.count).double() * torch.rand(B, generator=g, device="cuda").double()).to(torch.int32)
        return s
    H, KV, D, dt = case["heads"], case["kv"], case["dim"], DTYPES[case["dtype"]]
    s.H, s.KV, s.D, s.dt = H, KV, D, dt
    if s.op == "paged_write":
        # the QKV product in fp32, the rows' positions (the last of each sequence) and slots, pages with older content
        s.qkv = torch.randn((s.T, (H + 2 * KV) * D), generator=g, device="cuda")
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), s.count.long(), output_size=s.T)
        j = torch.arange(s.T, device="cuda") - s.row_start.long()[seq]
        pos = (s.lens - s.count).long()[seq] + j
        s.row_pos = pos.to(torch.int32)
        s.slot = (s.table.long()[seq, pos // page] * page + pos % page).to(torch.int32)
        angle = (torch.arange(max(lens), device="cuda", dtype=torch.float64)[:, None]
                 * THETA ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) * 2 / D))
        s.rope = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
    shape = (s.n_pages, page, KV, D) if case["layout"] == "slot" else (s.n_pages, KV, page, D)
    make = lambda: torch.randn(shape, generator=g, device="cuda", dtype=dt)  # noqa: E731
    k, v = make(), make()
    s.k, s.v = (k, v) if case["layout"] == "slot" else (k.transpose(1, 2), v.transpose(1, 2))
    if s.op == "paged_attention":
        s.q = torch.randn((s.T, H, D), generator=g, device="cuda", dtype=dt) * 1.5
        s.L = max(1, max(lens))
        # what no sequence covers holds whatever was there before: free pages and the ends of last pages
        used = torch.zeros((s.n_pages, page), dtype=torch.bool, device="cuda")
        for b in range(B):
            if need[b]:
                used[s.table[b, :need[b]].long()] = True
                used[s.table[b, need[b] - 1].long(), lens[b] - (need[b] - 1) * page:] = False
        s.k[~used] = float("nan")
        s.v[~used] = float("nan")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"page_table": _plain_table, "slot_map": _plain_slots, "paged_write": _plain_write,
            "paged_attention": _plain_attention}[s.op](s)


def _run_own(s):
    from dynamic_layer_wise_b200 import dcu
    if s.op == "page_table":
        table, held, nxt = dcu.dcu_page_table(s.lens, s.page, s.max_pages, s.n_pages, pool=s.pool, first=s.first)
        return {"table": table, "held": held, "next": nxt}
    if s.op == "slot_map":
        row_start, row_pos, slot = dcu.dcu_slot_map(s.table, s.count, s.page, s.n_pages, s.T, pos=s.pos, first=s.first)
        return {"row_start": row_start, "row_pos": row_pos, "slot": slot}
    if s.op == "paged_write":
        q = dcu.dcu_paged_write(s.qkv, s.row_start, s.row_pos, s.slot, s.rope, s.k, s.v, s.H)
        return {"q": q, "k": s.k, "v": s.v}
    return dcu.dcu_paged_attention(s.q, s.row_start, s.lens, s.table, s.k, s.v)


def _plain_table(s):
    need = (s.lens.clamp(min=0).long() + (s.page - 1)) // s.page
    need = torch.where(need <= s.max_pages, need, 0)
    end = torch.cumsum(need, 0)
    first = s.first.long()
    fits = first + end <= s.pool.numel()
    held = torch.where(fits, need, 0)
    at = torch.arange(s.max_pages, device=need.device)
    src = (first + (end - need)[:, None] + at).clamp(max=s.pool.numel() - 1)
    table = torch.where(at < held[:, None], s.pool[src].long(), -1)
    nxt = first + torch.where(fits, end, 0).amax()
    return {"table": table.to(torch.int32), "held": held.to(torch.int32), "next": nxt.to(torch.int32)}


def _plain_slots(s):
    end = torch.cumsum(s.count.long(), 0)
    row_start = torch.nn.functional.pad(end, (1, 0))
    t = torch.arange(s.T, device=end.device)
    seq = torch.searchsorted(end, t, right=True)
    j = t - row_start[seq]
    pos = s.pos[seq, j].long() if s.pos is not None else s.first.long()[seq] + j
    slot = s.table[seq, pos // s.page].long() * s.page + pos % s.page
    return {"row_start": row_start.to(torch.int32), "row_pos": pos.to(torch.int32), "slot": slot.to(torch.int32)}


def _plain_write(s):
    T, H, KV, D = s.T, s.H, s.KV, s.D
    x = s.qkv.view(T, H + 2 * KV, D)
    cos, sin = s.rope[s.row_pos.long()].unbind(-1)
    a, b = x[:, :H + KV, :D // 2], x[:, :H + KV, D // 2:]
    c, d = cos[:, None], sin[:, None]
    r = torch.cat([a * c - b * d, b * c + a * d], -1).to(s.dt)
    page, off = s.slot.long() // s.page, s.slot.long() % s.page
    s.k[page, off] = r[:, H:]
    s.v[page, off] = x[:, H + KV:].to(s.dt)
    return {"q": r[:, :H].contiguous(), "k": s.k, "v": s.v}


def _plain_attention(s):
    B, R, L, H, KV, D = s.lens.numel(), s.R, s.L, s.H, s.KV, s.D
    row = s.row_start[:-1, None].long() + torch.arange(R, device="cuda")
    q = s.q[row.clamp(max=s.T - 1)].float().view(B, R, KV, H // KV, D).permute(0, 2, 1, 3, 4).reshape(B, KV, -1, D)
    at = torch.arange(L, device="cuda")
    valid = at < s.lens[:, None]
    page = s.table[:, at // s.page].clamp(min=0).long()
    keep = valid[:, :, None, None]
    k = torch.where(keep, s.k[page, at % s.page].float(), 0.0).permute(0, 2, 1, 3)
    x = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    del k
    x = x.masked_fill(~valid[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = torch.exp(x - m)
    del x
    v = torch.where(keep, s.v[page, at % s.page].float(), 0.0).permute(0, 2, 1, 3)
    o = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.view(B, KV, R, H // KV, D).permute(0, 2, 1, 3, 4).reshape(B, R, H, D)
    t = torch.arange(s.T, device="cuda")
    seq = torch.searchsorted(s.row_start[1:].long(), t, right=True)
    return o[seq, t - s.row_start[seq]].to(s.dt)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    if case["op"] in ("page_table", "slot_map"):
        return None  # whole numbers only
    s = prepare(case, seed)
    if s.op == "paged_write":
        x = s.qkv.double().cpu().numpy().reshape(s.T, s.H + 2 * s.KV, s.D)
        half = s.D // 2
        freq = THETA ** (-2.0 * np.arange(half) / s.D)
        turn = np.exp(1j * s.row_pos.cpu().numpy().astype(np.float64)[:, None] * freq)
        z = (x[:, :s.H + s.KV, :half] + 1j * x[:, :s.H + s.KV, half:]) * turn[:, None, :]
        qk = torch.from_numpy(np.concatenate([z.real, z.imag], -1))
        k, v = s.k.double().cpu(), s.v.double().cpu()
        for t, at in enumerate(s.slot.tolist()):
            k[at // s.page, at % s.page] = qk[t, s.H:]
            v[at // s.page, at % s.page] = torch.from_numpy(x[t, s.H + s.KV:])
        return {"q": qk[:, :s.H], "k": k, "v": v}
    out = torch.zeros((s.T, s.H, s.D), dtype=torch.float64, device="cuda")
    starts, lens = s.row_start.tolist(), s.lens.tolist()
    for b, n in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi or n == 0:
            continue
        pages = s.table[b, :_pages(n, s.page)].long()
        k = s.k[pages].reshape(-1, s.KV, s.D)[:n].double()
        v = s.v[pages].reshape(-1, s.KV, s.D)[:n].double()
        for h in range(s.H):
            kv = h // (s.H // s.KV)
            w = torch.softmax(s.q[lo:hi, h].double() @ k[:, kv].T / math.sqrt(s.D), -1)
            out[lo:hi, h] = w @ v[:, kv]
    return out
