"""The paged K/V cache operators against plain numpy forms: whole numbers exactly, numbers within
bounds derived in paged_ref from the roundings that the kernels make."""
import numpy as np
import pytest
import torch

import oracle as O
from dynamic_layer_wise_b200 import dcu
from tests import paged_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# rounding of the softmax weights before P V: bf16 high + low parts, or one bf16 (half a step: 2^-8) on the tensor-core
# path for many queries
P_STEP = {"bf16": 2.0 ** -16, "f32": 0.0}
P_STEP_TC = 2.0 ** -8


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ block table

TABLES = [  # lens, page, max_pages, spare pages (negative: short)
    ([1], 16, 1, 0), ([0], 16, 3, 0), ([-5, 7, 0, 33], 16, 4, 2), ([2048] * 4, 64, 32, 0),
    ([100, 3000, 17, 9], 16, 20, 5), ([5] * 9, 1, 7, -8), ([64, 64, 64], 64, 2, -1), ([2 ** 31 - 1, 16], 16, 4, 3),
    (list(range(700)), 7, 120, 11), (list(range(1300, 0, -1)), 5, 300, -400), ([9000, 1, 70000], 2, 40000, 1),
]


@pytest.mark.parametrize("case", range(len(TABLES)))
@pytest.mark.parametrize("mode", ["identity", "pool", "first"])
def test_page_table(case, mode):
    lens, page, max_pages, spare = TABLES[case]
    rng = np.random.default_rng(case)
    total = sum(n for n in (-(-max(x, 0) // page) for x in lens) if n <= max_pages)
    n_pool = max(0, total + spare)
    first, pool, n_pages = 0, None, max(1, n_pool)
    if mode != "identity":
        n_pages = n_pool + 40
        pool = rng.permutation(n_pages)[:n_pool].astype(np.int32)
        if n_pool > 3:
            pool[n_pool // 2] = n_pages  # an entry outside the pool
            pool[0] = -1
    elif n_pool == 0:
        pytest.skip("a pool has at least one page")
    if mode == "first":
        first = min(3, n_pool)
    st = status_word()
    table, held, nxt = dcu.dcu_page_table(i32(lens), page, max_pages, n_pages, None if pool is None else i32(pool),
                                          i32([first]) if mode == "first" else None, st)
    w_table, w_held, w_next, w_status = R.page_table(lens, page, max_pages, n_pages, pool, first)
    assert np.array_equal(table.cpu().numpy(), w_table)
    assert np.array_equal(held.cpu().numpy(), w_held)
    assert nxt.item() == w_next and st.item() == w_status


def test_page_table_chains_calls_on_one_pool():
    pool = np.random.default_rng(0).permutation(50).astype(np.int32)
    t0, h0, n0 = dcu.dcu_page_table(i32([100, 33]), 16, 8, 50, i32(pool))
    t1, h1, n1 = dcu.dcu_page_table(i32([64, 200]), 16, 20, 50, i32(pool), n0)
    got = [p for t in (t0, t1) for p in t.cpu().numpy().ravel() if p >= 0]
    assert got == list(pool[:7 + 3 + 4 + 13]) and n1.item() == 27


@pytest.mark.parametrize("first", [-1, 9, 2 ** 31 - 1])
def test_page_table_first_outside_the_pool_serves_nothing(first):
    st = status_word()
    table, held, nxt = dcu.dcu_page_table(i32([5, 0]), 16, 2, 8, None, i32([first]), st)
    assert (table == -1).all() and (held == 0).all() and nxt.item() == first and st.item() == R.NO_PAGE


# ------------------------------------------------------------------ slot map

def make_table(rng, lens, page, spare=3):
    need = [-(-int(n) // page) for n in lens]
    n_pages = sum(need) + spare
    order, at = rng.permutation(n_pages), 0
    table = np.full((len(lens), max(1, max(need))), -1, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


MAPS = [(1, 1, 1, 1), (1, 1024, 65, 64), (3, 50, 50, 16), (5, 40, 7, 1), (64, 300, 20, 7), (700, 90, 9, 16),
        (1025, 30, 3, 5), (2100, 12, 2, 128), (2, 20000, 4000, 100)]


@pytest.mark.parametrize("B,N,rows,page", MAPS)
@pytest.mark.parametrize("given", [True, False])
def test_slot_map(B, N, rows, page, given):
    rng = np.random.default_rng(B + N)
    lens = rng.integers(1, N + 1, B)
    count = np.array([rng.integers(0, min(rows, n) + 1) for n in lens])
    count[rng.integers(B)] = min(rows, lens.min())
    table, n_pages = make_table(rng, lens, page)
    pos = first = None
    if given:
        pos = rng.integers(-9, 9, (B, N)).astype(np.int32)  # what is past the count is not looked at
        for b in range(B):
            pos[b, :count[b]] = np.sort(rng.choice(lens[b], count[b], replace=False))
    else:
        first = np.array([rng.integers(0, n - k + 1) for n, k in zip(lens, count)])
    T = int(count.sum()) + 9
    st = status_word()
    start, rp, sl = dcu.dcu_slot_map(i32(table), i32(count), page, n_pages, T, None if pos is None else i32(pos),
                                     None if first is None else i32(first), st)
    w = R.slot_map(table, count, page, n_pages, T, pos, first)
    n = T - 9
    assert np.array_equal(start.cpu().numpy(), w[0])
    assert np.array_equal(rp.cpu().numpy()[:n], w[1]) and np.array_equal(sl.cpu().numpy()[:n], w[2])
    assert st.item() == w[3] == 0


def test_slot_map_bad_rows():
    """Uncovered positions, negative counts, counts above the row length, repeats, and more rows than fit."""
    table = np.array([[4, -1, 7], [99, 2, -3], [0, 1, 3]], np.int32)
    pos = np.array([[0, 17, 33, 48, 50], [3, 16, 40, 41, 60], [5, 5, 4, 9, 10]], np.int32)
    for count, cap in (([5, 5, 5], 15), ([5, -2, 7], 12), ([2, 0, 3], 9), ([5, 5, 5], 8), ([5, 5, 5], 0)):
        st = status_word()
        args = (i32(table), i32(count), 16, 8, cap, i32(pos), None, st)
        start, rp, sl = dcu.dcu_slot_map(*args)
        w = R.slot_map(table, count, 16, 8, cap, pos)
        n = len(w[1])
        assert np.array_equal(start.cpu().numpy(), w[0]) and st.item() == w[3]
        assert np.array_equal(rp.cpu().numpy()[:n], w[1]) and np.array_equal(sl.cpu().numpy()[:n], w[2])
    st = status_word()
    _, rp, sl = dcu.dcu_slot_map(i32(table), i32([2, 2, 2]), 16, 8, 6, None, i32([2 ** 31 - 1, -1, 47]), st)
    assert sl.cpu().tolist() == [-1, -1, -1, -1, 3 * 16 + 15, -1] and st.item() == R.BAD_PAGE


def test_slot_map_leaves_rows_behind_the_last_sequence():
    table, n_pages = make_table(np.random.default_rng(0), [40, 40], 16)
    t, c = i32(table), i32([3, 4])
    start, rp, sl = (torch.full((n,), -77, dtype=torch.int32, device="cuda") for n in (3, 600, 600))
    rc = dcu.lib().dcu_slot_map(t.data_ptr(), 2, table.shape[1], 16, n_pages, c.data_ptr(), None, 0, None, 600,
                                start.data_ptr(), rp.data_ptr(), sl.data_ptr(), None,
                                torch.cuda.current_stream().cuda_stream)
    assert rc == dcu.DCU_OK and start.cpu().tolist() == [0, 3, 7]
    assert (rp[7:] == -77).all() and (sl[7:] == -77).all() and (sl[:7] >= 0).all()


# ------------------------------------------------------------------ RoPE + K/V write

def make_pages(rng_seed, n_pages, page, KV, hd, dtype, layout, fill=None):
    g = torch.Generator(device="cuda").manual_seed(rng_seed)
    shape = (n_pages, KV, page, hd) if layout == "head" else (n_pages, page, KV, hd)
    if layout == "mixed":  # K and V of a page side by side, padded heads
        both = torch.randn((n_pages, 2, page, KV, hd + 16), generator=g, device="cuda").to(dtype)
        return both[:, 0, :, :, :hd], both[:, 1, :, :, :hd]
    k, v = (torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2))
    return (k.transpose(1, 2), v.transpose(1, 2)) if layout == "head" else (k, v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,KV,hd,page,layout", [(32, 32, 128, 64, "slot"), (28, 4, 128, 16, "head"),
                                                 (4, 4, 64, 16, "mixed"), (1, 1, 16, 1, "slot"),
                                                 (6, 3, 80, 5, "head"), (3, 1, 256, 7, "slot"),
                                                 (40, 5, 48, 3, "mixed")])
@pytest.mark.parametrize("rope", [True, False])
def test_paged_write(dtype, H, KV, hd, page, layout, rope):
    rng = np.random.default_rng(H + hd)
    T, used, n_pages, max_pos = 23, 19, 9 + 60 // page, 5000
    k, v = make_pages(5, n_pages, page, KV, hd, DT[dtype], layout)
    k0, v0 = k.clone(), v.clone()
    qkv = rng.standard_normal((T, (H + 2 * KV) * hd)).astype(np.float32)
    slot = rng.permutation(n_pages * page)[:T].astype(np.int32)
    pos = rng.integers(0, max_pos, T).astype(np.int32)
    slot[3], slot[4], pos[6], pos[7] = -1, n_pages * page, -1, max_pos
    pos[8] = max_pos - 1
    tab = dcu.dcu_rope_table(max_pos, hd) if rope else None
    st = status_word()
    q = torch.full((T, H, hd), 7.0, dtype=DT[dtype], device="cuda")
    dcu.dcu_paged_write(torch.tensor(qkv).cuda(), i32([0, used]), i32(pos), i32(slot), tab, k, v, H, q=q, status=st)
    assert st.item() == R.BAD_PAGE | (R.BAD_ROW if rope else 0)
    x = qkv.astype(np.float64).reshape(T, H + 2 * KV, hd)
    lost = (6, 7) if rope else ()
    r = R.rotate(x[:, :H + KV], np.clip(pos, 0, None), 10000.0) if rope else x[:, :H + KV]
    r[list(lost)] = 0.0
    # |a cos - b sin|: the table's rounding (2^-24 of each factor), two products and a sum in fp32 (an fma at most
    # drops one rounding): 3 * 2^-24 (|a| + |b|) at most; then half a step of dtype
    mag = np.abs(x[:, :H + KV, :hd // 2]) + np.abs(x[:, :H + KV, hd // 2:])
    tol = (3 * 2.0 ** -24 if rope else 0.0) * np.concatenate([mag, mag], -1)
    half = torch.finfo(DT[dtype]).eps / 2 if dtype == "bf16" or rope else 0.0
    check = lambda got, want, t: np.all(np.abs(got - want) <= t * (1 + half) + half * np.abs(want))  # noqa: E731
    assert check(f64(q[:used]), r[:used, :H], tol[:used, :H])
    assert (q[used:] == 7.0).all()
    wk, wv, tk = f64(k0), f64(v0), np.zeros_like(f64(k0))
    touched = np.zeros((n_pages, page), bool)
    half_v = torch.finfo(DT[dtype]).eps / 2 if dtype == "bf16" else 0.0
    for t in range(used):
        if t in (3, 4) + lost:
            continue
        at = slot[t] // page, slot[t] % page
        wk[at], wv[at], tk[at], touched[at] = r[t, H:], x[t, H + KV:], tol[t, H:], True
    assert check(f64(k)[touched], wk[touched], tk[touched])
    assert np.all(np.abs(f64(v) - wv)[touched] <= half_v * np.abs(wv)[touched])
    assert np.array_equal(f64(k)[~touched], f64(k0)[~touched]) and np.array_equal(f64(v)[~touched], f64(v0)[~touched])


def test_rope_table_far_positions():
    """Angles of positions near 10^6 keep their 24 bits."""
    n, hd = 1000001, 32
    tab = f64(dcu.dcu_rope_table(n, hd, 500000.0)[-3:])
    ang = np.arange(n - 3, n)[:, None] * 500000.0 ** (-2.0 * np.arange(hd // 2) / hd)
    want = np.stack([np.cos(ang), np.sin(ang)], -1)
    # fp64 angle: 10^6 * 2^-53 * a few; fp32 rounding of a value up to 1: 2^-25
    assert np.max(np.abs(tab - want)) <= 2.0 ** -25 + 1e-9


# ------------------------------------------------------------------ attention

def case_inputs(seed, dtype, H, KV, hd, page, layout, lens, rows, tail=2, q_scale=1.5):
    rng = np.random.default_rng(seed)
    table, n_pages = make_table(rng, [max(n, 1) for n in lens], page)
    k, v = make_pages(seed, n_pages, page, KV, hd, DT[dtype], layout)
    used = np.zeros((n_pages, page), bool)
    for b, n in enumerate(lens):
        at = np.arange(n)
        used[table[b, at // page], at % page] = True
    hole = torch.tensor(~used, device="cuda")
    k[hole], v[hole] = float("nan"), float("inf")  # free pages and the ends of last pages hold anything
    T = sum(rows)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (torch.randn((T + tail, H, hd), generator=g, device="cuda") * q_scale).to(DT[dtype])
    start = np.concatenate([[0], np.cumsum(rows)])
    return q, start, np.array(lens), table, k, v


def check_attention(got, q, start, lens, table, k, v, dtype, scale):
    hd = q.shape[-1]
    many = dtype == "bf16" and q.shape[0] * (q.shape[1] // k.shape[2]) > 8 * len(lens)
    p_step = P_STEP_TC if many else P_STEP[dtype]
    kn, vn = np.nan_to_num(f64(k), nan=0, posinf=0), np.nan_to_num(f64(v), nan=0, posinf=0)
    want, A, mag = R.attention(f64(q), start, lens, table, kn, vn, scale)
    tol = R.attention_bound(want, A, mag, DT[dtype], max(1, max(lens)), hd, p_step)
    n = int(start[-1])
    err = np.abs(f64(got)[:n] - want[:n])
    assert np.all(np.isfinite(f64(got)[:n]))
    worst = np.max(err / tol[:n]) if n else 0.0
    assert worst <= 1.0, f"error {worst:.2f} times its bound"


EDGE = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 257]
ATTN = [  # H, KV, hd, page, layout, lens, rows
    (4, 4, 64, 16, "slot", EDGE, [1] * len(EDGE)),
    (28, 4, 128, 16, "slot", EDGE, [1] * len(EDGE)),
    (32, 32, 128, 64, "head", [300], [65]),
    (28, 4, 128, 64, "mixed", [513, 70], [33, 9]),
    (8, 2, 80, 5, "slot", [40, 0, 333, 1], [3, 2, 0, 5]),
    (1, 1, 16, 1, "slot", [1], [1]),
    (6, 6, 16, 7, "head", [19, 100, 64], [8, 7, 16]),
    (12, 3, 48, 100, "slot", [1000, 99, 101], [1, 40, 2]),
    (16, 1, 256, 32, "slot", [700, 5], [3, 1]),
    (6, 3, 224, 3, "head", [77, 150], [30, 1]),
    (64, 1, 64, 16, "slot", [150], [2]),
    (4, 2, 112, 256, "mixed", [4000], [1]),
    (2, 1, 128, 16, "slot", [6000, 3], [1, 1]),
    (3, 3, 32, 16, "slot", [60] * 70, [2] * 70),
    (2, 2, 64, 16, "slot", [0] * 5, [1] * 5),
    (4, 4, 128, 128, "head", [600, 1100], [200, 129]),
    (8, 1, 128, 16, "slot", [1000, 129, 127, 1, 0, 128, 700], [40, 32, 17, 33, 50, 1, 64]),  # tiles of one and two halves
    (4, 2, 64, 32, "mixed", [3000, 40, 256], [300, 129, 128]),
    (2, 2, 112, 256, "slot", [513], [77]),
    (3, 3, 48, 64, "head", [5000, 64], [65, 256]),
    (28, 4, 128, 48, "slot", [200, 333], [65, 1]),
    (32, 32, 128, 64, "slot", [1024], [65]),
    (8, 1, 128, 16, "slot", [300, 0, 64, 65, 4000, 1, 500], [1, 17, 33, 48, 2, 16, 120]),  # queries in 1 .. 4 warps
    (2, 1, 64, 16, "head", [9000], [100]),
    (4, 2, 128, 5, "slot", [333, 70], [33, 20]),  # many queries on pages that do not hold whole blocks
    (5, 1, 64, 7, "mixed", [100, 0, 31], [9, 4, 2]),
    (14, 2, 256, 16, "head", [500, 20], [9, 3]),
    (4, 4, 208, 64, "slot", [1000, 65, 0, 130], [100, 20, 3, 128]),
    (16, 1, 144, 32, "mixed", [90, 3000], [1, 9]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_paged_attention(dtype, case):
    H, KV, hd, page, layout, lens, rows = ATTN[case]
    q, start, lens, table, k, v = case_inputs(case, dtype, H, KV, hd, page, layout, lens, rows)
    st = status_word()
    out = torch.full_like(q, 3.0)
    dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v, out=out, status=st)
    assert st.item() == 0
    assert (out[int(start[-1]):] == 3.0).all()  # rows behind the last sequence
    empty = [r for b, n in enumerate(lens) if n == 0 for r in range(start[b], start[b + 1])]
    assert (out[empty] == 0).all()
    check_attention(out, q, start, lens, table, k, v, dtype, hd ** -0.5)
    again = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v)
    assert torch.equal(again[:int(start[-1])], out[:int(start[-1])])  # equal inputs, equal bits


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_paged_attention_scales_and_peaked_scores(dtype, scale):
    q, start, lens, table, k, v = case_inputs(3, dtype, 4, 2, 64, 16, "slot", [250, 31], [5, 2], q_scale=4.0)
    out = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v, scale=scale)
    check_attention(out, q, start, lens, table, k, v, dtype, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_attention_growing_scores(dtype):
    """Scores that grow along the cache move the running maximum at every step."""
    q, start, lens, table, k, v = case_inputs(4, dtype, 2, 1, 64, 16, "slot", [2000], [9])
    at = np.arange(2000)
    k[i32(table[0, at // 16]).long(), i32(at % 16).long()] *= torch.linspace(0.01, 6, 2000, device="cuda")[:, None, None].to(k.dtype)
    out = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v)
    check_attention(out, q, start, lens, table, k, v, dtype, 64 ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_attention_bad_pages_and_lengths(dtype):
    """Keys on pages outside the pool, and lengths past the table row, are left out and flagged."""
    q, start, lens, table, k, v = case_inputs(6, dtype, 4, 2, 64, 16, "slot", [100, 60, 40, 30], [2, 1, 3, 1])
    n_pages = k.shape[0]
    bad = table.copy()
    bad[0, 2], bad[1, 0], bad[2, :] = n_pages, -7, 2 ** 31 - 1
    st = status_word()
    long = lens.copy()
    long[3] = -3
    out = dcu.dcu_paged_attention(q, i32(start), i32(long), i32(bad), k, v, status=st)
    assert st.item() == R.BAD_PAGE and (out[3:7] == 0).all()
    check_attention(out, q, start, np.maximum(long, 0), bad, k, v, dtype, 64 ** -0.5)
    full = np.full(4, table.shape[1] * 16)
    tab = np.where(table < 0, 0, table).astype(np.int32)
    k.nan_to_num_(0, 0), v.nan_to_num_(0, 0)
    st = status_word()
    ref = dcu.dcu_paged_attention(q, i32(start), i32(full), i32(tab), k, v, status=st)
    assert st.item() == 0
    for n in (full[0] + 1, 2 ** 31 - 1):
        st = status_word()
        out = dcu.dcu_paged_attention(q, i32(start), i32([n] * 4), i32(tab), k, v, status=st)
        assert st.item() == R.BAD_PAGE and torch.equal(out[:7], ref[:7])


@pytest.mark.parametrize("page,rows", [(16, [130, 9]), (32, [40, 33]), (64, [200, 1]), (16, [1, 1]), (5, [3, 40])])
def test_paged_attention_bad_pages_all_along(page, rows):
    """A fifth of the pages of long sequences is not there."""
    q, start, lens, table, k, v = case_inputs(60 + page, "bf16", 4, 2, 128, page, "head", [3001, 700], rows)
    rng = np.random.default_rng(page)
    bad = np.where((rng.random(table.shape) < 0.2) & (table >= 0), np.where(rng.random(table.shape) < 0.5, -1, 10 ** 9),
                   table).astype(np.int32)
    st = status_word()
    out = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(bad), k, v, status=st)
    assert st.item() == R.BAD_PAGE
    check_attention(out, q, start, lens, bad, k, v, "bf16", 128 ** -0.5)


@pytest.mark.parametrize("H,KV,hd,page,rows,n", [(4, 2, 64, 16, 20, 90), (8, 1, 128, 64, 17, 60), (2, 2, 256, 32, 30, 40)])
def test_paged_attention_many_items_in_a_range(H, KV, hd, page, rows, n):
    rng = np.random.default_rng(n)
    q, start, lens, table, k, v = case_inputs(70 + n, "bf16", H, KV, hd, page, "slot", list(rng.integers(0, 500, n)),
                                              list(rng.integers(0, 2 * rows, n)))
    out = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v)
    check_attention(out, q, start, lens, table, k, v, "bf16", hd ** -0.5)


@pytest.mark.parametrize("dtype,rows", [("bf16", 2), ("bf16", 90), ("f32", 9)])
@pytest.mark.parametrize("n", [40, 5000])
def test_paged_attention_keeps_a_bad_query_to_itself(dtype, rows, n):
    """NaN in a query makes its own output NaN, whether its keys are split or not, and no other."""
    q, start, lens, table, k, v = case_inputs(8, dtype, 4, 2, 64, 16, "slot", [n], [rows])
    call = lambda x: dcu.dcu_paged_attention(x, i32(start), i32(lens), i32(table), k, v)[:rows]
    ref = call(q)
    x = q.clone()
    x[rows // 2, 1, 5] = float("nan")
    out = call(x)
    hit = torch.zeros(rows, 4, 64, dtype=torch.bool, device="cuda")
    hit[rows // 2, 1] = True
    assert out[hit].isnan().all() and torch.equal(out[~hit], ref[~hit])


@pytest.mark.parametrize("H,KV,hd,page,layout,lens,rows", [
    (4, 2, 128, 8, "slot", [3001, 0, 63, 65], [130, 3, 9, 40]), (8, 1, 64, 8, "head", [700, 9], [20, 17]),
    (4, 4, 128, 24, "mixed", [500, 1, 129], [70, 33, 9]), (2, 2, 256, 40, "slot", [333, 64], [65, 20]),
    (28, 4, 128, 8, "slot", [2000, 31], [2, 30])])
def test_paged_attention_pages_of_eights(H, KV, hd, page, layout, lens, rows):
    q, start, lens, table, k, v = case_inputs(90 + page, "bf16", H, KV, hd, page, layout, lens, rows)
    st = status_word()
    out = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v, status=st)
    assert st.item() == 0
    check_attention(out, q, start, lens, table, k, v, "bf16", hd ** -0.5)
    bad = np.where((np.arange(table.shape[1]) % 5 == 3) & (table >= 0), -1, table).astype(np.int32)
    out = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(bad), k, v, status=st)
    check_attention(out, q, start, lens, bad, k, v, "bf16", hd ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,KV,hd,page,lens,rows", [(32, 32, 128, 16, [512], [65]), (4, 4, 64, 16, [256], [33]),
                                                    (8, 2, 128, 64, [250, 0, 1, 129], [1, 2, 1, 1]),
                                                    (4, 2, 256, 16, [60, 33], [40, 7]), (28, 4, 128, 8, [384], [1])])
def test_paged_attention_short_and_wide_tables(dtype, H, KV, hd, page, lens, rows):
    """What a table could hold decides whether items are cut; the keys there are decide the result."""
    q, start, lens, table, k, v = case_inputs(95, dtype, H, KV, hd, page, "slot", lens, rows)
    wide = np.full((len(lens), 5000), -1, np.int32)
    wide[:, :table.shape[1]] = table
    for tab in (table, wide):
        st = status_word()
        out = torch.full_like(q, 3.0)
        dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(tab), k, v, out=out, status=st)
        assert st.item() == 0 and (out[int(start[-1]):] == 3.0).all()
        check_attention(out, q, start, lens, tab, k, v, dtype, hd ** -0.5)


def test_paged_attention_row_starts_outside_the_rows():
    q, start, lens, table, k, v = case_inputs(7, "bf16", 4, 2, 64, 16, "slot", [50, 60], [2, 3], tail=0)
    out = torch.full_like(q, 3.0)
    dcu.dcu_paged_attention(q, i32([-4, 2, 900]), i32(lens), i32(table), k, v, out=out)
    ref = dcu.dcu_paged_attention(q, i32([0, 2, 5]), i32(lens), i32(table), k, v)
    assert torch.equal(out, ref)


def test_paged_attention_offsets_past_32_bits():
    """Pages whose elements lie beyond 2^31 elements and 2^32 bytes."""
    n_pages, page, KV, hd = 70000, 64, 4, 128  # 2.3e9 elements a tensor
    k = torch.zeros((n_pages, page, KV, hd), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    far = [69999, 3, 69998, 40000, 66000]
    g = torch.Generator(device="cuda").manual_seed(1)
    for p in far:
        k[p], v[p] = (torch.randn((page, KV, hd), generator=g, device="cuda").to(k.dtype) for _ in range(2))
    q = torch.randn((2, 8, hd), generator=g, device="cuda").to(k.dtype)
    out = dcu.dcu_paged_attention(q, i32([0, 2]), i32([300]), i32([far]), k, v)
    idx = torch.tensor(far, device="cuda")
    small = dcu.dcu_paged_attention(q, i32([0, 2]), i32([300]), i32([[0, 1, 2, 3, 4]]), k[idx], v[idx])
    assert torch.equal(out, small) and out.abs().max() > 0
    qkv = torch.randn((3, 16 * hd), generator=g, device="cuda")
    slot = [69997 * 64 + 5, 69990 * 64, 12]
    dcu.dcu_paged_write(qkv, i32([0, 3]), i32([0, 1, 2]), i32(slot), None, k, v, 8)
    x = qkv.view(3, 16, hd).to(k.dtype)
    for t, s in enumerate(slot):
        assert torch.equal(k[s // 64, s % 64], x[t, 8:12]) and torch.equal(v[s // 64, s % 64], x[t, 12:])


# ------------------------------------------------------------------ graphs, streams, a run together

def test_replayed_graph_follows_the_lengths():
    """One captured run serves whatever the device arrays hold at replay."""
    H, KV, hd, page, B, cap = 8, 2, 64, 16, 6, 40
    rng = np.random.default_rng(2)
    k, v = make_pages(3, 64, page, KV, hd, torch.bfloat16, "slot")
    lens, count, pos = i32([100] * B), i32([3] * B), i32(np.zeros((B, 160)))
    qkv = torch.randn((cap, (H + 2 * KV) * hd), device="cuda")
    rope = dcu.dcu_rope_table(200, hd)
    ws = torch.empty(dcu.dcu_paged_attention_workspace(k, v), dtype=torch.uint8, device="cuda")

    def step():
        table, _, _ = dcu.dcu_page_table(lens, page, 10, 64)
        start, rp, sl = dcu.dcu_slot_map(table, count, page, 64, cap, pos)
        q = dcu.dcu_paged_write(qkv, start, rp, sl, rope, k, v, H)
        return start, dcu.dcu_paged_attention(q, start, lens, table, k, v, workspace=ws)

    step()
    torch.cuda.synchronize()
    k0, v0 = k.clone(), v.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        start, out = step()
    for trial in range(3):
        n = rng.integers(0, 161, B)
        c = np.minimum(rng.integers(0, 7, B), n)
        p = np.zeros((B, 160), np.int32)
        for b in range(B):
            p[b, :c[b]] = np.sort(rng.choice(n[b], c[b], replace=False)) if n[b] else 0
        lens.copy_(i32(n)), count.copy_(i32(c)), pos.copy_(i32(p))
        k.copy_(k0), v.copy_(v0)
        graph.replay()
        torch.cuda.synchronize()
        T = int(c.sum())
        got = out[:T].clone()
        k.copy_(k0), v.copy_(v0)
        s2, o2 = step()
        assert torch.equal(start, s2) and torch.equal(got, o2[:T])


def test_another_stream_and_two_calls_at_once():
    a = case_inputs(11, "bf16", 28, 4, 128, 16, "slot", [3000, 900, 5], [1, 1, 1])
    b = case_inputs(12, "bf16", 28, 4, 128, 16, "slot", [50, 2500, 700], [1, 2, 1])
    args = [(q, i32(s), i32(n), i32(t), k, v) for q, s, n, t, k, v in (a, b)]
    want = [dcu.dcu_paged_attention(*x) for x in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(dcu.dcu_paged_attention(*args[i], stream=s if _ % 2 else s.cuda_stream))
    torch.cuda.synchronize()
    for i in range(2):
        n = int(args[i][1][-1].item())
        assert all(torch.equal(o[:n], want[i][:n]) for o in got[i])


def test_many_rows_on_far_pages():
    """The tensor-core path over pages whose elements lie beyond 2^31 elements and 2^32 bytes."""
    n_pages, page, KV, hd = 70000, 64, 4, 128
    k = torch.zeros((n_pages, page, KV, hd), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    far = [69999, 3, 69998, 40000, 66000]
    g = torch.Generator(device="cuda").manual_seed(5)
    for p in far:
        k[p], v[p] = (torch.randn((page, KV, hd), generator=g, device="cuda").to(k.dtype) for _ in range(2))
    q = torch.randn((90, 8, hd), generator=g, device="cuda").to(k.dtype)
    out = dcu.dcu_paged_attention(q, i32([0, 90]), i32([300]), i32([far]), k, v)
    idx = torch.tensor(far, device="cuda")
    small = dcu.dcu_paged_attention(q, i32([0, 90]), i32([300]), i32([[0, 1, 2, 3, 4]]), k[idx], v[idx])
    assert torch.equal(out, small) and out.abs().max() > 0


def test_many_rows_replayed_and_on_two_streams():
    """The tensor-core path in a captured call over changing lengths and rows, and two calls at once."""
    H, KV, hd, page, B, cap = 8, 2, 128, 16, 5, 400
    rng = np.random.default_rng(21)
    k, v = make_pages(22, 600, page, KV, hd, torch.bfloat16, "slot")
    g = torch.Generator(device="cuda").manual_seed(23)
    q = torch.randn((cap, H, hd), generator=g, device="cuda").to(k.dtype)
    start, lens = i32(np.zeros(B + 1)), i32(np.zeros(B))
    table = i32(rng.permutation(600)[:B * 120].reshape(B, 120))
    ws = torch.empty(dcu.dcu_paged_attention_workspace(k, v), dtype=torch.uint8, device="cuda")
    dcu.dcu_paged_attention(q, start, lens, table, k, v, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dcu.dcu_paged_attention(q, start, lens, table, k, v, workspace=ws)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for trial in range(4):
        rows = rng.integers(0, 80, B)
        lens.copy_(i32(rng.integers(0, 1921, B))), start.copy_(i32(np.concatenate([[0], np.cumsum(rows)])))
        T = int(rows.sum())
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert (out[T:] == 3.0).all()
        check_attention(out, q, f64(start).astype(int), f64(lens).astype(int), f64(table).astype(int), k, v, "bf16",
                        hd ** -0.5)
        got = [dcu.dcu_paged_attention(q, start, lens, table, k, v, stream=s) for s in streams * 4]
        torch.cuda.synchronize()
        assert all(torch.equal(o[:T], out[:T]) for o in got)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_layers_attention_run_together(dtype):
    """Token selection, slots, QKV product, RoPE + write, attention and the O product over pages, as a step runs
    them, against the same in fp64 with dense caches."""
    D, H, KV, hd, page, B, N = 256, 8, 2, 64, 16, 3, 150
    rng = np.random.default_rng(8)
    lens = np.array([150, 77, 120])
    d = np.abs(rng.standard_normal((B, N))).astype(np.float32)
    for b in range(B):
        d[b, lens[b]:] = 0.0  # beyond a sequence's end nothing drifts
    keys = np.zeros((B, N), np.int32)
    keys[:, 0] = [20, 40, 60]
    idx, cnt, _ = dcu.dcu_select_tokens(torch.tensor(d).cuda(), i32(keys), i32([1, 1, 1]), i32([9, 4, 0]), 4)
    pool = rng.permutation(40).astype(np.int32)
    table, _, _ = dcu.dcu_page_table(i32(lens), page, 10, 40, i32(pool))
    cap = 64
    start, rp, sl = dcu.dcu_slot_map(table, cnt, page, 40, cap, idx)
    n_idx, n_cnt = idx.cpu().numpy(), cnt.cpu().numpy()
    T = int(n_cnt.sum())
    x = O.store(rng.standard_normal((cap, D)), dtype)
    w = O.store(rng.standard_normal(((H + 2 * KV) * hd, D)) * 0.06, dtype)
    wo = O.store(rng.standard_normal((D, H * hd)) * 0.06, dtype)
    dev = lambda a: torch.tensor(a).to(DT[dtype]).cuda()  # noqa: E731
    k, v = make_pages(9, 40, page, KV, hd, DT[dtype], "slot")
    k0, v0 = f64(k), f64(v)
    y = dcu.dcu_linear(dev(x), dev(w))
    st = status_word()
    q = dcu.dcu_paged_write(y, start, rp, sl, dcu.dcu_rope_table(N, hd), k, v, H, status=st)
    att = dcu.dcu_paged_attention(q, start, i32(lens), table, k, v, status=st)
    res = dcu.dcu_linear(att.view(cap, H * hd), dev(wo))
    assert st.item() == 0
    # fp64, dense
    want = np.zeros((T, D))
    yy = (x @ w.T).reshape(cap, H + 2 * KV, hd)
    t, tab = 0, table.cpu().numpy()
    for b in range(B):
        p = n_idx[b, :n_cnt[b]]
        at = np.arange(lens[b])
        kd, vd = k0[tab[b, at // page], at % page], v0[tab[b, at // page], at % page]
        rows = slice(t, t + len(p))
        qk = O.store(R.rotate(yy[rows, :H + KV], p, 10000.0), dtype)
        kd[p], vd[p] = qk[:, H:], O.store(yy[rows, H + KV:], dtype)
        for h in range(H):
            s = qk[:, h] @ kd[:, h // (H // KV)].T / np.sqrt(hd)
            e = np.exp(s - s.max(1, keepdims=True))
            o = O.store(e / e.sum(1, keepdims=True) @ vd[:, h // (H // KV)], dtype)
            want[rows] += o @ wo[:, h * hd:(h + 1) * hd].T
        t += len(p)
    # stored roundings of q, k, v and the attention output that fall the other way on the two sides move a value by a
    # whole step (2 half steps); their effects add in the norm: 4 stages of one step each
    step = {"bf16": 2.0 ** -7, "f32": 1e-6}[dtype]
    assert np.linalg.norm(f64(res)[:T] - want) <= 4 * step * np.linalg.norm(want)
