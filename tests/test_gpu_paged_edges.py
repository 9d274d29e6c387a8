"""Calls of the paged K/V cache operators at the edges of what their documentation allows: what is flagged, and
batches of many sequences."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from dynamic_layer_wise_b200 import build, dcu
from tests import paged_ref as R
from tests.test_gpu_paged import DT, case_inputs, check_attention, f64, i32, make_pages, make_table, status_word

pytestmark = pytest.mark.gpu


def worst_error(got, q, start, lens, table, k, v, dtype, scale, p_step):
    """Largest error of the rows in terms of its bound, the weights' rounding given."""
    want, A, mag = R.attention(f64(q), start, lens, table, np.nan_to_num(f64(k), nan=0, posinf=0),
                               np.nan_to_num(f64(v), nan=0, posinf=0), scale)
    tol = R.attention_bound(want, A, mag, DT[dtype], max(1, max(lens)), q.shape[-1], p_step)
    n = int(start[-1])
    return np.max(np.abs(f64(got)[:n] - want[:n]) / tol[:n])


def round_once(q, start, lens, table, k, v, scale):
    """The mistake that the bound of two bf16 parts has to see: weights of one bf16, in fp64 otherwise."""
    qn, kn, vn = f64(q), np.nan_to_num(f64(k), nan=0, posinf=0), np.nan_to_num(f64(v), nan=0, posinf=0)
    out, page, KV = np.zeros(qn.shape), kn.shape[1], kn.shape[2]
    for b, n in enumerate(lens):
        rows, at = slice(start[b], start[b + 1]), np.arange(n)
        for h in range(qn.shape[1] if n else 0):
            kv = h // (qn.shape[1] // KV)
            x = qn[rows, h] @ kn[table[b, at // page], at % page, kv].T * scale
            w = np.exp(x - x.max(1, keepdims=True, initial=-np.inf)) if x.size else x
            bf = torch.tensor(w).to(torch.bfloat16).double().numpy()
            out[rows, h] = bf @ vn[table[b, at // page], at % page, kv] / w.sum(1, keepdims=True)
    return torch.tensor(out).to(torch.bfloat16)


# ------------------------------------------------------------------ RoPE + K/V write

@pytest.mark.parametrize("slot,flag", [(-1, 0), (-2, R.BAD_PAGE), (-2 ** 31, R.BAD_PAGE), (64, R.BAD_PAGE),
                                       (2 ** 31 - 1, R.BAD_PAGE), (63, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_write_flags_slots_outside_the_pages(dtype, slot, flag):
    H, KV, hd = 4, 2, 16
    k, v = make_pages(1, 4, 16, KV, hd, DT[dtype], "slot")
    k0, v0 = k.clone(), v.clone()
    qkv = torch.randn((3, (H + 2 * KV) * hd), device="cuda")
    st = status_word()
    q = dcu.dcu_paged_write(qkv, i32([0, 3]), i32([0, 1, 2]), i32([5, slot, 6]), None, k, v, H, status=st)
    assert st.item() == flag
    x = qkv.view(3, H + 2 * KV, hd).to(DT[dtype])
    assert torch.equal(q, x[:, :H])
    for t, s in enumerate([5, slot, 6]):
        if 0 <= s < 64:
            k0[s // 16, s % 16], v0[s // 16, s % 16] = x[t, H:H + KV], x[t, H + KV:]
    assert torch.equal(k, k0) and torch.equal(v, v0)


@pytest.mark.parametrize("used,flag", [(6, R.BAD_ROW), (2 ** 31 - 1, R.BAD_ROW), (5, 0), (0, 0), (-3, 0)])
def test_paged_write_flags_more_rows_than_there_are(used, flag):
    H, KV, hd = 4, 2, 16
    k, v = make_pages(2, 4, 16, KV, hd, torch.bfloat16, "slot")
    qkv = torch.randn((5, (H + 2 * KV) * hd), device="cuda")
    st = status_word()
    q = torch.full((5, H, hd), 7.0, dtype=k.dtype, device="cuda")
    dcu.dcu_paged_write(qkv, i32([0, used]), i32(range(5)), i32(range(5)), None, k, v, H, q=q, status=st)
    n = max(0, min(used, 5))
    assert st.item() == flag and torch.equal(q[:n], qkv.view(5, -1, hd)[:n, :H].to(k.dtype)) and (q[n:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_not_in_use_may_hold_anything(dtype):
    """Write and attention of 5 rows in buffers of 40 whose other rows hold NaN, far slots and far positions."""
    H, KV, hd, T, n = 8, 2, 64, 40, 5
    k, v = make_pages(3, 6, 16, KV, hd, DT[dtype], "slot")
    qkv = torch.full((T, (H + 2 * KV) * hd), float("nan"), device="cuda")
    qkv[:n] = torch.randn((n, (H + 2 * KV) * hd), device="cuda")
    pos, slot = np.full(T, -2 ** 31), np.full(T, 2 ** 31 - 1)
    pos[1::2], slot[1::2] = 2 ** 31 - 1, 7
    pos[:n], slot[:n] = [0, 1, 2, 30, 31], [16, 17, 18, 62, 63]
    tab, start, lens, table = dcu.dcu_rope_table(64, hd), i32([0, 3, n]), i32([3, 32]), i32([[1, 0], [2, 3]])

    def run(rows):
        kk, vv, st = k.clone(), v.clone(), status_word()
        q = torch.full((rows, H, hd), 7.0, dtype=DT[dtype], device="cuda")
        dcu.dcu_paged_write(qkv[:rows], start, i32(pos[:rows]), i32(slot[:rows]), tab, kk, vv, H, q=q, status=st)
        full = q.clone()
        full[n:] = float("nan")
        out = torch.full_like(q, 3.0)
        dcu.dcu_paged_attention(full, start, lens, table, kk, vv, out=out, status=st)
        return kk, vv, q, out, st.item()

    got, want = run(T), run(n)
    assert got[4] == want[4] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[2][:n], want[2]) and (got[2][n:] == 7.0).all() and (got[3][n:] == 3.0).all()
    # (the number of rows that there may be chooses the kernel, so the numbers agree to the roundings of two kernels)
    assert torch.isfinite(got[3]).all()
    for o in (got, want):
        check_attention(o[3], o[2], start.cpu().numpy(), lens.cpu().numpy(), table.cpu().numpy(), o[0], o[1], dtype,
                        hd ** -0.5)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("dtype,rows", [("bf16", 2), ("bf16", 40), ("f32", 9)])
def test_paged_attention_flags_row_starts_out_of_order_or_range(dtype, rows):
    q, start, lens, table, k, v = case_inputs(7, dtype, 4, 2, 64, 16, "slot", [50, 60, 33], [rows] * 3, tail=3)
    T = 3 * rows

    def call(s, max_rows=T + 3):
        st, out = status_word(), torch.full_like(q[:max_rows], 3.0)
        dcu.dcu_paged_attention(q[:max_rows], i32(s), i32(lens), i32(table), k, v, out=out, status=st)
        return st.item(), out

    flag, ref = call(start)
    assert flag == 0 and (ref[T:] == 3.0).all()
    # outside the rows: taken as the nearer end
    flag, out = call([-4, rows, 2 * rows, T])
    assert flag == R.BAD_ROW and torch.equal(out, ref)
    flag, out = call([0, rows, 2 * rows, T + 1], T)
    assert flag == R.BAD_ROW and torch.equal(out, ref[:T])
    flag, out = call([0, rows, 2 ** 31 - 1, 2 ** 31 - 1], 2 * rows)
    assert flag == R.BAD_ROW and torch.equal(out[:rows], ref[:rows])
    # out of order: rows that no sequence covers stay as they were
    for s in ([0, rows + 1, rows, 2 * rows], [0, 2 * rows, 0, rows], [rows, 0, 0, 0], [2, 1, 1, 2]):
        flag, out = call(s)
        covered = torch.zeros(T + 3, dtype=torch.bool)
        for a, z in zip(s, s[1:]):
            covered[a:z] = True
        assert flag == R.BAD_ROW and (out[~covered.cuda()] == 3.0).all()


# Sequences per thread in the search for a block's range: more than one from 129 (head dims above 128, bf16), 257 (bf16),
# 385 (float32) and 641 (tensor cores) sequences on.
MANY = [  # dtype, H, KV, hd, page, sequences, rows of a sequence, keys up to
    ("bf16", 2, 1, 64, 16, 700, 2, 60), ("bf16", 2, 1, 128, 5, 1500, 2, 40), ("f32", 2, 2, 64, 16, 700, 3, 50),
    ("f32", 1, 1, 16, 7, 1500, 4, 30), ("bf16", 4, 1, 256, 16, 300, 1, 40), ("f32", 2, 1, 256, 16, 300, 2, 40),
    ("bf16", 2, 1, 64, 16, 700, 20, 70), ("bf16", 1, 1, 128, 64, 1500, 30, 200), ("bf16", 2, 2, 224, 8, 800, 40, 30),
    ("bf16", 2, 1, 64, 5, 700, 30, 70),
]


@pytest.mark.parametrize("where", ["ragged", "sparse", "first", "last"])
@pytest.mark.parametrize("case", range(len(MANY)))
def test_paged_attention_of_many_sequences(case, where):
    """More sequences than a block has threads: all with rows, or rows in a few, in the first or in the last ones only."""
    dtype, H, KV, hd, page, B, rows, keys = MANY[case]
    rng = np.random.default_rng(100 + case)
    lens, n = rng.integers(0, keys + 1, B), np.zeros(B, int)
    if where == "ragged":
        n = rng.integers(0, 2 * rows + 1, B)
    else:
        at = {"sparse": rng.choice(B, 13, replace=False), "first": np.arange(3), "last": np.arange(B - 3, B)}[where]
        n[at] = rng.integers(1, 700, len(at)) if rows >= 8 else rng.integers(1, 9, len(at))
        lens[at] = rng.integers(keys // 2, 4 * keys, len(at))
    # rows behind the last sequence: the kernel is chosen by the rows there may be
    tail = 2 + max(0, rows * B - int(n.sum()))
    q, start, lens, table, k, v = case_inputs(200 + case, dtype, H, KV, hd, page, "slot", [int(x) for x in lens],
                                              [int(x) for x in n], tail=tail)
    st = status_word()
    out = torch.full_like(q, 3.0)
    dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v, out=out, status=st)
    assert st.item() == 0 and (out[int(start[-1]):] == 3.0).all()
    check_attention(out, q, start, lens, table, k, v, dtype, hd ** -0.5)


@pytest.mark.parametrize("H,KV,prompt,tokens", [(4, 4, 400, 64), (28, 4, 10, 64), (2, 2, 40, 255), (4, 4, 900, 64),
                                                (28, 4, 90, 64)])
def test_paged_attention_of_a_prompt_beside_tokens(H, KV, prompt, tokens):
    """One kernel takes all sequences of a call, the one for few rows in the first three."""
    rng = np.random.default_rng(prompt)
    at = tokens // 3
    rows, lens = [1] * tokens, [int(x) for x in rng.integers(0, 300, tokens)]
    rows.insert(at, prompt)
    lens.insert(at, prompt)
    q, start, lens, table, k, v = case_inputs(300 + prompt, "bf16", H, KV, 64, 16, "slot", lens, rows, tail=0)
    out = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v)
    check_attention(out, q, start, lens, table, k, v, "bf16", 64 ** -0.5)


@pytest.mark.parametrize("H,KV,hd,page,layout,lens,rows,scale", [
    (4, 2, 128, 5, "slot", [333, 70], [33, 20], None), (4, 4, 64, 20, "head", [700, 0, 129], [65, 3, 40], None),
    (6, 2, 48, 100, "mixed", [1000, 31], [30, 50], None), (14, 2, 256, 7, "slot", [500, 20], [9, 3], None),
    (4, 2, 64, 16, "slot", [250, 31], [40, 22], 0.0), (4, 2, 128, 16, "head", [600, 31], [70, 22], -0.1),
    (4, 2, 208, 16, "slot", [250, 31], [40, 22], -0.07), (4, 2, 128, 16, "skew", [600, 31], [70, 22], None)])
def test_many_rows_off_the_tensor_memory_path_keep_two_parts_of_a_weight(H, KV, hd, page, layout, lens, rows, scale):
    """Many rows a sequence over pages, scales or strides that the tcgen05 kernel does not take: weights as a high and a
    low bf16 part, 2^-16 in place of 2^-8, in all groups of 8 queries of a tile."""
    q, start, lens, table, k, v = case_inputs(400 + hd, "bf16", H, KV, hd, page, "slot" if layout == "skew" else layout,
                                              lens, rows, tail=0)
    if layout == "skew":  # slots whose distance is no multiple of a head's
        skew = lambda x: torch.empty((x.shape[0], page, KV * hd + 8), dtype=x.dtype, device="cuda")[..., :KV * hd].view(  # noqa: E731
            x.shape[0], page, KV, hd).copy_(x)
        k, v = skew(k), skew(v)
    out = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v, scale=scale)
    args = (q, start, lens, table, k, v)
    sc = hd ** -0.5 if scale is None else scale
    err = worst_error(out, *args, "bf16", sc, 2.0 ** -16)
    assert err <= 1.0, f"error {err:.2f} times its bound"
    if sc != 0.0:  # (equal weights are exact in one part)
        assert worst_error(round_once(*args, sc), *args, "bf16", sc, 2.0 ** -16) > 1.0


@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("bf16", 9), ("f32", 1)])
def test_the_largest_batch(dtype, rows):
    """65536 sequences through all four operators."""
    B, page = 65536, 8
    rng = np.random.default_rng(rows)
    lens = rng.integers(0, 20, B)
    n = np.minimum(rng.integers(rows, rows + 2, B), lens)
    first = lens - n
    need = -(-lens // page)
    n_pages, T = int(need.sum()), int(n.sum())
    pool = rng.permutation(n_pages).astype(np.int32)
    st = status_word()
    table, held, nxt = dcu.dcu_page_table(i32(lens), page, 3, n_pages, i32(pool), None, st)
    w_table, w_held, w_next, _ = R.page_table(lens, page, 3, n_pages, pool)
    assert np.array_equal(table.cpu().numpy(), w_table) and np.array_equal(held.cpu().numpy(), w_held)
    assert nxt.item() == w_next
    start, rp, slot = dcu.dcu_slot_map(table, i32(n), page, n_pages, T, None, i32(first), st)
    w_start, w_rp, w_slot, _ = R.slot_map(w_table, n, page, n_pages, T, None, first)
    assert np.array_equal(start.cpu().numpy(), w_start) and np.array_equal(rp.cpu().numpy(), w_rp)
    assert np.array_equal(slot.cpu().numpy(), w_slot)
    k, v = make_pages(5, n_pages, page, 1, 16, DT[dtype], "slot")
    qkv = torch.randn((T, 3 * 16), device="cuda")
    q = dcu.dcu_paged_write(qkv, start, rp, slot, None, k, v, 1, status=st)
    x = qkv.to(DT[dtype])
    at = slot.long()
    assert torch.equal(q[:, 0], x[:, :16]) and torch.equal(k.view(-1, 16)[at], x[:, 16:32])
    assert torch.equal(v.view(-1, 16)[at], x[:, 32:])
    # buffers as long as the rows that there may be: nine a sequence are many for the choice of the kernel
    room = torch.zeros((max(T, rows * B) + 7, 1, 16), dtype=DT[dtype], device="cuda")
    room[:T] = q
    out = dcu.dcu_paged_attention(room, start, i32(lens), table, k, v, status=st)
    assert st.item() == 0
    check_attention(out, room, w_start, lens, w_table, k, v, dtype, 0.25)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 200])
@pytest.mark.parametrize("B", [1, 3, 700])
def test_paged_attention_without_any_rows(dtype, T, B):
    k, v = make_pages(1, 4, 16, 2, 64, DT[dtype], "slot")
    q, st = torch.randn((T, 4, 64), device="cuda").to(k.dtype), status_word()
    for at in (0, T):
        out = torch.full_like(q, 3.0)
        dcu.dcu_paged_attention(q, i32([at] * (B + 1)), i32([40] * B), i32([[0, 1, 2]] * B), k, v, out=out, status=st)
        assert st.item() == 0 and (out == 3.0).all()


@pytest.mark.parametrize("dtype,rows", [("bf16", 2), ("bf16", 50), ("f32", 3)])
def test_paged_attention_of_rows_that_begin_later(dtype, rows):
    """Rows before row_start[0] belong to no sequence."""
    q, start, lens, table, k, v = case_inputs(17, dtype, 4, 2, 64, 16, "slot", [50, 60], [rows, rows], tail=9)
    call = lambda x, s: dcu.dcu_paged_attention(x, i32(s), i32(lens), i32(table), k, v,  # noqa: E731
                                                out=torch.full_like(x, 3.0))
    ref = call(q, start)
    out = call(torch.roll(q, 5, 0), start + 5)
    assert torch.equal(out[5:5 + 2 * rows], ref[:2 * rows])
    assert (out[:5] == 3.0).all() and (out[5 + 2 * rows:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,KV,hd,page,lens,rows", [
    (5000, 1, 16, 16, [90], [2]), (4097, 1, 32, 5, [40, 0, 7], [1, 3, 2]), (1800, 900, 16, 16, [70, 20], [1, 1]),
    (700, 700, 32, 8, [33], [30]), (4, 2, 64, 4096, [5000, 4096, 4097], [3, 1, 20]), (4, 2, 64, 30000, [29999], [40])])
def test_paged_attention_of_many_heads_and_long_pages(dtype, H, KV, hd, page, lens, rows):
    q, start, lens, table, k, v = case_inputs(500 + hd, dtype, H, KV, hd, page, "slot", lens, rows)
    st, out = status_word(), torch.full_like(q, 3.0)
    dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v, out=out, status=st)
    assert st.item() == 0 and (out[int(start[-1]):] == 3.0).all()
    check_attention(out, q, start, lens, table, k, v, dtype, hd ** -0.5)


@pytest.mark.parametrize("dtype,rows,page", [("bf16", 2, 16), ("bf16", 2, 5), ("bf16", 50, 16), ("bf16", 50, 5), ("f32", 9, 16)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_cached_value_that_is_not_finite_stays_with_its_sequence_head_and_dim(dtype, rows, page, bad):
    q, start, lens, table, k, v = case_inputs(19, dtype, 4, 2, 64, page, "slot", [700, 200], [rows, rows], tail=0)
    call = lambda k, v: dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v)  # noqa: E731
    ref = call(k, v)
    at = 333  # a key of the first sequence, kv head 1 (query heads 2 and 3)
    kb, vb = k.clone(), v.clone()
    vb[table[0, at // page], at % page, 1, 7] = bad
    out, hit = call(k, vb), torch.zeros_like(ref, dtype=torch.bool)
    hit[:rows, 2:, 7] = True
    assert torch.equal(out[~hit], ref[~hit]) and not out[hit].isfinite().any()
    # a key: scores of +inf or NaN make their rows NaN, a score of -inf has no weight
    kb[table[0, at // page], at % page, 1, 7] = bad
    out, hit = call(kb, v), torch.zeros_like(ref, dtype=torch.bool)
    lost = (q[:rows, 2:, 7].float() * bad) != float("-inf")
    hit[:rows, 2:] = lost[..., None]
    assert out[hit].isnan().all() and out[~hit].isfinite().all()
    rest = torch.ones_like(ref, dtype=torch.bool)
    rest[:rows, 2:] = False
    assert torch.equal(out[rest], ref[rest])
    there = np.delete(np.arange(700), at)  # the other keys, for the rows that gave this one no weight
    kn, vn = (f64(x)[table[0, there // page], there % page, 1] for x in (k, v))
    for r, h in torch.nonzero(~lost).tolist():
        x = kn @ f64(q[r, 2 + h]) / 8
        w = np.exp(x - x.max())
        w /= w.sum()
        # weights off by 2^-8 at most, the result by half a step, and 64 + 700 fp32 sums
        assert np.all(np.abs(f64(out[r, 2 + h]) - w @ vn) <= (2.0 ** -8 + 1e-4) * (w @ np.abs(vn)) + 2.0 ** -8 * np.abs(w @ vn))
    # no key with a weight: zeros
    qp = q.clone()
    qp[:rows, 2:, 7] = 1.0
    kb[torch.tensor(table[0, np.arange(700) // page]).long(), torch.arange(700) % page, 1, 7] = float("-inf")
    out = dcu.dcu_paged_attention(qp, i32(start), i32(lens), i32(table), kb, v)
    assert (out[:rows, 2:] == 0).all() and torch.equal(out[rest], ref[rest])


@pytest.mark.parametrize("dtype,rows", [("bf16", 2), ("bf16", 50), ("f32", 9)])
def test_paged_attention_of_shared_pages(dtype, rows):
    """Two sequences with one prefix, pages twice in a row of the table, and V in the pages of K."""
    q, start, lens, table, k, v = case_inputs(18, dtype, 4, 2, 64, 16, "slot", [100, 130], [rows, rows])
    k, v = k.nan_to_num(0, 0), v.nan_to_num(0, 0)
    table[1, :6] = table[0, :6]
    table[1, 7] = table[1, 6]
    out = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, v)
    check_attention(out, q, start, lens, table, k, v, dtype, 0.125)
    out = dcu.dcu_paged_attention(q, i32(start), i32(lens), i32(table), k, k)
    check_attention(out, q, start, lens, table, k, k, dtype, 0.125)


def test_slot_map_of_more_rows_than_32_bits_count():
    """Prefix sums of the counts pass 2^32; the rows there is room for are mapped and the rest flagged."""
    table, n_pages = make_table(np.random.default_rng(0), [40, 40, 40], 16)
    for count in ([3, 2 ** 31 - 1, 2 ** 31 - 1], [2 ** 31 - 1] * 3, [3, 2, 2 ** 31 - 1]):
        st = status_word()
        start, rp, sl = dcu.dcu_slot_map(i32(table), i32(count), 16, n_pages, 12, None, i32([1, 0, 5]), st)
        w = [0] + [min(12, int(x)) for x in np.cumsum(np.array(count, np.int64))]
        pos = [f + j for b, f in enumerate([1, 0, 5]) for j in range(w[b + 1] - w[b])]
        seq = [b for b in range(3) for _ in range(w[b + 1] - w[b])]
        assert start.cpu().tolist() == w and rp.cpu().tolist() == pos and st.item() == R.BAD_ROW
        assert sl.cpu().tolist() == [int(table[b, p // 16]) * 16 + p % 16 for b, p in zip(seq, pos)]


@pytest.mark.parametrize("rows", [1, 40])
def test_a_captured_call_may_be_the_first(rows):
    """Nothing has to run before a capture: kernels, limits and tensor maps are set up within it."""
    code = f"""
import torch
from dynamic_layer_wise_b200 import dcu
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
k = torch.randn(8, 16, 2, 64, device="cuda").to(torch.bfloat16)
v = torch.randn_like(k)
qkv = torch.randn({rows}, 8 * 64, device="cuda")
lens, count, first = i32([100]), i32([{rows}]), i32([100 - {rows}])
torch.cuda.synchronize()
def step():
    table, _, _ = dcu.dcu_page_table(lens, 16, 7, 8)
    start, pos, slot = dcu.dcu_slot_map(table, count, 16, 8, {rows}, None, first)
    rope = dcu.dcu_rope_table(100, 64)
    q = dcu.dcu_paged_write(qkv, start, pos, slot, rope, k, v, 4)
    return dcu.dcu_paged_attention(q, start, lens, table, k, v)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, step()) and out.abs().max() > 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=build.ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
