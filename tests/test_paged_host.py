"""Refusals of the paged K/V cache entry points: checked on the host, no GPU needed."""
import ctypes

import pytest
import torch

from dynamic_layer_wise_b200 import build, dcu

P = 4096  # a 16-byte aligned address that is never read


@pytest.fixture(scope="module")
def L():
    build.build_all()
    return dcu.lib()


def _pages(**kw):
    base = dict(k=P, v=P, page_stride=16 * 4 * 64, slot_stride=4 * 64, head_stride=64, n_pages=8, page_size=16,
                n_kv_heads=4, head_dim=64, dtype=dcu.DCU_BF16)
    base.update(kw)
    return ctypes.byref(dcu.dcu_pages(**base))


BAD_PAGES = [dict(k=None), dict(v=None), dict(dtype=5), dict(n_pages=0), dict(page_size=0), dict(n_kv_heads=0),
             dict(head_dim=24), dict(head_dim=272), dict(head_dim=0), dict(k=P + 8), dict(v=P + 2),
             dict(page_stride=-64), dict(slot_stride=260), dict(head_stride=68), dict(n_pages=1 << 28),
             dict(dtype=dcu.DCU_F32, head_stride=66)]

TABLE = dict(lens=P, B=2, page_size=16, max_pages=4, n_pages=8, pool=P, n_pool=8, first=None, table=P, held=P,
             next=P + 64, status=None, stream=None)
MAP = dict(table=P, B=2, max_pages=4, page_size=16, n_pages=8, count=P, pos=None, pos_stride=0, first=None,
           max_rows=4, row_start=P, row_pos=P, slot=P, status=None, stream=None)
WRITE = dict(qkv=P, max_rows=4, n_rows=P, row_pos=P, slot=P, rope=P, max_pos=64, n_heads=8, pages={}, q=P,
             status=None, stream=None)
ATTN = dict(q=P, max_rows=4, row_start=P, B=2, kv_len=P, table=P, max_pages=4, n_heads=8, pages={}, scale=0.125,
            out=2 * P, ws=P, ws_bytes=1 << 40, status=None, stream=None)


def _call(fn, base, **kw):
    a = dict(base, **kw)
    if "pages" in a and isinstance(a["pages"], dict):
        a["pages"] = _pages(**a["pages"])
    return fn(*a.values())


@pytest.mark.parametrize("bad", [dict(lens=None), dict(B=0), dict(B=65537), dict(page_size=0), dict(max_pages=0),
                                 dict(n_pages=0), dict(n_pages=1 << 30), dict(n_pool=-1), dict(pool=None, n_pool=3),
                                 dict(table=None), dict(held=None), dict(next=None), dict(first=P + 64)])
def test_page_table_refusals(L, bad):
    assert _call(L.dcu_page_table, TABLE, **bad) == dcu.DCU_EINVAL
    assert b"dcu_page_table" in L.dcu_last_error(None)


@pytest.mark.parametrize("bad", [dict(table=None), dict(B=0), dict(B=65537), dict(max_pages=0), dict(page_size=-1),
                                 dict(n_pages=0), dict(count=None), dict(pos=P), dict(pos=P, pos_stride=4, first=P),
                                 dict(max_rows=-1), dict(row_start=None), dict(row_pos=None), dict(slot=None)])
def test_slot_map_refusals(L, bad):
    assert _call(L.dcu_slot_map, MAP, **bad) == dcu.DCU_EINVAL


@pytest.mark.parametrize("bad", [dict(qkv=None), dict(max_rows=-1), dict(row_pos=None), dict(slot=None),
                                 dict(max_pos=0), dict(n_heads=0), dict(q=None), dict(qkv=P + 4), dict(rope=P + 8),
                                 dict(q=P + 2), dict(pages=dict(slot_stride=0)), dict(pages=dict(page_stride=0)),
                                 dict(pages=dict(head_stride=0))])
def test_paged_write_refusals(L, bad):
    assert _call(L.dcu_paged_write, WRITE, **bad) == dcu.DCU_EINVAL


@pytest.mark.parametrize("bad", [dict(q=None), dict(max_rows=-1), dict(row_start=None), dict(B=0), dict(B=65537),
                                 dict(kv_len=None), dict(table=None), dict(max_pages=0), dict(n_heads=0),
                                 dict(n_heads=6), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38),
                                 dict(out=None), dict(out=P), dict(q=P + 8), dict(out=P + 4), dict(ws=None),
                                 dict(ws=P + 8), dict(ws_bytes=0)])
def test_paged_attention_refusals(L, bad):
    assert _call(L.dcu_paged_attention, ATTN, **bad) == dcu.DCU_EINVAL


@pytest.mark.parametrize("bad", BAD_PAGES)
def test_page_geometry_refusals(L, bad):
    n = ctypes.c_int64(0)
    assert L.dcu_paged_attention_workspace(_pages(**bad), ctypes.byref(n)) == dcu.DCU_EINVAL
    assert _call(L.dcu_paged_write, WRITE, pages=bad) == dcu.DCU_EINVAL
    assert _call(L.dcu_paged_attention, ATTN, pages=bad) == dcu.DCU_EINVAL


@pytest.mark.parametrize("bad", [dict(tab=None), dict(max_pos=0), dict(head_dim=7), dict(theta=0.0),
                                 dict(theta=float("inf")), dict(theta=float("nan"))])
def test_rope_table_refusals(L, bad):
    assert _call(L.dcu_rope_table, dict(tab=P, max_pos=8, head_dim=64, theta=1e4, stream=None), **bad) == dcu.DCU_EINVAL


def test_zero_rows_are_no_work(L):
    assert _call(L.dcu_paged_write, WRITE, max_rows=0, qkv=None, q=None) == dcu.DCU_OK
    assert _call(L.dcu_paged_attention, ATTN, max_rows=0, q=None, out=None) == dcu.DCU_OK


def test_binding_refuses_cpu_tensors_and_wrong_types(L):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        dcu.dcu_page_table(i, 16, 4, 8)
    with pytest.raises(TypeError):
        dcu.dcu_page_table([1, 2], 16, 4, 8)
    with pytest.raises(ValueError):
        dcu.dcu_slot_map(i[None], i, 16, 8, 4)
    k = torch.zeros(2, 16, 4, 64)
    with pytest.raises(ValueError):
        dcu.dcu_paged_attention(torch.zeros(3, 8, 64), i, i, i[None], k, k)
    with pytest.raises(ValueError):
        dcu.dcu_paged_write(torch.zeros(3, 1024), i, i, i, None, k, k, 8)
    with pytest.raises(ValueError):
        dcu.dcu_rope_table(0, 64, device="cuda:0")


def test_sizes_and_overlaps_that_are_refused(L):
    # a launch's second grid dimension ends at 65535: 4096 table columns per block
    assert _call(L.dcu_page_table, TABLE, max_pages=(1 << 27) + 1) == dcu.DCU_EINVAL
    # queries of a kv head, 2^27 rows x 8 heads
    assert _call(L.dcu_paged_attention, ATTN, max_rows=1 << 27, n_heads=32, out=1 << 46) == dcu.DCU_EINVAL
    # 4 rows x 8 heads x 64 dims x 2 bytes of q end where out may begin
    assert _call(L.dcu_paged_attention, ATTN, out=P + 4096 - 16) == dcu.DCU_EINVAL
    assert _call(L.dcu_paged_attention, ATTN, q=2 * P, out=P + 16) == dcu.DCU_EINVAL
    # q may not be written over the float32 rows that are still to be read, nor K over V
    other = dict(pages=dict(v=1 << 30), q=P + 4 * 16 * 64 * 4 - 16)
    assert _call(L.dcu_paged_write, WRITE, **other) == dcu.DCU_EINVAL
    assert b"overlaps" in L.dcu_last_error(None)
    assert _call(L.dcu_paged_write, WRITE, q=1 << 30) == dcu.DCU_EINVAL
    assert b"share" in L.dcu_last_error(None)
    # 32 items a head of 256 dims, 512 a block, 65535 slices of a row
    assert _call(L.dcu_paged_write, WRITE, n_heads=(1 << 19) - 7) == dcu.DCU_EINVAL
    assert b"heads" in L.dcu_last_error(None)


def test_binding_refuses_empty_tensors_that_would_pass_for_none(L):
    """An empty tensor has no address, and without one the library counts positions from 0 and rotates nothing."""
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="pos: expected at least one column"):
        dcu.dcu_slot_map(i[None], i[:1], 16, 8, 4, pos=torch.zeros(1, 0, dtype=torch.int32))
    k = torch.zeros(2, 16, 4, 64)
    with pytest.raises(ValueError, match="rope: expected at least one position"):
        dcu.dcu_paged_write(torch.zeros(4, 1024), i, i, i, torch.zeros(0, 32, 2), k, k, 8)


@pytest.mark.parametrize("call", [
    lambda i, k: dcu.dcu_page_table(i, (1 << 32) + 16, 4, 8), lambda i, k: dcu.dcu_page_table(i, 16, (1 << 32) + 4, 8),
    lambda i, k: dcu.dcu_page_table(i, 16, 4, (1 << 32) + 8), lambda i, k: dcu.dcu_slot_map(i[None], i[:1], 1 << 32, 8, 4),
    lambda i, k: dcu.dcu_slot_map(i[None], i[:1], 16, (1 << 32) + 8, 4),
    lambda i, k: dcu.dcu_slot_map(i[None], i[:1], 16, 8, 1 << 31),
    lambda i, k: dcu.dcu_rope_table((1 << 32) + 8, 64, device="cuda:0"),
    lambda i, k: dcu.dcu_rope_table(8, 1 << 32, device="cuda:0"),
    lambda i, k: dcu.dcu_slot_map(i[None], i[:1], 16, 8, 4, pos=i[:1].expand(1, (1 << 32) + 2)),
    lambda i, k: dcu.dcu_paged_attention(k[0, :3], i, i, i[:1].expand(1, (1 << 32) + 2), k, k),
    lambda i, k: dcu.dcu_paged_attention(k[0, :3], i, i, i[None], *[k[:, :1].expand(2, (1 << 32) + 1, 4, 64)] * 2)])
def test_binding_refuses_sizes_past_32_bits(L, call):
    """ctypes keeps the low 32 bits of an integer: 2^32 + 16 would become 16."""
    with pytest.raises(ValueError, match="sizes above"):
        call(torch.zeros(4, dtype=torch.int32), torch.zeros(2, 16, 4, 64))


# arrays far apart: what follows moves one output onto another array, 4 bytes of overlap each time
APART = {
    "dcu_page_table": dict(TABLE, lens=1 << 20, pool=2 << 20, first=3 << 20, table=4 << 20, held=5 << 20, next=6 << 20,
                           status=7 << 20),
    "dcu_slot_map": dict(MAP, table=1 << 20, count=2 << 20, pos=None, first=3 << 20, row_start=4 << 20,
                         row_pos=5 << 20, slot=6 << 20, status=7 << 20),
    "dcu_paged_write": dict(WRITE, qkv=1 << 20, n_rows=2 << 20, row_pos=3 << 20, slot=4 << 20, rope=5 << 20,
                            q=6 << 20, status=7 << 20, pages=dict(k=1 << 30, v=2 << 30)),
    "dcu_paged_attention": dict(ATTN, q=1 << 20, row_start=2 << 20, kv_len=3 << 20, table=4 << 20, out=5 << 20,
                                ws=1 << 34, status=7 << 20, pages=dict(k=1 << 30, v=2 << 30)),
}


@pytest.mark.parametrize("fn,move", [
    ("dcu_page_table", dict(held=1 << 20)), ("dcu_page_table", dict(held=(1 << 20) + 4)),
    ("dcu_page_table", dict(table=(2 << 20) - 28)), ("dcu_page_table", dict(next=(2 << 20) + 28)),
    ("dcu_page_table", dict(table=3 << 20)), ("dcu_page_table", dict(held=(4 << 20) + 28)),
    ("dcu_page_table", dict(next=(5 << 20) + 4)), ("dcu_page_table", dict(status=6 << 20)),
    ("dcu_slot_map", dict(row_start=2 << 20)), ("dcu_slot_map", dict(row_pos=(1 << 20) + 28)),
    ("dcu_slot_map", dict(slot=(3 << 20) + 4)), ("dcu_slot_map", dict(slot=(5 << 20) - 12)),
    ("dcu_slot_map", dict(row_start=6 << 20)), ("dcu_slot_map", dict(pos=5 << 20, pos_stride=4, first=None)),
    ("dcu_slot_map", dict(status=(5 << 20) + 12)),
    ("dcu_paged_write", dict(q=3 << 20)), ("dcu_paged_write", dict(q=4 << 20)), ("dcu_paged_write", dict(q=2 << 20)),
    ("dcu_paged_write", dict(q=(5 << 20) + 64 * 64 * 4 - 16)), ("dcu_paged_write", dict(status=6 << 20)),
    ("dcu_paged_attention", dict(ws=1 << 20)), ("dcu_paged_attention", dict(ws=5 << 20)),
    ("dcu_paged_attention", dict(out=2 << 20)), ("dcu_paged_attention", dict(out=3 << 20)),
    ("dcu_paged_attention", dict(out=4 << 20)), ("dcu_paged_attention", dict(status=(1 << 20) + 4096 - 4)),
    ("dcu_paged_attention", dict(kv_len=(1 << 34) + 1024))])
def test_outputs_over_other_arrays_are_refused(L, fn, move):
    """Threads read the inputs and write the outputs in no order: a call in place would give wrong answers."""
    assert _call(getattr(L, fn), APART[fn], **move) == dcu.DCU_EINVAL
    assert fn.encode() in L.dcu_last_error(None) and b"overlap" in L.dcu_last_error(None)


REFUSALS = [("dcu_page_table", test_page_table_refusals), ("dcu_slot_map", test_slot_map_refusals),
            ("dcu_paged_write", test_paged_write_refusals), ("dcu_paged_attention", test_paged_attention_refusals)]


@pytest.mark.parametrize("fn,bad", [(fn, bad) for fn, t in REFUSALS for bad in t.pytestmark[0].args[1]
                                    if bad not in (dict(first=P + 64), dict(out=P))])
def test_refusals_do_not_rest_on_an_overlap(L, fn, bad):
    """The arguments refused above, on arrays that lie apart (the two left out are overlaps themselves)."""
    assert _call(getattr(L, fn), APART[fn], **bad) == dcu.DCU_EINVAL
    assert b"overlap" not in L.dcu_last_error(None)
