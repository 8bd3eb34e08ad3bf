"""Refusals and sizes of the paged-cache calls, found on the host (no GPU:
every call here fails its checks before anything is enqueued, or asks for a
size only)."""
import pytest

import kv_cache_transform_amd as K

P = 1 << 20          # an aligned address that no call here dereferences
BIG = 1 << 40


def _pages(**kw):
    a = dict(k=P, v=P, n_blocks=8, block_size=16, kv_heads=2, head_dim=64, dtype=K.KVTC_BF16,
             k_capacity=8 * 16 * 128 * 2, v_capacity=8 * 16 * 128 * 2)
    a.update(kw)
    return K.make_pages(**a)


def _requests(**kw):
    a = dict(block_table=P, table_width=4, lens=P, n_requests=3)
    a.update(kw)
    return K.make_requests(**a)


def _queries(**kw):
    a = dict(q=P, out=P, q_heads=4, scale=0.125)
    a.update(kw)
    return K.make_queries(**a)


def _plan(**kw):
    a = dict(old_lens=P, new_lens=P, n_requests=3, block_size=16, free_blocks=P, n_free=4, n_blocks=8,
             block_table=P, table_width=4, slots=P, n_slots=10)
    a.update(kw)
    return K.make_page_plan(**a)


def _rows(**kw):
    a = dict(k=P, v=P, n_rows=3, slots=P, dtype=K.KVTC_BF16, k_stride=128, v_stride=128)
    a.update(kw)
    return K.make_page_rows(**a)


def _refused(status, f, *a, **kw):
    with pytest.raises(K.KvtcError) as e:
        f(*a, **kw)
    assert e.value.status == status, e.value
    assert len(str(e.value)) > 20


INV, CAP, UNS = K.KVTC_E_INVALID, K.KVTC_E_CAPACITY, K.KVTC_E_UNSUPPORTED

BAD_PAGES = [
    (INV, dict(k=0)), (INV, dict(k=P + 8)), (INV, dict(n_blocks=0)), (INV, dict(block_size=0)), (INV, dict(block_size=-16)),
    (INV, dict(kv_heads=0)), (INV, dict(head_dim=0)), (INV, dict(dtype=2)), (UNS, dict(head_dim=60)), (UNS, dict(head_dim=264)),
    (UNS, dict(n_blocks=1 << 20, block_size=1 << 11)), (CAP, dict(k_capacity=8 * 16 * 128 * 2 - 1)),
    (CAP, dict(dtype=K.KVTC_F32)),
]
BAD_REQUESTS = [
    (INV, dict(block_table=0)), (INV, dict(lens=0)), (INV, dict(lens=P + 2)), (INV, dict(n_requests=0)), (INV, dict(n_requests=-1)),
    (CAP, dict(n_requests=K.KVTC_MAX_JOBS + 1)), (INV, dict(table_width=0)), (INV, dict(table_stride=3)),
    (UNS, dict(table_width=1 << 27)), (UNS, dict(table_width=1 << 18, n_requests=1 << 12)), (UNS, dict(table_width=1 << 26)), (INV, dict(status=P + 1)),
]


@pytest.mark.parametrize("st,kw", BAD_PAGES)
def test_bad_pages(st, kw):
    bad = _pages(**kw)
    _refused(st, K.kvtc_page_write, bad, _rows())
    _refused(st, K.kvtc_page_bounds, bad, _requests(), None, P, BIG)
    _refused(st, K.kvtc_page_attend, bad, _requests(), _queries(), None, P, BIG)


@pytest.mark.parametrize("kw", [dict(v=0), dict(v=P + 4)])
def test_v_pages_are_checked_where_they_are_used(kw):
    _refused(INV, K.kvtc_page_write, _pages(**kw), _rows())
    _refused(INV, K.kvtc_page_attend, _pages(**kw), _requests(), _queries(), None, P, BIG)
    _refused(CAP, K.kvtc_page_attend, _pages(v_capacity=100), _requests(), _queries(), None, P, BIG)


@pytest.mark.parametrize("st,kw", BAD_REQUESTS)
def test_bad_requests(st, kw):
    bad = _requests(**kw)
    _refused(st, K.kvtc_page_bounds, _pages(), bad, None, P, BIG)
    _refused(st, K.kvtc_page_attend, _pages(), bad, _queries(), None, P, BIG)
    _refused(st, K.kvtc_page_select, _pages(), bad, _queries(), P, K.make_selection(P, 4), P, BIG, BIG)


@pytest.mark.parametrize("st,kw", [
    (INV, dict(q=0)), (INV, dict(q=P + 8)), (INV, dict(q_heads=0)), (INV, dict(q_heads=3)), (INV, dict(q_stride=128)),
    (INV, dict(q_stride=260)), (INV, dict(q_stride=-256)), (INV, dict(q_heads=1 << 17)),
])
def test_bad_queries(st, kw):
    bad = _queries(**kw)
    _refused(st, K.kvtc_page_attend, _pages(), _requests(), bad, None, P, BIG)
    _refused(st, K.kvtc_page_select, _pages(), _requests(), bad, P, K.make_selection(P, 4), P, BIG, BIG)


@pytest.mark.parametrize("kw", [dict(out=0), dict(out=P + 8), dict(out_stride=128), dict(out_stride=257), dict(lse=P + 2),
                                dict(scale=float("nan")), dict(scale=float("inf"))])
def test_bad_outputs(kw):
    _refused(INV, K.kvtc_page_attend, _pages(), _requests(), _queries(**kw), None, P, BIG)


@pytest.mark.parametrize("a", [(0, 4), (P + 2, 4), (P, 0), (P, -1), (P, 4, -1, 0), (P, 4, 0, -1), (P, 4, 3, 2),
                               (P, 4, 2**31 - 1, 2**31 - 1)])
def test_bad_selection(a):
    _refused(INV, K.kvtc_page_select, _pages(), _requests(), _queries(), P, K.make_selection(*a), P, BIG, BIG)


def test_null_descriptors_and_buffers():
    pages, req, q, sel = _pages(), _requests(), _queries(), K.make_selection(P, 4)
    _refused(INV, K.kvtc_page_tables, None)
    _refused(INV, K.kvtc_page_write, None, _rows())
    _refused(INV, K.kvtc_page_write, pages, None)
    _refused(INV, K.kvtc_page_bounds, None, req, None, P, BIG)
    _refused(INV, K.kvtc_page_bounds, pages, None, None, P, BIG)
    _refused(INV, K.kvtc_page_bounds, pages, req, None, 0, BIG)
    _refused(INV, K.kvtc_page_bounds, pages, req, P + 2, P, BIG)
    _refused(CAP, K.kvtc_page_bounds, pages, req, None, P, 8 * 2 * 128 * 2 - 1)
    _refused(INV, K.kvtc_page_attend, None, req, q, None, P, BIG)
    _refused(INV, K.kvtc_page_attend, pages, None, q, None, P, BIG)
    _refused(INV, K.kvtc_page_attend, pages, req, None, None, P, BIG)
    _refused(INV, K.kvtc_page_attend, pages, req, q, None, 0, BIG)
    _refused(INV, K.kvtc_page_attend, pages, req, q, None, P + 8, BIG)
    _refused(INV, K.kvtc_page_attend, pages, req, q, K.make_selection(0, 4), P, BIG)
    _refused(INV, K.kvtc_page_select, pages, req, q, P, None, P, BIG, BIG)
    _refused(INV, K.kvtc_page_select, pages, req, q, 0, sel, P, BIG, BIG)
    _refused(CAP, K.kvtc_page_select, pages, req, q, P, sel, P, BIG, 8 * 2 * 128 * 2 - 1)


@pytest.mark.parametrize("st,kw", [
    (INV, dict(new_lens=0)), (INV, dict(block_table=0)), (INV, dict(free_blocks=0)), (INV, dict(slots=0)), (INV, dict(block_size=0)),
    (INV, dict(n_blocks=0)), (INV, dict(n_free=-1)), (INV, dict(n_slots=-1)), (INV, dict(n_requests=0)),
    (CAP, dict(n_requests=K.KVTC_MAX_JOBS + 1)), (INV, dict(table_width=0)), (INV, dict(table_stride=3)),
    (UNS, dict(n_blocks=1 << 27)), (UNS, dict(table_width=1 << 26)), (UNS, dict(table_width=1 << 18, n_requests=1 << 12)), (INV, dict(old_lens=P + 1)), (INV, dict(slots=P + 2)),
    (INV, dict(free_from=P, taken=P)), (INV, dict(free_from=P, starts=P)),
])
def test_bad_plan(st, kw):
    _refused(st, K.kvtc_page_tables, _plan(**kw))


@pytest.mark.parametrize("kw", [dict(k=0), dict(v=0), dict(slots=0), dict(k=P + 1), dict(v=P + 1), dict(slots=P + 2), dict(n_rows=-1),
                                dict(dtype=7), dict(k_stride=-128), dict(v_stride=-1), dict(status=P + 2),
                                dict(dtype=K.KVTC_F32, k=P + 2)])
def test_bad_rows(kw):
    _refused(INV, K.kvtc_page_write, _pages(), _rows(**kw))


def test_no_rows_is_no_work():
    K.kvtc_page_write(_pages(), _rows(n_rows=0))


def test_workspace_sizes():
    pages, req, q = _pages(), _requests(), _queries()
    n = K.kvtc_page_workspace_bytes(pages, req, q)
    m = K.kvtc_page_workspace_bytes(pages, req, q, K.make_selection(P, 4, 1, 1))
    assert 0 < n <= m
    _refused(CAP, K.kvtc_page_attend, pages, req, q, None, P, n - 1)
    _refused(CAP, K.kvtc_page_select, pages, req, q, P, K.make_selection(P, 4, 1, 1), P, m - 1, BIG)
    # sizes only: no pointer is needed, and what the calls refuse has none
    bare = K.kvtc_pages(None, None, 0, 0, 8, 16, 2, 64, K.KVTC_BF16)
    assert K.kvtc_page_workspace_bytes(bare, K.kvtc_requests(None, None, None, 3, 4, 4),
                                       K.kvtc_queries(None, None, None, 0, 0, 4, 1.0)) == n
    for bad in (dict(head_dim=60), dict(block_size=0)):
        assert K.kvtc_page_workspace_bytes(_pages(**bad), req, q) == 0
    assert K.kvtc_page_workspace_bytes(pages, _requests(n_requests=0), q) == 0
    assert K.kvtc_page_workspace_bytes(pages, req, _queries(q_heads=3)) == 0
    assert K.kvtc_page_workspace_bytes(pages, req, q, K.make_selection(P, 0)) == 0
    assert K.kvtc_page_workspace_bytes(None, req, q) == 0


def test_make_pages_needs_a_capacity_for_raw_pointers():
    with pytest.raises(ValueError):
        K.make_pages(P, P, 8, 16, 2, 64, K.KVTC_BF16)
    with pytest.raises(ValueError):
        K.kvtc_page_attend(_pages(), _requests(), _queries(), None, P)


def test_descriptors_have_the_headers_layout():
    import ctypes as C
    assert C.sizeof(K.kvtc_pages) == 56 and C.sizeof(K.kvtc_requests) == 40
    assert C.sizeof(K.kvtc_page_plan) == 9 * 8 + 7 * 4 + 4 and C.sizeof(K.kvtc_page_rows) == 56
    assert C.sizeof(K.kvtc_queries) == 48 and C.sizeof(K.kvtc_selection) == 24
