"""The paged cache's calls without a GPU: sizes, and what is refused before anything is launched."""
import ctypes as C

import pytest
import torch

from lossless_kv_cache_scalar_amd import build as B
from lossless_kv_cache_scalar_amd import skv


@pytest.fixture(scope="module")
def lib():
    if not B.is_built():
        B.build()
    return skv.load()


def test_sizes(lib):
    sh = skv.pages_shape(3, 5, 64, 32, 7, 4, 9)
    assert skv.pages_pool_size(sh) == 3 * 7 * 2 * 5 * 32 * 64 * 2
    assert skv.pages_pool_size(skv.pages_shape(3, 5, 64, 32, 7, 4, 9, skv.SYM_E4M3)) == 3 * 7 * 2 * 5 * 32 * 64
    assert skv.pages_workspace_size(sh) > 0
    a = skv.attend_workspace_size(sh, 10)
    assert a > 0 and a == skv.attend_workspace_size(skv.pages_shape(3, 5, 64, 32, 70000, 4000, 900), 10)


@pytest.mark.parametrize("bad,code", [
    ((0, 1, 64, 16, 1, 1, 1), skv.ERR_ARG), ((1, 0, 64, 16, 1, 1, 1), skv.ERR_ARG), ((1, 1, 96, 16, 1, 1, 1), skv.ERR_UNSUPPORTED),
    ((1, 1, 64, 8, 1, 1, 1), skv.ERR_ARG), ((1, 1, 64, 48, 1, 1, 1), skv.ERR_ARG), ((1, 1, 64, 512, 1, 1, 1), skv.ERR_ARG),
    ((1, 1, 64, 16, 0, 1, 1), skv.ERR_ARG), ((1, 1, 64, 16, 1, 0, 1), skv.ERR_ARG), ((1, 1, 64, 16, 1, 1, 0), skv.ERR_ARG),
    ((1, 1, 64, 16, 1, 1, 1 << 27), skv.ERR_ARG), ((1, 1, 64, 16, 1, 1, 1, 2), skv.ERR_ARG),
    ((1 << 20, 1 << 16, 512, 256, 1 << 30, 1, 1), skv.ERR_ARG)])
def test_bad_shapes_rejected(lib, bad, code):
    n = C.c_size_t(0)
    sh = skv.pages_shape(*bad)
    assert lib.skv_pages_pool_size(C.byref(sh), C.byref(n)) == code
    assert lib.skv_pages_workspace_size(C.byref(sh), C.byref(n)) == code
    assert lib.skv_attend_workspace_size(C.byref(sh), 8, C.byref(n)) == code
    p = skv.SkvPages(4096, 4096, 4096, 4096)
    assert lib.skv_pages_reset(C.byref(sh), C.byref(p), None) == code
    assert lib.skv_attend(C.byref(sh), C.byref(p), 0, 4096, 64, 1, 1.0, None, None, 4096, 1, 4096, None, 4096, 1 << 30, 4096, None) == code


def test_reserved_word_is_zero(lib):
    n = C.c_size_t(0)
    sh = skv.pages_shape(1, 1, 64, 16, 1, 1, 1)
    sh.reserved = 1
    assert lib.skv_pages_pool_size(C.byref(sh), C.byref(n)) == skv.ERR_ARG


P = 4096  # an address that no refused call touches


def _refused(fn, good, changes):
    """Each change alone is refused with SKV_ERR_ARG (the arguments as given would launch, so they are never passed whole)."""
    for at, value in changes:
        args = list(good)
        args[at] = value
        assert fn(*args) == skv.ERR_ARG, (at, value)


def test_page_calls_check_their_arguments(lib):
    sh = skv.pages_shape(2, 2, 64, 16, 8, 4, 8)
    S, good = C.byref(sh), C.byref(skv.SkvPages(P, P, P, P))
    ws = skv.pages_workspace_size(sh)
    holed = [C.byref(skv.SkvPages(*[None if i == j else P for i in range(4)])) for j in range(4)]
    odd = [C.byref(skv.SkvPages(P + 8, P, P, P)), C.byref(skv.SkvPages(P, P + 2, P, P)), C.byref(skv.SkvPages(P, P, P, P + 4))]
    pages = [(1, x) for x in [None] + holed + odd]
    # shape, pages, seqs, n_new, n, workspace, bytes, status, stream
    _refused(lib.skv_pages_extend, [S, good, P, P, 3, P, ws, P, None],
             pages + [(0, None), (2, None), (3, None), (3, P + 1), (4, -1), (4, 5), (5, None), (5, P + 8), (6, ws - 1), (7, None), (7, P + 2)])
    _refused(lib.skv_pages_truncate, [S, good, P, None, 3, P, ws, P, None],
             pages + [(0, None), (2, None), (3, P + 1), (4, -1), (4, 5), (5, None), (6, ws - 1), (7, None)])
    _refused(lib.skv_pages_fork, [S, good, P, P, None, 3, P, ws, P, None],
             pages + [(0, None), (2, None), (3, None), (4, P + 1), (5, -1), (5, 5), (6, None), (7, ws - 1), (8, None)])
    _refused(lib.skv_pages_compact, [S, good, P, P, ws, P, None], pages + [(0, None), (2, None), (3, None), (4, ws - 1), (5, None)])
    # an empty list does nothing
    assert lib.skv_pages_extend(S, good, None, None, 0, P, ws, P, None) == skv.OK
    assert lib.skv_pages_fork(S, good, None, None, None, 0, P, ws, P, None) == skv.OK
    assert lib.skv_pages_truncate(S, good, None, None, 0, P, ws, P, None) == skv.OK
    # shape, pages, layer, k, k_stride, v, v_stride, k_scale, v_scale, seqs, pos, n, status, stream
    _refused(lib.skv_pages_store, [S, good, 1, P, 128, P, 128, None, None, P, P, 3, P, None],
             pages + [(2, -1), (2, 2), (3, None), (3, P + 8), (4, 127), (4, 120), (4, 132), (4, 1 << 62), (5, None), (6, 64), (7, P), (8, P),
                      (9, None), (10, None), (11, -1), (12, None)])
    assert lib.skv_pages_store(S, good, 1, None, 128, None, 128, None, None, None, None, 0, P, None) == skv.OK
    # shape, pages, seq, first, tokens, x, status, stream
    for fn in (lib.skv_pages_gather, lib.skv_pages_scatter):
        _refused(fn, [S, good, 1, 3, 20, P, P, None],
                 pages + [(2, -1), (2, 4), (3, -1), (3, 129), (4, -1), (4, 126), (5, None), (5, P + 8), (6, None)])
        assert fn(S, good, 1, 3, 0, None, P, None) == skv.OK


def test_attend_checks_its_arguments(lib):
    sh = skv.pages_shape(2, 2, 64, 16, 8, 4, 8)
    S, good = C.byref(sh), C.byref(skv.SkvPages(P, P, P, P))
    ws = skv.attend_workspace_size(sh, 6)
    holed = [(1, C.byref(skv.SkvPages(*[None if i == j else P for i in range(4)]))) for j in range(4)]
    # shape, pages, layer, q, q_stride, q_heads, scale, k_scale, v_scale, seqs, n, out, lse, workspace, bytes, status, stream
    args = [S, good, 1, P, 384, 6, 0.125, None, None, P, 3, P, None, P, ws, P, None]
    _refused(lib.skv_attend, args, holed + [
        (0, None), (1, None), (2, -1), (2, 2), (3, None), (3, P + 8), (4, 376), (4, 388), (4, 1 << 62), (5, 0), (5, -2), (5, 5),
        (6, float("nan")), (6, float("inf")), (7, P), (8, P), (9, None), (10, -1), (10, 65537), (11, None), (11, P + 2), (12, P + 2), (13, None),
        (13, P + 8), (14, ws - 1), (15, None)])
    args[10] = 0
    assert lib.skv_attend(*args) == skv.OK


def test_binding_refuses_other_types_and_devices(lib):
    """Arrays that the library would read wrongly, or on the host, are refused by name."""
    sh = skv.pages_shape(1, 2, 64, 16, 8, 4, 8)
    pool = torch.zeros(1, 8, 2, 2, 16, 64, dtype=torch.int16)
    table = torch.zeros(4, 8, dtype=torch.int32)
    lens, refs = torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(skv.SkvError, match="together"):
        skv.Pages(sh, pool=pool)
    with pytest.raises(skv.SkvError, match="pool"):
        skv.Pages(sh, pool[:, :7], table, lens, refs)
    with pytest.raises(skv.SkvError, match="table"):
        skv.Pages(sh, pool, table.long(), lens, refs)
    with pytest.raises(skv.SkvError, match="contiguous"):
        skv.Pages(sh, pool, torch.zeros(8, 4, dtype=torch.int32).t(), lens, refs)
    with pytest.raises(skv.SkvError, match="table"):
        skv.Pages(sh, pool, torch.zeros(4, 16, dtype=torch.int32), lens, refs)  # rows of another length
    with pytest.raises(skv.SkvError, match="refs"):
        skv.Pages(sh, pool, table, lens, torch.zeros(9, dtype=torch.int32))
    with pytest.raises(skv.SkvError, match="pool"):
        skv.Pages(sh, pool.view(torch.uint8), table, lens, refs)
    with pytest.raises(skv.SkvError, match="pool: on cpu"):
        skv.Pages(sh, pool, table, lens, refs)
