"""Branches of the page calls that short rows and short lists do not reach: growth by more free pages than LDS holds,
refused lists of more places than a workgroup has threads, rows of more pages than a wave or a workgroup has threads."""
import random

import pytest

from lossless_kv_cache_scalar_amd import skv
from gpu_util import ensure_built
from pages_util import Model
from test_gpu_pages import both, fill, ints, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def holed(n_pages, max_pages, seed, rows=6):
    """A cache with holes all over its pool: pages given to two rows in turn, one of which is freed."""
    sh = skv.pages_shape(1, 1, 8, 16, n_pages, rows, max_pages, skv.SYM_E4M3)
    pages, m = skv.Pages(sh), Model(sh)
    fill(pages, m, seed)
    rng = random.Random(seed)
    for _ in range(12):
        both(pages, m, "extend", [0, 1], [rng.randint(1, 40) * 16, rng.randint(1, 60) * 16])
    both(pages, m, "truncate", [1], None)
    same(pages, m)
    return pages, m


@pytest.mark.parametrize("need", [2047, 2048, 2049, 4095, 4097, 6000])
@pytest.mark.parametrize("rows", [1, 3])
def test_growth_by_thousands_of_pages(need, rows):
    """A few rows take that many pages at once, a copy of a shared last page among them."""
    pages, m = holed(9000, 6100, need)
    both(pages, m, "extend", [2], [5])
    both(pages, m, "fork", [2], [3])
    cut = [need] if rows == 1 else [need // 3, 1, need - need // 3 - 1]
    # row 3's first page is its copy; what it grows by ends inside its last page
    grow = [(cut[0] - 1) * 16 + 11] + [k * 16 for k in cut[1:]]
    assert both(pages, m, "extend", [3, 4, 5][:rows], grow) == skv.OK
    assert sum(m.pages(m.lens[s]) for s in (3, 4, 5)) == need
    same(pages, m)
    assert m.table[3, 0] != m.table[2, 0]
    free = int((m.refs == 0).sum())
    assert both(pages, m, "extend", [2, 5], [0, free * 16 + 1]) == skv.ERR_PAGES
    same(pages, m)
    assert both(pages, m, "truncate", [4, 3], None) == skv.OK
    assert int(pages.compact().item()) == m.compact()
    same(pages, m)


def test_growth_takes_every_page():
    pages, m = holed(5001, 5001, 7)
    free = int((m.refs == 0).sum())
    assert both(pages, m, "extend", [4, 1], [16 * (free - 2000) + 1, 16 * 2000]) == skv.ERR_PAGES
    assert both(pages, m, "extend", [4, 1], [16 * (free - 2000), 16 * 2000 - 3]) == skv.OK
    assert (m.refs == 1).all()
    same(pages, m)


@pytest.mark.parametrize("n", [1024, 1025, 1500, 2999])
def test_long_lists_are_refused_whole(n):
    """One place of a long list breaks a rule: nothing changes, wherever the place is."""
    sh = skv.pages_shape(1, 1, 8, 16, 6000, 3000, 3, skv.SYM_E4M3)
    pages, m = skv.Pages(sh), Model(sh)
    fill(pages, m, n)
    rng = random.Random(n)
    rows = list(range(3000))
    rng.shuffle(rows)
    both(pages, m, "extend", rows[:1300], [rng.choice([1, 16, 21]) for _ in range(1300)])
    held, free = rows[:1300], rows[1300:]
    k = min(n, 1700)

    def spoiled(good, change):
        """The list with one place's value taken from `change`, at several places of it."""
        for at in (0, 1, 63, 64, n // 2, n - 1):
            if at < len(good):
                bad = list(good)
                bad[at] = change(bad, at)
                yield bad

    def other(v, at):
        return v[(at + 1 + rng.randrange(len(v) - 1)) % len(v)]

    def refuse(name, *args):
        assert both(pages, m, name, *args) == skv.ERR_ARG, (name,)

    grow = [rng.choice([0, 1, 5]) for _ in range(n)]
    listed = rows[:n]
    for bad in list(spoiled(listed, other)) + list(spoiled(listed, lambda v, at: 3000)):
        refuse("extend", bad, grow)
        refuse("truncate", bad, None)
    for bad in spoiled(grow, lambda v, at: -1):
        refuse("extend", listed, bad)
    keep = [rng.randint(0, int(m.lens[s])) for s in listed]
    for bad in spoiled(keep, lambda v, at: -1):
        refuse("truncate", listed, bad)
    for bad in spoiled(keep, lambda v, at: int(m.lens[listed[at]]) + 1):
        refuse("truncate", listed, bad)
    src, dst = [rng.choice(held) for _ in range(k)], free[:k]
    for bad in list(spoiled(dst, other)) + list(spoiled(dst, lambda v, at: held[0])) + list(spoiled(dst, lambda v, at: 3000)):
        refuse("fork", src, bad, None)
    for bad in list(spoiled(src, lambda v, at: dst[(at * 7 + 3) % k])) + list(spoiled(src, lambda v, at: 3000)):
        refuse("fork", bad, dst, None)
    part = [rng.randint(0, int(m.lens[s])) for s in src]
    for bad in list(spoiled(part, lambda v, at: -1)) + list(spoiled(part, lambda v, at: int(m.lens[src[at]]) + 1)):
        refuse("fork", src, dst, bad)
    same(pages, m)
    # with the place padded the rest is done
    pad = [s if i != n // 2 else -1 for i, s in enumerate(listed)]
    assert both(pages, m, "extend", pad, grow) == skv.OK
    same(pages, m)
    free = [s for s in rows if m.lens[s] == 0]
    k = min(k, len(free))
    assert both(pages, m, "fork", [s if i % 97 else -1 for i, s in enumerate(src[:k])], free[:k]) == skv.OK
    same(pages, m)
    assert both(pages, m, "truncate", pad, None) == skv.OK
    same(pages, m)


@pytest.mark.parametrize("forks", [1, 5, 6, 20])
def test_rows_of_many_pages(forks):
    """Rows of 65, 300 and 700 pages forked whole and in part, cut and freed, in one launch (up to 5 rows here) and in two."""
    sh = skv.pages_shape(1, 1, 8, 16, 2000 + 2 * forks, 3 + forks, 700, skv.SYM_E4M3)
    pages, m = skv.Pages(sh), Model(sh)
    fill(pages, m, forks)
    rng = random.Random(forks)
    assert both(pages, m, "extend", [0, 1, 2], [65 * 16, 300 * 16 - 7, 700 * 16]) == skv.OK
    dst = list(range(3, 3 + forks))
    src = [(2, 0, 1)[i % 3] for i in range(forks)]
    assert both(pages, m, "fork", src, dst, None) == skv.OK
    same(pages, m)
    assert both(pages, m, "truncate", dst, None) == skv.OK
    same(pages, m)
    for trial in range(3):
        part = [rng.choice([0, 1, 64 * 16, 64 * 16 + 1, 65 * 16, 255 * 16 + 1, 256 * 16, 257 * 16, 300 * 16 - 7, 513 * 16, 700 * 16]) for _ in src]
        part = [min(n, int(m.lens[s])) for n, s in zip(part, src)]
        assert both(pages, m, "fork", src, dst, part) == skv.OK
        same(pages, m)
        assert both(pages, m, "extend", dst, [min(1, 700 * 16 - n) for n in part]) == skv.OK  # shared last pages are copied
        same(pages, m)
        assert both(pages, m, "truncate", dst, [rng.randint(0, int(m.lens[s])) for s in dst]) == skv.OK
        same(pages, m)
        assert both(pages, m, "truncate", dst, None) == skv.OK
        same(pages, m)
    assert both(pages, m, "fork", src, dst, None) == skv.OK
    assert both(pages, m, "truncate", [0, 1, 2], None) == skv.OK  # the forks alone hold the pages now
    same(pages, m)
    assert int(pages.compact().item()) == m.compact()
    same(pages, m)
