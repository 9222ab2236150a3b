"""Attention over pages where its split changes: many query heads to a KV head, many KV heads, the longest lists,
long rows that many workgroups share, and sequences that share pages."""
import pytest
import torch

from lossless_kv_cache_scalar_amd import skv
from gpu_util import DEV, ensure_built
from test_gpu_attend import Case, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("D,kv_heads,group", [(64, 2, 64), (64, 2, 65), (128, 1, 128), (128, 2, 129), (256, 1, 100), (512, 1, 65), (8, 3, 70),
                                              (64, 1, 1000)])
def test_many_query_heads_to_a_kv_head(fmt, D, kv_heads, group):
    """More heads than a workgroup's waves take at once (64, or 32 at 512 channels): a KV head then has several rows."""
    lens = [0, 1, 33, 64, 700, 2049]
    c = Case(fmt, lens, D, 16, kv_heads, kv_heads * group, layers=1)
    seqs = [5, -1, 0, 3, 1, 4, 2, 5]
    q = c.q(len(seqs))
    out, lse = c.attend(0, q, seqs)
    c.compare(0, q, seqs, out, lse)


@pytest.mark.parametrize("fmt,kv_heads,group", [(0, 40, 1), (1, 37, 3), (0, 300, 2), (1, 9, 17)])
def test_many_kv_heads(fmt, kv_heads, group):
    c = Case(fmt, [130, 1, 0, 517], 64, 32, kv_heads, kv_heads * group, layers=1)
    q = c.q(4)
    out, lse = c.attend(0, q, [3, 0, 1, 2])
    c.compare(0, q, [3, 0, 1, 2], out, lse)


@pytest.mark.parametrize("rows", [65535, 65536])
def test_the_longest_lists(rows):
    """Long rows at both ends and in the middle of a list whose other places are padded, empty or short."""
    c = Case(0, [1500, 5, 0, 2500, 40], 64, 64, 1, 2, layers=1)
    seqs = [(-1, 2, 1, 4, -1, 1)[i % 6] for i in range(rows)]
    for at, s in ((0, 0), (rows // 2, 3), (rows - 1, 0), (rows - 64, 3)):
        seqs[at] = s
    q = c.q(rows)
    out, lse = c.attend(0, q, seqs)
    pick = sorted({0, 1, 2, 3, rows // 2 - 1, rows // 2, rows // 2 + 1, rows - 65, rows - 64, rows - 63, rows - 2, rows - 1} |
                  set(range(5, rows, 611)))
    c.compare(0, q[pick], [seqs[i] for i in pick], out[pick], lse[pick])


@pytest.mark.parametrize("fmt,D,kv_heads,group,n", [(0, 64, 1, 3, 300001), (1, 128, 1, 16, 262144), (1, 64, 2, 20, 100003), (0, 512, 1, 1, 65537),
                                                    (0, 16, 1, 40, 200000)])
def test_long_rows(fmt, D, kv_heads, group, n):
    """One long sequence beside a short one: hundreds of workgroups to a row, and their join."""
    c = Case(fmt, [n, 3], D, 16, kv_heads, kv_heads * group, layers=1)
    q = c.q(2)
    out, lse = c.attend(0, q, [0, 1])
    c.compare(0, q, [0, 1], out, lse)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("group", [4, 20])
def test_forks_of_a_prompt(fmt, group):
    """Sequences that share a prompt's pages, whole, in part and grown, read the same keys and values."""
    D, heads, n = 128, 2, 1003
    sh = skv.pages_shape(1, heads, D, 16, 200, 12, 80, fmt)
    c = Case(fmt, [1], D, 16, heads, heads * group, layers=1)  # scales, queries and the comparison
    c.pages = p = skv.Pages(sh, q_heads=heads * group)
    p.pool.fill_(0x7FC0 if fmt == skv.SYM_BF16 else 0x7F)
    x = torch.randn(1, 2, heads, n + 30, D, generator=c.g)
    x = x.to(torch.bfloat16).view(torch.int16) if fmt == 0 else x.to(torch.float8_e4m3fn).view(torch.uint8)
    p.extend(ints([0]), ints([n]))
    p.scatter(0, 0, n, x[:, :, :, :n].contiguous().to(DEV))
    cut = [n, 1, 16, 17, 500, 992, n, n, 0]
    p.fork(ints([0] * 9), ints(range(1, 10)), ints(cut))
    c.x, c.lens = {0: x[:, :, :, :n]}, [n] + cut + [0]
    for s, k in enumerate(cut):
        c.x[s + 1] = x[:, :, :, :k]
    for s, more in ((7, 1), (8, 30), (2, 5)):  # each grows by the tokens of the end of x
        p.extend(ints([s]), ints([more]))
        new = x[:, :, :, n + 30 - more:]
        p.scatter(s, c.lens[s], more, new.contiguous().to(DEV))
        c.x[s] = torch.cat([c.x[s], new], 3)
        c.lens[s] += more
    seqs = [8, 3, -1, 0, 7, 1, 9, 2, 4, 5, 6, 0, 10]
    c.x[10] = x[:, :, :, :0]
    q = c.q(len(seqs))
    out, lse = c.attend(0, q, seqs)
    c.compare(0, q, seqs, out, lse)
