"""The paged cache's calls at sizes and with arguments where a launch, a binding or a branch of a plan changes."""
import pytest
import torch

from lossless_kv_cache_scalar_amd import skv
from gpu_util import DEV, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device=DEV)


def test_gather_scatter_of_more_work_than_a_launch_takes():
    """2^24 + 2048 blocks of 64 tokens (2^24 workgroups of 256 threads are no launch), three to a row, so that the launches part inside a row."""
    layers, heads, P, D, n, first = 2731, 1024, 16, 8, 130, 5
    sh = skv.pages_shape(layers, heads, D, P, 9, 1, 9, skv.SYM_E4M3)
    pages = skv.Pages(sh)
    pages.extend(ints([0]), ints([first + n]))
    pool = pages.pool
    for l in range(0, layers, 100):  # in parts: torch's own launches are kept small
        pool[l:l + 100].random_(0, 256)
    order = pages.table[0].long()

    def rows(l):  # [2][heads][9 * P][D] of a layer, in the sequence's order
        return pool[l, order].permute(1, 2, 0, 3, 4).reshape(2, heads, 9 * P, D)

    x = pages.gather(0, first, n)
    pages.check()
    for l in range(layers):
        assert torch.equal(x[l], rows(l)[:, :, first:first + n]), l
    before = pool.clone()
    for l in range(layers):
        x[l].bitwise_not_()
    pages.scatter(0, first, n, x)
    pages.check()
    for l in range(layers):
        want = before[l, order].permute(1, 2, 0, 3, 4).reshape(2, heads, 9 * P, D).clone()
        want[:, :, first:first + n].bitwise_not_()
        assert torch.equal(rows(l), want), l


def test_store_of_more_work_than_a_launch_takes():
    """2^26 + 5 tokens of 520 values, eight to a workgroup: all but the first, the last and those about the launches' border are padding."""
    heads, D, n = 65, 8, (1 << 26) + 5
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of GPU memory")
    x = torch.empty(n, heads, D, dtype=torch.bfloat16, device=DEV)  # keys and values alike
    at = [0, 1, (1 << 26) - 1, 1 << 26, (1 << 26) + 4]
    some = torch.randn(len(at), heads, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    seqs, pos = torch.full((n,), -1, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    for j, i in enumerate(at):
        x[i], seqs[i], pos[i] = some[j], 0, 3 * j
    pages = skv.Pages(skv.pages_shape(1, heads, D, 16, 1, 1, 1))
    pages.pool.zero_()
    pages.extend(ints([0]), ints([16]))
    pages.store(0, x, x, seqs, pos)
    pages.check()
    want = torch.zeros(16, heads, D, dtype=torch.bfloat16, device=DEV)
    want[[3 * j for j in range(len(at))]] = some
    for which in (0, 1):
        assert torch.equal(pages.pool[0, 0, which].transpose(0, 1), want.view(torch.int16))
