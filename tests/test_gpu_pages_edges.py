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


@pytest.mark.parametrize("fmt", [0, 1])
def test_arrays_whose_rows_hold_more_tokens(fmt):
    """gather and scatter move nothing and say so, on a stream of their own and in a graph too; an earlier error stays the first."""
    sh = skv.pages_shape(2, 3, 64, 16, 20, 2, 8, fmt)
    dt = torch.int16 if fmt == 0 else torch.uint8
    pages = skv.Pages(sh)
    pages.extend(ints([0, 1]), ints([50, 50]))
    pages.pool.random_(0, 255)
    pool = pages.pool.clone()
    long = torch.full((2, 2, 3, 41, 64), 7, dtype=dt, device=DEV)

    def untouched():
        torch.cuda.synchronize()
        return torch.equal(pages.pool, pool) and bool((long == 7).all())

    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream, 0):
        for call in (pages.gather, pages.scatter):
            torch.cuda.synchronize()
            call(0, 9, 40, long, stream=stream)
            assert untouched()
            with pytest.raises(skv.SkvError, match="invalid argument"):
                pages.check(stream=stream)
            pages.check()
    pages.extend(ints([0]), ints([129]))  # the row overflows
    pages.gather(0, 9, 40, long)
    assert int(pages.status.item()) == skv.ERR_PAGES
    pages.status.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pages.scatter(1, 9, 40, long)
    for _ in range(3):
        graph.replay()
        assert untouched()
        with pytest.raises(skv.SkvError, match="invalid argument"):
            pages.check()
    assert pages.gather(0, 9, 41, long) is long
    pages.check()
    assert torch.equal(long, pages.gather(0, 9, 41))


def test_arrays_of_other_shapes_are_refused():
    """A flat buffer begins with the packed symbols; any other array has exactly their number, and their size."""
    sh = skv.pages_shape(2, 3, 64, 16, 20, 2, 8)
    pages = skv.Pages(sh)
    pages.extend(ints([0]), ints([50]))
    n = 2 * 2 * 3 * 40 * 64
    want = torch.randint(0, 1000, (2, 2, 3, 40, 64), dtype=torch.int16, device=DEV)
    for x in (want, want.view(torch.bfloat16), want.view(12, -1), want.flatten(), want.flatten().view(torch.uint8),
              torch.cat([want.flatten(), want.flatten()[:99]])):
        pages.scatter(0, 3, 40, torch.zeros_like(want))
        pages.scatter(0, 3, 40, x)
        assert torch.equal(pages.gather(0, 3, 40), want)
        back = torch.zeros_like(x)
        assert pages.gather(0, 3, 40, back) is back
        assert torch.equal(back.flatten().view(torch.int16)[:n], want.flatten())
    for x in (torch.zeros(2, 2, 3, 41 * 64, dtype=torch.int16, device=DEV), torch.zeros(2, 2, 4, 40, 64, dtype=torch.int16, device=DEV),
              torch.zeros(3, 2, 3, 40, 64, dtype=torch.int16, device=DEV), torch.zeros(2, 2, 3, 40, 65, dtype=torch.int16, device=DEV),
              want.float(), want.view(torch.uint8), torch.zeros(2 * n, device=DEV), want[:, :, :, :39].contiguous(), want[:, :, :, :39]):
        for call in (pages.gather, pages.scatter):
            with pytest.raises(skv.SkvError, match="x: "):
                call(0, 3, 40, x)
    pages.check()


def test_address_0_is_the_default_stream():
    """What a call makes, and what check() waits for, is the default stream's: work enqueued there before comes first."""
    pages = skv.Pages(skv.pages_shape(1, 2, 64, 16, 20, 4, 8), q_heads=2)
    with torch.cuda.stream(torch.cuda.Stream()):
        with pages._made_on(0):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
        with pages._made_on(torch.cuda.default_stream()):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
    busy = torch.randn(4096, 4096, device=DEV)
    one, bad = ints([1]), ints([4])
    q = torch.randn(1, 2, 64, device=DEV).to(torch.bfloat16)
    pages.extend(one, ints([40]))
    pages.scatter(1, 0, 40, torch.randint(0, 1000, (1, 2, 2, 40, 64), dtype=torch.int16, device=DEV))
    want = pages.attend(0, q, one)
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-3
    out = pages.attend(0, q, one, stream=0)
    live = pages.compact(stream=0)
    pages.extend(bad, one, stream=0)
    with pytest.raises(skv.SkvError, match="invalid argument"):
        pages.check(stream=0)
    pages.check(stream=0)
    assert torch.equal(out, want) and int(live.item()) == 3


def test_the_constructor_waits_on_the_device_of_its_arrays(monkeypatch):
    """Not on the current one, which may be another as long as no call is made."""
    asked, real = [], torch.cuda.current_stream
    sh = skv.pages_shape(1, 2, 64, 16, 20, 4, 8)
    made = skv.Pages(sh)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: (asked.append(device), real(device))[1])
    skv.Pages(sh, made.pool, made.table, made.lens, made.refs)
    assert asked == [made.pool.device]


def test_tensors_dropped_after_a_call_on_a_stream():
    """Lists, queries and whole caches whose last name goes while the stream has yet to come to the call: their memory is not given out."""
    st = torch.cuda.Stream()
    sh = skv.pages_shape(1, 2, 64, 16, 20, 4, 8, skv.SYM_E4M3)
    pages = skv.Pages(sh, q_heads=2)
    with torch.cuda.stream(st):
        busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()

    def dropped(call, *tensors):
        """The call, with the stream busy before it; the tensors' addresses."""
        with torch.cuda.stream(st):
            a = busy
            for _ in range(20):
                a = a @ busy
        call(*tensors)
        assert not st.query()
        return [(t.data_ptr(), t.numel(), t.dtype) for t in tensors]

    def later(places):
        """New tensors of the same sizes lie elsewhere while the stream is at work."""
        keep = [torch.empty(n, dtype=dt, device=DEV) for _, n, dt in places for _ in range(40)]
        assert not st.query()
        assert not {p for p, _, _ in places} & {t.data_ptr() for t in keep}
        st.synchronize()

    bf = dict(dtype=torch.bfloat16, device=DEV)
    f32 = dict(dtype=torch.float32, device=DEV)
    later(dropped(lambda a, b: pages.extend(a, b, stream=st), ints([1]), ints([40])))
    later(dropped(lambda k, v, s, p, x, y: pages.store(0, k, v, s, p, x, y, stream=st), torch.ones(2, 2, 64, **bf), torch.ones(2, 2, 64, **bf),
                  ints([1, 1]), ints([3, 4]), torch.ones(2, **f32), torch.ones(2, **f32)))
    later(dropped(lambda a, b, c: pages.fork(a, b, c, stream=st), ints([1]), ints([2]), ints([33])))
    later(dropped(lambda x: pages.gather(1, 0, 40, x, stream=st), torch.zeros(1, 2, 2, 40, 64, dtype=torch.uint8, device=DEV)))
    later(dropped(lambda x: pages.scatter(2, 32, 1, x, stream=st), torch.zeros(1, 2, 2, 1, 64, dtype=torch.uint8, device=DEV)))
    assert int(pages.status.item()) == skv.ERR_ARG  # token 32 lies in a page that row 1 holds too
    pages.status.zero_()
    later(dropped(lambda q, s, x, y, o, l: pages.attend(0, q, s, k_scale=x, v_scale=y, out=o, lse=l, stream=st), torch.ones(1, 2, 64, **bf), ints([1]),
                  torch.ones(2, **f32), torch.ones(2, **f32), torch.zeros(1, 2, 64, **bf), torch.zeros(1, 2, **f32)))
    later(dropped(lambda a, b: pages.truncate(a, b, stream=st), ints([2]), ints([1])))
    later(dropped(lambda n: pages.compact(n, stream=st), ints([0])))
    pages.check()
    assert pages.lens.tolist() == [0, 40, 1, 0]
    own = [pages.pool, pages.table, pages.lens, pages.refs, pages.workspace, pages.attend_workspace, pages.status]
    row, one = ints([3]), ints([1])
    places = dropped(lambda *own: pages.extend(row, one, stream=st), *own)
    del own, pages
    later(places)
    # named by its address, as in C, the stream is not told to the allocator: the caller keeps the tensors
    pages = skv.Pages(sh)
    pages.extend(row, one, stream=st.cuda_stream)
    torch.cuda.synchronize()
    pages.check()


def test_captured_calls_that_name_their_stream():
    """The capturing stream given by name, arguments dropped within the capture; replays as the eager calls, and the cache dropped after."""
    sh = skv.pages_shape(1, 2, 64, 16, 20, 4, 8)
    x = torch.randint(0, 1000, (1, 2, 2, 40, 64), dtype=torch.int16, device=DEV)
    q = torch.randn(2, 2, 64, device=DEV).to(torch.bfloat16)
    one, two = skv.Pages(sh, q_heads=2), skv.Pages(sh, q_heads=2)
    rows, grow, out = ints([1, 2]), ints([40, 3]), torch.zeros_like(q)

    def step(p, stream):
        p.extend(rows.clone(), grow.clone(), stream=stream)
        p.scatter(1, 0, 40, x.clone(), stream=stream)
        p.attend(0, q.clone(), rows.clone(), out=out, stream=stream)
        p.truncate(rows.clone(), stream=stream)

    step(two, None)
    want = out.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(one, torch.cuda.current_stream())
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and int(one.lens.sum()) == 0
    one.check()
    del graph, one
    torch.cuda.synchronize()
    assert int(torch.zeros(4, device=DEV).sum()) == 0
